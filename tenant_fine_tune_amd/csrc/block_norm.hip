// Norms before and after a block with its gate and residual scale, weights
// per variant (bitdelta_block_norm).
//
//   y = b * rsqrt(mean b^2 + eps) * w_post;  r' = r + scale * act(g) * y
//   x = bf16(r' * rsqrt(mean r'^2 + eps) * w_pre)
//
// One workgroup per token keeps the row in registers between the two sums, so
// every input is read once and every output written once: memory bound.  All
// loads of a row are issued before the first sum is waited for; the second
// sum needs only what is in registers.  Sums and norms are fp32, r' enters the
// second norm before its rounding.  4096 x 8192 bf16 takes 55 us (4.9 TB/s),
// 4099 x 8192 with an fp32 residual and a gate 93 us (5.0 TB/s; a copy of 2 GiB
// reaches 5.4), four rows 5 us, of which the launch is most.
#include "bd_device.h"
#include "decoder_launch.h"

namespace bd {
namespace {

// Eight consecutive elements as loaded, of which n (1..8) exist, the others
// zero.  Global memory takes 16-byte accesses at any element alignment, so one
// form serves odd widths and strides too.  Outputs are stored past the L2, whose
// lines the reader, on another die, would not find (512 x 8192: 11.8 -> 10.1 us,
// 2048 x 5000: 30 -> 26.5; two norms with the kernels that write and read around
// them: 512 rows 37.4 -> 35.8, 2048 88.8 -> 93.3, 4099 in fp32 278 -> 269).
typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct Eight;

template <>
struct Eight<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t *p, int n)
    {
        if (n == 8) {
            w = *reinterpret_cast<const u32x4a2 *>(p);
            return;
        }
        w = (u32x4){0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? hi_f32(w[i >> 1]) : lo_f32(w[i >> 1]); }
    __device__ __forceinline__ void set(const float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void store(uint16_t *p, int n) const
    {
        if (n == 8) {
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4a2 *>(p));
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
};

template <>
struct Eight<float> {
    float f[8];
    __device__ __forceinline__ void load(const float *p, int n)
    {
        if (n == 8) {
            const u32x4 a = *reinterpret_cast<const u32x4a4 *>(p), b = *reinterpret_cast<const u32x4a4 *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = __uint_as_float(a[i]), f[4 + i] = __uint_as_float(b[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = i < n ? p[i] : 0.0f;
    }
    __device__ __forceinline__ float get(int i) const { return f[i]; }
    __device__ __forceinline__ void set(const float *g)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = g[i];
    }
    __device__ __forceinline__ void store(float *p, int n) const
    {
        if (n == 8) {
            u32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = __float_as_uint(f[i]), b[i] = __float_as_uint(f[4 + i]);
            __builtin_nontemporal_store(a, reinterpret_cast<u32x4a4 *>(p));
            __builtin_nontemporal_store(b, reinterpret_cast<u32x4a4 *>(p + 4));
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = f[i];
    }
};

// Sum over the workgroup; every thread gets it.  `part` holds one float a wave.
__device__ __forceinline__ float sum_all(float v, float *part)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    const int waves = blockDim.x >> 6;
    if (waves == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    // each wave sums the parts for itself
    const int lane = threadIdx.x & 63;
    v = lane < waves ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    return __shfl(v, 0);
}

// C groups of eight columns a thread.  Inputs stay as loaded until they are
// used (half the registers for bf16), so that 32 waves fit a CU.
template <int C, typename RT, typename WT>
__global__ __launch_bounds__(1024, C == 1 ? 8 : 4) void block_norm_rows(NormArgs a)
{
    __shared__ float part[2][16];
    const int64_t i = blockIdx.y * kTokensAcross + blockIdx.x;
    if (i >= a.m)
        return;
    const int d = a.d, T = blockDim.x;
    const int v = a.ids ? a.ids[i] : 0;
    const bool known = (unsigned)v < (unsigned)a.n_variants;
    const RT *res = static_cast<const RT *>(a.residual) + i * a.residual_stride;
    const bool blk = a.block && known, gated = blk && a.gate, posted = blk && a.post_weight;
    const bool wants_x = a.pre_weight != nullptr, pre = wants_x && known;
    const int64_t wrow = known ? (int64_t)v * d : 0;

    Eight<RT> r[C];
    Eight<uint16_t> b[C], g[C];
    Eight<WT> wo[C], wi[C];
    int n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * T + (int)threadIdx.x) * 8;
        n[c] = min(max(d - at, 0), 8);
        if (n[c] > 0) {
            r[c].load(res + at, n[c]);
            if (blk)
                b[c].load(a.block + i * a.block_stride + at, n[c]);
            if (gated)
                g[c].load(a.gate + i * a.gate_stride + at, n[c]);
            if (posted)
                wo[c].load(static_cast<const WT *>(a.post_weight) + wrow + at, n[c]);
            if (pre)
                wi[c].load(static_cast<const WT *>(a.pre_weight) + wrow + at, n[c]);
        }
    }
    float k = a.scale;
    if (posted) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n[c] > 0)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s = fmaf(b[c].get(j), b[c].get(j), s);
        k *= 1.0f / sqrtf(sum_all(s, part[0]) / (float)d + a.eps);
    }
    float s = 0.0f, x[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (n[c] > 0) {
            const int at = (c * T + (int)threadIdx.x) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[c][j] = r[c].get(j);
                if (blk) {
                    float y = b[c].get(j) * k;
                    if (posted)
                        y *= wo[c].get(j);
                    if (gated) {
                        const float z = g[c].get(j);
                        // exp(-z) past the range gives sigmoid 0 (and silu -0) as it should
                        const float sig = 1.0f / (1.0f + __expf(-z));
                        y *= a.gate_act == BD_GATE_NONE ? z : a.gate_act == BD_GATE_SIGMOID ? sig : z * sig;
                    }
                    x[c][j] += y;
                }
                // columns past the row's end are zero, also with a gate (their block is)
                s = fmaf(x[c][j], x[c][j], s);
            }
            if (a.residual_out) {
                Eight<RT> out;
                out.set(x[c]);
                out.store(static_cast<RT *>(a.residual_out) + i * a.out_stride + at, n[c]);
            }
        }
    if (!wants_x)
        return;
    k = pre ? 1.0f / sqrtf(sum_all(s, part[1]) / (float)d + a.eps) : 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (n[c] > 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[c][j] = pre ? x[c][j] * k * wi[c].get(j) : 0.0f;
            Eight<uint16_t> out;
            out.set(x[c]);
            out.store(a.x + i * (int64_t)d + (c * T + (int)threadIdx.x) * 8, n[c]);
        }
}

template <int C>
void start(const NormArgs &a, hipStream_t s)
{
    // as many waves as the row has groups of 512 columns
    const int threads = (a.d + 512 * C - 1) / (512 * C) * 64;
    const dim3 grid((unsigned)(a.m < kTokensAcross ? a.m : kTokensAcross),
                    (unsigned)((a.m + kTokensAcross - 1) / kTokensAcross));
    if (a.residual_f32) {
        if (a.weight_f32)
            block_norm_rows<C, float, float><<<grid, threads, 0, s>>>(a);
        else
            block_norm_rows<C, float, uint16_t><<<grid, threads, 0, s>>>(a);
    } else {
        if (a.weight_f32)
            block_norm_rows<C, uint16_t, float><<<grid, threads, 0, s>>>(a);
        else
            block_norm_rows<C, uint16_t, uint16_t><<<grid, threads, 0, s>>>(a);
    }
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t s)
{
    // two groups a thread: half the waves to add up (4096 x 8192 bf16: 65 -> 55 us,
    // 4099 x 8192 fp32, gated: 103 -> 98 us); one where a row is a few waves
    if (a.d <= 2048)
        start<1>(a, s);
    else if (a.d <= 16384)
        start<2>(a, s);
    else
        start<4>(a, s);
    return hipGetLastError();
}

}  // namespace bd
