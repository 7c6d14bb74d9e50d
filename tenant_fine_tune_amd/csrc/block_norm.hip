// Norms before and after a block with its gate and residual scale, weights
// per variant (bitdelta_block_norm).
//
//   y = b * rsqrt(mean b^2 + eps) * w_post;  r' = r + scale * act(g) * y
//   x = bf16(r' * rsqrt(mean r'^2 + eps) * w_pre)
//
// One workgroup per token keeps the row in registers between the two sums, so
// every input is read once and every output written once: memory bound.  All
// loads of a row are issued before the first sum is waited for; the second
// sum needs only what is in registers.
#include "bd_device.h"
#include "decoder_launch.h"

namespace bd {
namespace {

// Eight consecutive elements, of which n (1..8) exist.  Global memory takes
// 16-byte accesses at any element alignment, so one form serves odd widths
// and strides too.
typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void load8(const uint16_t *p, int n, float *f)
{
    if (n == 8) {
        const u32x4a2 w = *reinterpret_cast<const u32x4a2 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = lo_f32(w[i]);
            f[2 * i + 1] = hi_f32(w[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = i < n ? lo_f32(p[i]) : 0.0f;
}

__device__ __forceinline__ void load8(const float *p, int n, float *f)
{
    if (n == 8) {
        const u32x4a4 a = *reinterpret_cast<const u32x4a4 *>(p), b = *reinterpret_cast<const u32x4a4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __uint_as_float(a[i]);
            f[4 + i] = __uint_as_float(b[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = i < n ? p[i] : 0.0f;
}

__device__ __forceinline__ void store8(uint16_t *p, int n, const float *f)
{
    if (n == 8) {
        u32x4a2 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<u32x4a2 *>(p) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n)
            p[i] = to_bf16(f[i]);
}

__device__ __forceinline__ void store8(float *p, int n, const float *f)
{
    if (n == 8) {
        u32x4a4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(f[i]);
            b[i] = __float_as_uint(f[4 + i]);
        }
        *reinterpret_cast<u32x4a4 *>(p) = a;
        *reinterpret_cast<u32x4a4 *>(p + 4) = b;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n)
            p[i] = f[i];
}

// Sum over the workgroup; every thread gets it.  `part` holds one float a wave.
template <int T>
__device__ __forceinline__ float sum_all(float v, float *part)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    if (T == 64)
        return v;
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i)
        v += part[i];
    return v;
}

template <int T, int C, typename RT, typename WT>
__global__ __launch_bounds__(T) void block_norm_rows(NormArgs a)
{
    __shared__ float part[2][T / 64];
    const int64_t i = blockIdx.x;
    const int d = a.d;
    const int v = a.ids ? a.ids[i] : 0;
    const bool known = (unsigned)v < (unsigned)a.n_variants;
    const RT *res = static_cast<const RT *>(a.residual) + i * a.residual_stride;
    const bool blk = a.block && known, gated = blk && a.gate, posted = blk && a.post_weight;
    const bool wants_x = a.pre_weight != nullptr, pre = wants_x && known;
    const int64_t wrow = known ? (int64_t)v * d : 0;

    float r[C][8], b[C][8], g[C][8], wo[C][8], wi[C][8];
    int n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * T + (int)threadIdx.x) * 8;
        n[c] = min(max(d - at, 0), 8);
        if (n[c] > 0) {
            load8(res + at, n[c], r[c]);
            if (blk)
                load8(a.block + i * a.block_stride + at, n[c], b[c]);
            if (gated)
                load8(a.gate + i * a.gate_stride + at, n[c], g[c]);
            if (posted)
                load8(static_cast<const WT *>(a.post_weight) + wrow + at, n[c], wo[c]);
            if (pre)
                load8(static_cast<const WT *>(a.pre_weight) + wrow + at, n[c], wi[c]);
        }
    }
    if (blk) {
        float k = a.scale;
        if (posted) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (n[c] > 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        s = fmaf(b[c][j], b[c][j], s);
            k *= 1.0f / sqrtf(sum_all<T>(s, part[0]) / (float)d + a.eps);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n[c] > 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float y = b[c][j] * k;
                    if (posted)
                        y *= wo[c][j];
                    if (gated) {
                        const float z = g[c][j];
                        // exp(-z) past the range gives sigmoid 0 (and silu -0) as it should
                        const float sig = 1.0f / (1.0f + __expf(-z));
                        y *= a.gate_act == BD_GATE_NONE ? z : a.gate_act == BD_GATE_SIGMOID ? sig : z * sig;
                    }
                    r[c][j] += y;
                }
    }
    if (a.residual_out) {
        RT *out = static_cast<RT *>(a.residual_out) + i * a.out_stride;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n[c] > 0)
                store8(out + (c * T + (int)threadIdx.x) * 8, n[c], r[c]);
    }
    if (!wants_x)
        return;
    float k = 0.0f;
    if (pre) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n[c])
                    s = fmaf(r[c][j], r[c][j], s);
        k = 1.0f / sqrtf(sum_all<T>(s, part[1]) / (float)d + a.eps);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (n[c] > 0) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = pre ? r[c][j] * k * wi[c][j] : 0.0f;
            store8(a.x + i * (int64_t)d + (c * T + (int)threadIdx.x) * 8, n[c], x);
        }
}

template <int T, int C>
void start(const NormArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)a.m);
    if (a.residual_f32) {
        if (a.weight_f32)
            block_norm_rows<T, C, float, float><<<grid, T, 0, s>>>(a);
        else
            block_norm_rows<T, C, float, uint16_t><<<grid, T, 0, s>>>(a);
    } else {
        if (a.weight_f32)
            block_norm_rows<T, C, uint16_t, float><<<grid, T, 0, s>>>(a);
        else
            block_norm_rows<T, C, uint16_t, uint16_t><<<grid, T, 0, s>>>(a);
    }
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t s)
{
    if (a.d <= 512)
        start<64, 1>(a, s);
    else if (a.d <= 2048)
        start<256, 1>(a, s);
    else if (a.d <= 8192)
        start<1024, 1>(a, s);
    else if (a.d <= 16384)
        start<1024, 2>(a, s);
    else
        start<1024, 4>(a, s);
    return hipGetLastError();
}

}  // namespace bd
