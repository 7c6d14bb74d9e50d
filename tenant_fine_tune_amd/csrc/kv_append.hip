// Rotary positions and the append of keys and values to a paged cache
// (bitdelta_kv_append).
//
// A workgroup serves one token (part of its heads where tokens are few).  The
// angle pos * inv_freq[i] is formed and reduced to a fraction of a turn in
// fp64, because a position of 10^6 leaves fp32 no digits of a fast angle; the
// sine and cosine of the fraction are fp32, computed once per token and pair
// into LDS and shared by all heads.  A thread then moves two 8-column chunks of
// a head, half of the turned (or of the other) columns apart: eight pairs of
// halves, or eight neighbouring pairs, and neighbouring threads touch whole
// lines.  Memory bound: every q, k, v is read once, past the caches, and written
// once, q past them too where its lines are whole: 17122 tokens of 64 + 8 + 8
// heads of 128 take 120 us, 6.0 TB/s (133 through the caches); half-turned heads
// 51 us (54 with their half lines past the caches).  Between the kernels that
// write its inputs and read q, 17122 tokens gain the same (368 -> 344 us for all
// three), 6060 more (153 -> 129), 2015, which the last cache level holds, lose
// (47 -> 50).  6060 tokens into an 8-bit cache, half turned: 48 us from HBM, 4.9
// TB/s; 32 single tokens 5 us, launch latency: their heads are dealt over three
// workgroups each.
#include "bd_device.h"
#include "decoder_launch.h"
#include "paged.h"

namespace bd {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    Paged p;
    const uint16_t *q, *k, *v;
    uint16_t *q_out;
    uint8_t *kc, *vc;
    const float *k_scale, *v_scale;
    const double *inv_freq;
    int64_t q_stride, k_stride, v_stride;
    int32_t n_heads, rotary;
};

// Four numbers as e4m3, nearest even, clamped to +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    // fmin / fmax would turn a NaN into a bound
    const auto clamp = [](float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp(a), clamp(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp(c), clamp(d), w, true);
}

__device__ __forceinline__ void unpack8(uint4 w, float *f)
{
    f[0] = lo_f32(w.x), f[1] = hi_f32(w.x), f[2] = lo_f32(w.y), f[3] = hi_f32(w.y);
    f[4] = lo_f32(w.z), f[5] = hi_f32(w.z), f[6] = lo_f32(w.w), f[7] = hi_f32(w.w);
}

__device__ __forceinline__ uint4 pack8(const float *f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

template <int D, bool E4M3>
__device__ __forceinline__ void store_cell(uint8_t *cache, int64_t cell, int col, const float *f, float scale)
{
    if (E4M3) {
        uint2 w;
        w.x = e4m3x4(f[0] / scale, f[1] / scale, f[2] / scale, f[3] / scale);
        w.y = e4m3x4(f[4] / scale, f[5] / scale, f[6] / scale, f[7] / scale);
        *reinterpret_cast<uint2 *>(cache + cell * D + col) = w;
    } else {
        *reinterpret_cast<uint4 *>(cache + (cell * D + col) * 2) = pack8(f);
    }
}

template <int D, bool E4M3, bool INTER>
__global__ __launch_bounds__(kThreads) void append_tokens(AppendArgs a)
{
    __shared__ float2 turn[D / 2];
    const Paged &p = a.p;
    const int64_t t = blockIdx.z * kTokensAcross + blockIdx.x;
    if (t >= p.b.n_tokens)
        return;
    const int s = seq_of(p, t);
    bool placed = s >= 0;
    int64_t cell = -1;   // of head 0
    if (placed) {
        const int at = own_keys(p, s) - (seq_begin(p, s + 1) - (int)t);
        placed = at >= 0;
        const int g = group_around(p, s);
        if (placed) {
            cell = cell_of(p, p.b.page_table + (int64_t)s * p.b.max_pages, 0, at);
            const double pos = (double)at + (g >= 0 ? prefix_keys(p, g) : 0);
            for (int i = threadIdx.x; i < a.rotary / 2; i += kThreads) {
                // turns, to the nearest whole one, then radians / pi in [-1, 1]
                const double turns = pos * a.inv_freq[i] * 0.15915494309189533577;
                const float frac = (float)(2.0 * (turns - rint(turns)));
                float sn, cs;
                sincospif(frac, &sn, &cs);
                turn[i] = make_float2(cs, sn);
            }
        }
    }
    __syncthreads();

    const int H = a.n_heads, units = (H + 2 * p.n_kv) * (D / 16);
    for (int u = blockIdx.y * kThreads + threadIdx.x; u < units; u += gridDim.y * kThreads) {
        const int row = u / (D / 16), part = u % (D / 16);
        const bool is_q = row < H, is_v = row >= H + p.n_kv;
        if (!is_q && cell < 0)
            continue;
        const int head = is_q ? row : is_v ? row - H - p.n_kv : row - H;
        const bool turned = !is_v && part * 16 < a.rotary;
        // the two chunks: the same place in the halves of what is turned, or of what is not
        const int from = turned || is_v ? 0 : a.rotary, width = turned ? a.rotary : D - from;
        const int c0 = from + (part - from / 16) * 8, c1 = c0 + width / 2;
        float x[8], y[8];
        if (placed) {
            const uint16_t *src = (is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) +
                                  (int64_t)head * D;
            unpack8(ld_stream16(src + c0), x);
            unpack8(ld_stream16(src + c1), y);
            if (turned) {
                if (INTER) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 e = turn[c0 / 2 + i], f = turn[c1 / 2 + i];
                        const float x0 = x[2 * i], y0 = y[2 * i];
                        x[2 * i] = x0 * e.x - x[2 * i + 1] * e.y;
                        x[2 * i + 1] = x[2 * i + 1] * e.x + x0 * e.y;
                        y[2 * i] = y0 * f.x - y[2 * i + 1] * f.y;
                        y[2 * i + 1] = y[2 * i + 1] * f.x + y0 * f.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 e = turn[part * 8 + i];
                        const float x0 = x[i];
                        x[i] = x0 * e.x - y[i] * e.y;
                        y[i] = y[i] * e.x + x0 * e.y;
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = y[i] = 0.0f;
        }
        if (is_q) {
            uint16_t *dst = a.q_out + (t * H + head) * D;
            if (width == D) {
                st_stream16(dst + c0, pack8(x));
                st_stream16(dst + c1, pack8(y));
            } else {
                *reinterpret_cast<uint4 *>(dst + c0) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + c1) = pack8(y);
            }
        } else {
            const int64_t at = cell + ((int64_t)head << p.page_shift);
            const float *scales = is_v ? a.v_scale : a.k_scale;
            const float scale = E4M3 && scales ? scales[head] : 1.0f;
            uint8_t *dst = is_v ? a.vc : a.kc;
            store_cell<D, E4M3>(dst, at, c0, x, scale);
            store_cell<D, E4M3>(dst, at, c1, y, scale);
        }
    }
}

template <int D>
void start(const AppendArgs &a, bool e4m3, bool inter, dim3 grid, hipStream_t s)
{
    if (e4m3) {
        if (inter)
            append_tokens<D, true, true><<<grid, kThreads, 0, s>>>(a);
        else
            append_tokens<D, true, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (inter)
            append_tokens<D, false, true><<<grid, kThreads, 0, s>>>(a);
        else
            append_tokens<D, false, false><<<grid, kThreads, 0, s>>>(a);
    }
}

}  // namespace

hipError_t launch_kv_append(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                            const uint16_t *v, int64_t v_stride, int32_t n_heads, const double *inv_freq,
                            int32_t rotary, bool interleaved, const bd_kv_cache &c, const bd_batch &b,
                            uint16_t *q_out, hipStream_t s)
{
    AppendArgs a;
    a.p = {b, c.n_pages, c.n_kv_heads, __builtin_ctz((unsigned)c.page_size)};
    a.q = q, a.k = k, a.v = v, a.q_out = q_out;
    a.kc = static_cast<uint8_t *>(c.k), a.vc = static_cast<uint8_t *>(c.v);
    a.k_scale = c.k_scale, a.v_scale = c.v_scale;
    a.inv_freq = inv_freq;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.n_heads = n_heads, a.rotary = rotary;
    const int64_t units = (int64_t)(n_heads + 2 * c.n_kv_heads) * (c.head_dim / 16);
    const int64_t parts = b.n_tokens < 512 ? (units + kThreads - 1) / kThreads : 1;
    const dim3 grid((unsigned)(b.n_tokens < kTokensAcross ? b.n_tokens : kTokensAcross), (unsigned)parts,
                    (unsigned)((b.n_tokens + kTokensAcross - 1) / kTokensAcross));
    if (c.head_dim == 64)
        start<64>(a, c.dtype == BD_KV_E4M3, interleaved, grid, s);
    else
        start<128>(a, c.dtype == BD_KV_E4M3, interleaved, grid, s);
    return hipGetLastError();
}

}  // namespace bd
