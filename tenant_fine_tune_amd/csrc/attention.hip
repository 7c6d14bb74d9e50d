// Causal attention over a paged cache, with shared prefixes
// (bitdelta_attention).
//
// One workgroup per token and query head: its waves take the visible keys in
// turn, one key per wave and step, each with its own running maximum m, sum l
// and weighted value o (per key: m' = max(m, s), o = o e^(m - m') + e^(s - m') v),
// and the waves' states are joined at the end.
#include "bd_device.h"
#include "decoder_launch.h"
#include "paged.h"

namespace bd {
namespace {

constexpr int kWaves = 4;

struct AttnArgs {
    Paged p;
    const uint16_t *q;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    uint16_t *out;
    int64_t q_stride;
    int32_t n_heads;
    float scale;
};

template <int N, bool E4M3>
__device__ __forceinline__ void load_cell(const uint8_t *cache, int64_t at, float *f)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (E4M3)
            f[i] = __builtin_amdgcn_cvt_f32_fp8((int)cache[at + i], 0);
        else
            f[i] = lo_f32(reinterpret_cast<const uint16_t *>(cache)[at + i]);
}

template <int D, bool E4M3>
__global__ __launch_bounds__(kWaves * 64) void attention_rows(AttnArgs a)
{
    constexpr int N = D / 64;
    __shared__ float ml[kWaves][2], os[kWaves][D];
    const Paged &p = a.p;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, kvh = h / (a.n_heads / p.n_kv);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s = seq_of(p, t);
    int seen[2] = {0, 0};
    const int32_t *table[2] = {p.b.prefix_table, p.b.page_table};
    if (s >= 0) {
        seen[1] = max(0, own_keys(p, s) - (seq_begin(p, s + 1) - (int)t) + 1);
        table[1] += (int64_t)s * p.b.max_pages;
        const int g = group_of(p, s);
        if (g >= 0) {
            seen[0] = prefix_keys(p, g);
            table[0] += (int64_t)g * p.b.max_prefix_pages;
        }
    }
    const float scale = a.scale * (E4M3 && a.k_scale ? a.k_scale[kvh] : 1.0f);
    float q[N], o[N] = {}, m = -INFINITY, l = 0.0f;
    for (int i = 0; i < N; ++i)
        q[i] = lo_f32(a.q[t * a.q_stride + h * D + lane * N + i]) * scale;
    for (int part = 0; part < 2; ++part)
        for (int j = wave; j < seen[part]; j += kWaves) {
            const int page = table[part][j >> p.page_shift];
            if ((unsigned)page >= (unsigned)p.n_pages)
                continue;
            const int64_t at = (((((int64_t)page * p.n_kv + kvh) << p.page_shift) +
                                 (j & ((1 << p.page_shift) - 1))) * D) + lane * N;
            float k[N], v[N], x = 0.0f;
            load_cell<N, E4M3>(a.k, at, k);
            load_cell<N, E4M3>(a.v, at, v);
            for (int i = 0; i < N; ++i)
                x = fmaf(q[i], k[i], x);
            for (int w = 32; w > 0; w >>= 1)
                x += __shfl_xor(x, w);
            const float mn = fmaxf(m, x);
            const float keep = m == mn ? 1.0f : __expf(m - mn), e = x == mn ? 1.0f : __expf(x - mn);
            m = mn;
            l = l * keep + e;
            for (int i = 0; i < N; ++i)
                o[i] = o[i] * keep + e * v[i];
        }
    if (lane == 0)
        ml[wave][0] = m, ml[wave][1] = l;
    for (int i = 0; i < N; ++i)
        os[wave][lane * N + i] = o[i];
    __syncthreads();
    if (threadIdx.x < D) {
        float mm = -INFINITY, ll = 0.0f, oo = 0.0f;
        for (int w = 0; w < kWaves; ++w)
            mm = fmaxf(mm, ml[w][0]);
        for (int w = 0; w < kWaves; ++w) {
            const float e = ml[w][0] == -INFINITY ? 0.0f : __expf(ml[w][0] - mm);
            ll += e * ml[w][1];
            oo += e * os[w][threadIdx.x];
        }
        const float vs = E4M3 && a.v_scale ? a.v_scale[kvh] : 1.0f;
        a.out[(t * a.n_heads + h) * D + threadIdx.x] = to_bf16(ll > 0.0f || ll != ll ? oo / ll * vs : 0.0f);
    }
}

}  // namespace

size_t attention_workspace_bytes(int32_t, const bd_kv_cache &, const bd_batch &) { return 0; }

hipError_t launch_attention(const uint16_t *q, int64_t q_stride, int32_t n_heads, float scale, const bd_kv_cache &c,
                            const bd_batch &b, uint16_t *out, void *, hipStream_t s)
{
    AttnArgs a;
    a.p = {b, c.n_pages, c.n_kv_heads, __builtin_ctz((unsigned)c.page_size)};
    a.q = q, a.q_stride = q_stride, a.out = out, a.n_heads = n_heads, a.scale = scale;
    a.k = static_cast<const uint8_t *>(c.k), a.v = static_cast<const uint8_t *>(c.v);
    a.k_scale = c.k_scale, a.v_scale = c.v_scale;
    const dim3 grid((unsigned)b.n_tokens, (unsigned)n_heads);
    const bool e4m3 = c.dtype == BD_KV_E4M3;
    if (c.head_dim == 64) {
        if (e4m3)
            attention_rows<64, true><<<grid, kWaves * 64, 0, s>>>(a);
        else
            attention_rows<64, false><<<grid, kWaves * 64, 0, s>>>(a);
    } else {
        if (e4m3)
            attention_rows<128, true><<<grid, kWaves * 64, 0, s>>>(a);
        else
            attention_rows<128, false><<<grid, kWaves * 64, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace bd
