// Product of int8 rows with an int8 base and 1-bit deltas, many tokens
// (bitdelta_linear_int8; the formula stands in linear_int8.hip).  Bound by the
// matrix units.
//
// A workgroup of eight waves forms a tile of BM tokens x BN channels, 128
// columns a step.  The tokens' and the base's rows of a step are copied into
// LDS directly, NBUF - 1 steps ahead, and every wave reads its operands from
// there.  With a delta each tile has two sets of sums: the tokens' operands of a
// step meet the base's bytes and the signs', which the waves spread from bits
// to bytes of +-1 in registers (16 bytes of signs a channel and step come
// through LDS too).  Sums of whole numbers are exact, so the two products need
// no common scale, and nothing of W_eff is ever formed.
//
// In LDS the 16-byte chunk c of row r stands at c ^ ((r >> 1) & 7), so that the
// reads of 32 rows spread over the banks.  One barrier a step.
#include <type_traits>

#include "bd_launch.h"
#include "int8_device.h"
#include "int8_tiles.h"

namespace bd {
namespace {

constexpr int kStep = 128;    // columns (bytes) a step
constexpr int kWaves = 8;
constexpr int kXcds = 8;

__device__ __forceinline__ int64_t xcd_remap(int64_t b, int64_t nb)
{
    const int64_t per = nb / kXcds;
    if (b >= per * kXcds)
        return b;
    return (b % kXcds) * per + b / kXcds;
}

__device__ __forceinline__ i32x16 mfma32(u32x4 a, u32x4 b, i32x16 c)
{
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Four signs (bits at .. at + 3 of w) as bytes of +1 and -1: the bits spread to
// a byte each by a product, which then picks 0xFF or 0x01.
__device__ __forceinline__ uint32_t signed_bytes(uint32_t w, int at)
{
    const uint32_t spread = __umul24((w >> at) & 15u, 0x00204081u) & 0x01010101u;
    return __builtin_amdgcn_perm(0u, 0x000001FFu, spread);
}

// BM x BN tile by WM x WN waves; GATHER: tokens ordered by variant, the table of
// bucket_tokens.
template <int BM, int BN, int WM, int WN, int NBUF, bool DELTA, bool GATHER>
__global__ __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(2, 2)))
void int8_tiles(Int8Args a, int64_t m_tiles, int64_t n_fast, const int32_t *__restrict__ table)
{
    static_assert(WM * WN == kWaves && (NBUF == 2 || NBUF == 3), "waves, buffers");
    constexpr int MB = BM / WM / 32, NB = BN / WN / 32;
    constexpr int XI = BM / 8 / kWaves, WI = BN / 8 / kWaves, SI = DELTA ? BN / 16 / kWaves : 0;
    constexpr int kCopies = XI + WI + SI;      // of a wave and step
    __shared__ __attribute__((aligned(16))) uint8_t xs[NBUF][BM * kStep], ws[NBUF][BN * kStep];
    __shared__ __attribute__((aligned(16))) uint8_t ss[DELTA ? NBUF : 1][DELTA ? BN * 16 : 16];
    __shared__ int32_t rows_s[BM];
    __shared__ float scale_s[BM];

    const int lane = threadIdx.x & 63, hi = lane >> 5, low = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t K = a.d_in, N = a.d_out, G = K >> 3;
    const int64_t tile = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t mt = n_fast ? tile / n_fast : tile % m_tiles, nt = n_fast ? tile % n_fast : tile / m_tiles;
    const int64_t n0 = nt * BN;

    int variant = 0;
    if constexpr (GATHER) {
        if (mt >= table[0])
            return;
        const int32_t *perm = table + 4, *tile_v = perm + a.m, *row0 = tile_v + m_tiles, *rows = row0 + m_tiles;
        variant = tile_v[mt];
        for (int i = threadIdx.x; i < BM; i += kWaves * 64)
            rows_s[i] = i < rows[mt] ? perm[row0[mt] + i] : -1;
    } else {
        for (int i = threadIdx.x; i < BM; i += kWaves * 64)
            rows_s[i] = mt * BM + i < a.m ? (int32_t)(mt * BM + i) : -1;
    }
    __syncthreads();
    const bool known = variant < a.n_variants || !DELTA;
    for (int i = threadIdx.x; i < BM; i += kWaves * 64)
        scale_s[i] = rows_s[i] >= 0 ? a.q_scale[rows_s[i]] : 0.0f;
    const uint8_t *signs = DELTA ? a.signs + (int64_t)(known ? variant : 0) * N * G : nullptr;

    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.q, a.m * K), rw = make_rsrc(a.w, N * K);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(signs, DELTA ? N * G : 0);
    // copy i of this wave covers 8 rows; lane l writes place l & 7 of row l / 8.
    // Rows that do not exist have an offset out of range (zeros); the step's
    // columns go into the scalar offset, which is not checked, so the last step's
    // lanes past the row's end have theirs out of range too.
    const int place = lane & 7;
    uint32_t xoff[XI], woff[WI], soff[SI ? SI : 1];
    int xk[XI], wk[WI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int row = (wave * XI + i) * 8 + (lane >> 3);
        xk[i] = (place ^ ((row >> 1) & 7)) * 16;
        xoff[i] = rows_s[row] < 0 ? kInvalidOffset : (uint32_t)(rows_s[row] * K + xk[i]);
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int row = (wave * WI + i) * 8 + (lane >> 3);
        wk[i] = (place ^ ((row >> 1) & 7)) * 16;
        woff[i] = n0 + row < N ? (uint32_t)((n0 + row) * K + wk[i]) : kInvalidOffset;
    }
#pragma unroll
    for (int i = 0; i < SI; ++i) {
        const int row = (wave * SI + i) * 16 + (lane >> 2);
        soff[i] = n0 + row < N ? (uint32_t)((n0 + row) * G + (lane & 3) * 4) : kInvalidOffset;
    }
    const int T = (int)((K + kStep - 1) / kStep);
    const int last = (int)(K - (int64_t)(T - 1) * kStep);     // columns of the last step
    auto copy = [&](int t, int buf) {
        const uint32_t k = (uint32_t)t * kStep;
        const int have = t == T - 1 ? last : kStep;
#pragma unroll
        for (int i = 0; i < XI; ++i)
            copy16(rx, xs[buf] + (wave * XI + i) * 1024, xk[i] < have ? xoff[i] : kInvalidOffset, k);
#pragma unroll
        for (int i = 0; i < WI; ++i)
            copy16(rw, ws[buf] + (wave * WI + i) * 1024, wk[i] < have ? woff[i] : kInvalidOffset, k);
#pragma unroll
        for (int i = 0; i < SI; ++i)
            copy4(rs, ss[buf] + (wave * SI + i) * 256, (lane & 3) * 32 < have ? soff[i] : kInvalidOffset, k / 8);
    };
    const int sw = (low >> 1) & 7;
    auto read_x = [&](u32x4 (&f)[MB], int buf, int kb) {
        const uint8_t *p = xs[buf] + (wm * MB * 32 + low) * kStep + (((kb * 2 + hi) ^ sw) * 16);
#pragma unroll
        for (int i = 0; i < MB; ++i)
            f[i] = *reinterpret_cast<const u32x4 *>(p + i * 32 * kStep);
    };
    auto read_w = [&](u32x4 (&f)[NB], int buf, int kb) {
        const uint8_t *p = ws[buf] + (wn * NB * 32 + low) * kStep + (((kb * 2 + hi) ^ sw) * 16);
#pragma unroll
        for (int i = 0; i < NB; ++i)
            f[i] = *reinterpret_cast<const u32x4 *>(p + i * 32 * kStep);
    };
    auto read_s = [&](u32x4 (&f)[NB], int buf) {
        if constexpr (DELTA)
#pragma unroll
            for (int i = 0; i < NB; ++i)
                f[i] = *reinterpret_cast<const u32x4 *>(ss[buf] + (wn * NB * 32 + i * 32 + low) * 16);
    };

    // Sums in accumulation registers: left in the others, the matrix
    // instructions and the rest contend for one file.
    i32x16 acc[MB][NB], accd[DELTA ? MB : 1][DELTA ? NB : 1];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[i][j][v] = 0;
            asm volatile("" : "+a"(acc[i][j]));
            if constexpr (DELTA) {
                accd[i][j] = acc[i][j];
                asm volatile("" : "+a"(accd[i][j]));
            }
        }

#pragma unroll
    for (int t = 0; t < NBUF; ++t)
        copy(t < T ? t : T - 1, t);
    wait_vmcnt<(NBUF - 1) * kCopies>();
    __syncthreads();
    u32x4 X[2][MB], W[2][NB], S[2][NB];
    read_x(X[0], 0, 0);
    read_w(W[0], 0, 0);
    read_s(S[0], 0);

    auto product = [&](int kb, const u32x4 (&s)[NB]) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < MB; ++i)
                acc[i][j] = mfma32(X[kb & 1][i], W[kb & 1][j], acc[i][j]);
        if constexpr (DELTA)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                u32x4 b;
                const uint32_t w = s[j][kb] >> (16 * hi);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    b[c] = signed_bytes(w, 4 * c);
#pragma unroll
                for (int i = 0; i < MB; ++i)
                    accd[i][j] = mfma32(X[kb & 1][i], b, accd[i][j]);
            }
    };
    // Step t from buffer cur, whose first operands are in registers.  Before the
    // last of its four products every read of the buffer is done: the barrier, the
    // copies of step t + NBUF into it, and the first operands of step t + 1, which
    // has landed, while that product runs.
    auto step = [&](int t, auto cur_c, auto odd_c) {
        constexpr int cur = decltype(cur_c)::value, nxt = (cur + 1) % NBUF, o = decltype(odd_c)::value;
#pragma unroll
        for (int kb = 0; kb < 3; ++kb) {
            read_x(X[(kb + 1) & 1], cur, kb + 1);
            read_w(W[(kb + 1) & 1], cur, kb + 1);
            product(kb, S[o]);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_vmcnt_lgkm0<(NBUF - 2) * kCopies>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        copy(t + NBUF < T ? t + NBUF : T - 1, cur);
        __builtin_amdgcn_sched_barrier(0);
        read_x(X[0], nxt, 0);       // past the last step: copied again, not used
        read_w(W[0], nxt, 0);
        read_s(S[1 - o], nxt);
        product(3, S[o]);
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kTurn = NBUF % 2 ? 2 * NBUF : NBUF;     // steps until buffer and sign registers meet again
    for (int t = 0; t < T; t += kTurn) {
        step(t, std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{});
        if (t + 1 < T)
            step(t + 1, std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
        if constexpr (kTurn == 6) {
            if (t + 2 < T)
                step(t + 2, std::integral_constant<int, 2 % NBUF>{}, std::integral_constant<int, 0>{});
            if (t + 3 < T)
                step(t + 3, std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
            if (t + 4 < T)
                step(t + 4, std::integral_constant<int, 1>{}, std::integral_constant<int, 0>{});
            if (t + 5 < T)
                step(t + 5, std::integral_constant<int, 2 % NBUF>{}, std::integral_constant<int, 1>{});
        }
    }
    // copies still on their way must land before the workgroup's LDS is released
    __builtin_amdgcn_s_waitcnt(0);

#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int64_t n = n0 + (wn * NB + j) * 32 + low;
        const float c = n < N ? a.w_scale[n] : 0.0f;
        float alpha = 0.0f;
        if (DELTA && known && n < N)
            alpha = a.alpha[a.per_matrix ? variant : variant * N + n];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int row = (wm * MB + i) * 32 + 8 * (v >> 2) + 4 * hi + (v & 3);
                const int32_t token = rows_s[row];
                if (token < 0 || n >= N)
                    continue;
                const float y = known ? combine(scale_s[row], c, acc[i][j][v], alpha, DELTA ? accd[i][j][v] : 0) : 0.0f;
                if (a.f32)
                    static_cast<float *>(a.y)[token * N + n] = y;
                else
                    static_cast<uint16_t *>(a.y)[token * N + n] = to_bf16(y);
            }
    }
}

template <int BM, int BN, int WM, int WN, int NBUF, bool DELTA, bool GATHER>
hipError_t tiles(const Int8Args &a, int64_t m_tiles, const int32_t *table, hipStream_t s)
{
    const int64_t n_tiles = (a.d_out + BN - 1) / BN;
    const int64_t n_fast = !GATHER && a.d_out < a.m ? n_tiles : 0;
    const dim3 grid((unsigned)(m_tiles * n_tiles));
    int8_tiles<BM, BN, WM, WN, NBUF, DELTA, GATHER><<<grid, kWaves * 64, 0, s>>>(a, m_tiles, n_fast, table);
    return hipGetLastError();
}

}  // namespace

bool int8_tiles_take(const Int8Args &a)
{
    // a launch takes fewer than 2^32 threads
    const int64_t most = (a.m + 255) / 256 + (a.ids ? a.n_variants + 1 : 0);
    return a.d_in % 32 == 0 && ((uintptr_t)a.signs & 3) == 0 && most * ((a.d_out + 127) / 128) < (1 << 23);
}

size_t int8_tiles_workspace_bytes(int64_t m, int32_t n_variants)
{
    return n_variants > 1 ? grouped_workspace_bytes(m, n_variants) : 0;
}

hipError_t launch_int8_tiles(const Int8Args &a, void *workspace, hipStream_t s)
{
    const int64_t m_tiles = (a.m + 255) / 256;
    if (!a.signs)
        return tiles<256, 256, 2, 4, 2, false, false>(a, m_tiles, nullptr, s);
    if (!a.ids)
        return tiles<256, 128, 4, 2, 3, true, false>(a, m_tiles, nullptr, s);
    int32_t *table = static_cast<int32_t *>(workspace);
    const hipError_t e = launch_bucket_tokens(a.ids, a.m, a.n_variants, table, s);
    if (e != hipSuccess)
        return e;
    return tiles<256, 128, 4, 2, 3, true, true>(a, grouped_max_tiles(a.m, a.n_variants), table, s);
}

}  // namespace bd
