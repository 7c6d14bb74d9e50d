// Product of int8 rows with an int8 base and 1-bit deltas, many tokens
// (bitdelta_linear_int8; the formula stands in linear_int8.hip).  Bound by the
// matrix units.
//
// A workgroup of four waves forms a tile of BM (64 or 128) tokens x 128 channels,
// 128 columns a step.  The tokens' and the base's rows of a step are copied into
// LDS directly, a step ahead, and every wave reads its operands from there: its
// 32 channels and all the tokens.  With a delta each tile has two sets of sums: the
// tokens' operands of a step meet the base's bytes and the signs', which the wave
// spreads from bits to bytes of +-1 in registers, each once (16 bytes of signs a
// channel and step come through LDS too).  Sums of whole numbers are exact, so the
// two products need no common scale, nothing of W_eff is ever formed, and the
// columns may be split over workgroups where the tiles are few.
// Two or three workgroups a compute unit hide each other's waits.  2048 tokens
// through 8192 x 8192 with one delta 270 us; where shapes were compared four waves of 32
// channels took 262, four of 64 tokens x 64 channels 285, eight in a tile of 256 x 128
// alone on its unit 300.
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
constexpr int kBN = 128;      // channels a tile
constexpr int kWaves = 4;
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

// A call over rows of whole 32 columns: as given, or with the tokens' numbers and
// the signs in copies that zeros fill up, while w keeps its own stride (how its rows'
// ends are read and copied: int8_tiles.h).
struct TileArgs : Int8Args {
    int64_t w_stride;
};

// The output tile of a workgroup.  Tiles that meet the same rows of w (or, with
// n_fast, of the tokens) are neighbours, and so on one die.
struct Place {
    int64_t mt, nt;
    int split;
};
__device__ __forceinline__ Place place_of(int64_t at, int64_t m_tiles, int64_t n_tiles, bool n_fast, int splits)
{
    if (n_fast)
        return {at / n_tiles / splits, at % n_tiles, (int)(at / n_tiles % splits)};
    return {at % m_tiles, at / m_tiles / splits, (int)(at / m_tiles % splits)};
}

// Token of row `row` of a tile, or -1.
template <int BM, bool GATHER>
__device__ __forceinline__ int32_t token_of(const TileArgs &a, const int32_t *table, int64_t mt, int row)
{
    if constexpr (GATHER) {
        const int64_t entries = (a.m + BM - 1) / BM + a.n_variants + 1;    // of grouped_max_tiles
        const int32_t *perm = table + 4, *row0 = perm + a.m + entries, *rows = row0 + entries;
        return row < rows[mt] ? perm[row0[mt] + row] : -1;
    }
    return mt * BM + row < a.m ? (int32_t)(mt * BM + row) : -1;
}

// One tile, one of `splits` parts of the columns (with more than one the sums go to
// `partial`); GATHER: tokens ordered by variant, the table of bucket_tokens.
template <int BM, bool DELTA, bool GATHER>
__global__ __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(2, BM == 64 ? 3 : 2)))
void int8_tiles(TileArgs a, int64_t m_tiles, int64_t n_tiles, bool n_fast, int splits, const int32_t *__restrict__ table,
                i32x4 *__restrict__ partial)
{
    constexpr int MB = BM / 32;                // blocks of 32 tokens, by the wave's 32 channels
    constexpr int XI = BM / 8 / kWaves, WI = kBN / 8 / kWaves, SI = DELTA ? kBN / 16 / kWaves : 0;
    constexpr int kCopies = XI + WI + SI;      // of a wave and step
    __shared__ __attribute__((aligned(16))) uint8_t xs[2][BM * kStep], ws[2][kBN * kStep];
    __shared__ __attribute__((aligned(16))) uint8_t ss[DELTA ? 2 : 1][DELTA ? kBN * 16 : 16];
    __shared__ int32_t rows_s[BM];
    __shared__ float scale_s[BM];

    const int lane = threadIdx.x & 63, hi = lane >> 5, low = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t K = a.d_in, N = a.d_out, G = K >> 3;
    const int64_t at = xcd_remap(blockIdx.x, gridDim.x);
    const auto [mt, nt, split] = place_of(at, m_tiles, n_tiles, n_fast, splits);
    const int64_t n0 = nt * kBN;

    int variant = 0;
    if constexpr (GATHER) {
        if (mt >= table[0])
            return;
        variant = (table + 4 + a.m)[mt];
    }
    for (int i = threadIdx.x; i < BM; i += kWaves * 64)
        rows_s[i] = token_of<BM, GATHER>(a, table, mt, i);
    __syncthreads();
    const bool known = variant < a.n_variants || !DELTA;
    for (int i = threadIdx.x; i < BM; i += kWaves * 64)
        scale_s[i] = rows_s[i] >= 0 ? a.q_scale[rows_s[i]] : 0.0f;
    const uint8_t *signs = DELTA ? a.signs + (int64_t)(known ? variant : 0) * N * G : nullptr;

    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.q, a.m * K), rw = make_rsrc(a.w, N * a.w_stride);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(signs, DELTA ? N * G : 0);
    // copy i of this wave covers 8 rows; lane l writes place l & 7 of row l / 8.
    // Rows that do not exist have an offset out of range (zeros); the step's
    // columns go into the scalar offset, which is not checked, so the last step's
    // lanes past the row's end have theirs out of range too, and w's have the whole of
    // their place in it.
    const int place = lane & 7;
    const int steps = (int)((K + kStep - 1) / kStep), begin = (int)((int64_t)steps * split / splits);
    uint32_t xoff[XI], woff[WI], wlast[WI], soff[SI ? SI : 1];
    int xk[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int row = (wave * XI + i) * 8 + (lane >> 3);
        xk[i] = (place ^ ((row >> 1) & 7)) * 16;
        xoff[i] = rows_s[row] < 0 ? kInvalidOffset : (uint32_t)(rows_s[row] * K + xk[i]);
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int row = (wave * WI + i) * 8 + (lane >> 3);
        const int wk = (place ^ ((row >> 1) & 7)) * 16, column = chunk_column((steps - 1) * kStep + wk, (int)a.w_stride);
        woff[i] = n0 + row < N ? (uint32_t)((n0 + row) * a.w_stride + wk) : kInvalidOffset;
        wlast[i] = n0 + row < N && column >= 0 ? (uint32_t)((n0 + row) * a.w_stride + column) : kInvalidOffset;
    }
#pragma unroll
    for (int i = 0; i < SI; ++i) {
        const int row = (wave * SI + i) * 16 + (lane >> 2);
        soff[i] = n0 + row < N ? (uint32_t)((n0 + row) * G + (lane & 3) * 4) : kInvalidOffset;
    }
    const int T = (int)((int64_t)steps * (split + 1) / splits) - begin;
    const int last = (int)(K - (int64_t)(steps - 1) * kStep);     // columns of the last step
    auto copy = [&](int t, int buf) {
        const uint32_t k = (uint32_t)(begin + t) * kStep;
        const bool end = begin + t == steps - 1;
        const int have = end ? last : kStep;
#pragma unroll
        for (int i = 0; i < XI; ++i)
            copy16(rx, xs[buf] + (wave * XI + i) * 1024, xk[i] < have ? xoff[i] : kInvalidOffset, k);
#pragma unroll
        for (int i = 0; i < WI; ++i)
            copy16(rw, ws[buf] + (wave * WI + i) * 1024, end ? wlast[i] : woff[i], end ? 0 : k);
#pragma unroll
        for (int i = 0; i < SI; ++i)
            copy4(rs, ss[buf] + (wave * SI + i) * 256, (lane & 3) * 32 < have ? soff[i] : kInvalidOffset, k / 8);
    };
    const int sw = (low >> 1) & 7;
    auto read_x = [&](u32x4 (&f)[MB], int buf, int kb) {
        const uint8_t *p = xs[buf] + low * kStep + (((kb * 2 + hi) ^ sw) * 16);
#pragma unroll
        for (int i = 0; i < MB; ++i)
            f[i] = *reinterpret_cast<const u32x4 *>(p + i * 32 * kStep);
    };
    auto read_w = [&](u32x4 &f, int buf, int kb) {
        f = *reinterpret_cast<const u32x4 *>(ws[buf] + (wave * 32 + low) * kStep + (((kb * 2 + hi) ^ sw) * 16));
    };
    auto read_s = [&](u32x4 &f, int buf) {
        if constexpr (DELTA)
            f = *reinterpret_cast<const u32x4 *>(ss[buf] + (wave * 32 + low) * 16);
    };

    // Sums in accumulation registers: left in the others, the matrix
    // instructions and the rest contend for one file.
    i32x16 acc[MB], accd[DELTA ? MB : 1];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
        for (int v = 0; v < 16; ++v)
            acc[i][v] = 0;
        asm volatile("" : "+a"(acc[i]));
        if constexpr (DELTA) {
            accd[i] = acc[i];
            asm volatile("" : "+a"(accd[i]));
        }
    }

    copy(0, 0);
    copy(T > 1 ? 1 : 0, 1);
    wait_vmcnt<kCopies>();
    __syncthreads();
    u32x4 X[2][MB], W[2], S[2];
    read_x(X[0], 0, 0);
    read_w(W[0], 0, 0);
    read_s(S[0], 0);

    auto product = [&](int kb, const u32x4 &s) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
            acc[i] = mfma32(X[kb & 1][i], W[kb & 1], acc[i]);
        if constexpr (DELTA) {
            u32x4 b;
            const uint32_t w = s[kb] >> (16 * hi);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                b[c] = signed_bytes(w, 4 * c);
#pragma unroll
            for (int i = 0; i < MB; ++i)
                accd[i] = mfma32(X[kb & 1][i], b, accd[i]);
        }
    };
    // Step t from buffer cur, whose first operands are in registers.  Before the
    // last of its four products every read of the buffer is done: the barrier, the
    // copies of step t + 2 into it, and the first operands of step t + 1, which
    // has landed, while that product runs.
    auto step = [&](int t, auto cur_c) {
        constexpr int cur = decltype(cur_c)::value, nxt = 1 - cur;
#pragma unroll
        for (int kb = 0; kb < 3; ++kb) {
            read_x(X[(kb + 1) & 1], cur, kb + 1);
            read_w(W[(kb + 1) & 1], cur, kb + 1);
            product(kb, S[cur]);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_vmcnt_lgkm0<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        copy(t + 2 < T ? t + 2 : T - 1, cur);
        __builtin_amdgcn_sched_barrier(0);
        read_x(X[0], nxt, 0);       // past the last step: copied again, not used
        read_w(W[0], nxt, 0);
        read_s(S[nxt], nxt);
        product(3, S[cur]);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int t = 0; t < T; t += 2) {
        step(t, std::integral_constant<int, 0>{});
        if (t + 1 < T)
            step(t + 1, std::integral_constant<int, 1>{});
    }
    // copies still on their way must land before the workgroup's LDS is released
    __builtin_amdgcn_s_waitcnt(0);

    if (splits > 1) {
        // in the order of the registers: sums of base and delta, by fours of rows
        constexpr int kSums = DELTA ? 2 : 1;
        i32x4 *out = partial + (at * kWaves + wave) * (MB * 4 * kSums * 64) + lane;
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < kSums; ++e) {
                    const i32x16 &from = e ? accd[DELTA ? i : 0] : acc[i];
                    out[((i * 4 + q) * kSums + e) * 64] = i32x4{from[4 * q], from[4 * q + 1], from[4 * q + 2], from[4 * q + 3]};
                }
        return;
    }
    const int64_t n = n0 + wave * 32 + low;
    if (n >= N)
        return;
    const float c = a.w_scale[n], alpha = DELTA && known ? a.alpha[a.per_matrix ? variant : variant * N + n] : 0.0f;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int row = i * 32 + 8 * (v >> 2) + 4 * hi + (v & 3);
            const int32_t token = rows_s[row];
            if (token < 0)
                continue;
            const float y = known ? combine(scale_s[row], c, acc[i][v], alpha, DELTA ? accd[i][v] : 0) : 0.0f;
            if (a.f32)
                static_cast<float *>(a.y)[token * N + n] = y;
            else
                static_cast<uint16_t *>(a.y)[token * N + n] = to_bf16(y);
        }
}

// Adds up the parts of int8_tiles: a wave for 32 channels by 8 rows.
template <int BM, bool DELTA, bool GATHER>
__global__ __launch_bounds__(kWaves * 64) void int8_tiles_join(TileArgs a, int64_t m_tiles, int64_t n_tiles, bool n_fast,
                                                       int splits, const int32_t *__restrict__ table,
                                                       const i32x4 *__restrict__ partial)
{
    constexpr int MB = BM / 32, kParts = kWaves * MB * 4, kLane = DELTA ? 128 : 64;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = (int64_t)blockIdx.x * kWaves + wave, tile = id / kParts;
    if (tile >= m_tiles * n_tiles)
        return;
    const int part = (int)(id % kParts), q = part & 3, i = part / 4 % MB, w = part / 4 / MB;
    // this tile's place among its splits
    const int64_t mt = n_fast ? tile / n_tiles : tile % m_tiles, nt = n_fast ? tile % n_tiles : tile / m_tiles;
    if (GATHER && mt >= table[0])
        return;
    i32x4 acc = {0, 0, 0, 0}, accd = {0, 0, 0, 0};
    for (int split = 0; split < splits; ++split) {
        const int64_t at = n_fast ? (mt * splits + split) * n_tiles + nt : (nt * splits + split) * m_tiles + mt;
        const i32x4 *in = partial + (at * kParts + part) * kLane + lane;
        acc += in[0];
        if constexpr (DELTA)
            accd += in[64];
    }
    const int variant = GATHER ? (table + 4 + a.m)[mt] : 0;
    const bool known = !DELTA || variant < a.n_variants;
    const int64_t n = nt * kBN + w * 32 + (lane & 31), N = a.d_out;
    if (n >= N)
        return;
    const float c = a.w_scale[n], alpha = DELTA && known ? a.alpha[a.per_matrix ? variant : variant * N + n] : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int32_t token = token_of<BM, GATHER>(a, table, mt, i * 32 + 8 * q + 4 * (lane >> 5) + r);
        if (token < 0)
            continue;
        const float y = known ? combine(a.q_scale[token], c, acc[r], alpha, accd[r]) : 0.0f;
        if (a.f32)
            static_cast<float *>(a.y)[token * N + n] = y;
        else
            static_cast<uint16_t *>(a.y)[token * N + n] = to_bf16(y);
    }
}

// The copies of TileArgs, eight numbers or 32 signs a thread.  G: bytes of a row of
// signs, any alignment.
__global__ __launch_bounds__(256) void int8_pad(const uint64_t *__restrict__ q, uint64_t *__restrict__ q_to, uint32_t q_units,
                                                const uint8_t *__restrict__ signs, uint32_t *__restrict__ signs_to,
                                                uint32_t sign_units, uint32_t G, uint32_t padded)
{
    uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i < q_units) {
        const uint32_t row = i / padded;
        const int from = copied_group(i % padded, G);
        q_to[i] = from >= 0 ? q[row * G + from] : 0;
        return;
    }
    i -= q_units;
    if (i >= sign_units)
        return;
    const uint32_t row = i / (padded / 4), at = i % (padded / 4) * 4;
    uint32_t w = 0;
    for (uint32_t b = 0; b < 4; ++b) {
        const int from = copied_group(at + b, G);
        if (from >= 0)
            w |= (uint32_t)signs[(uint64_t)row * G + from] << (8 * b);
    }
    signs_to[i] = w;
}

size_t table_bytes(int64_t m, int32_t n_variants)
{
    return (grouped_workspace_bytes(m, n_variants, 64) + 15) / 16 * 16;
}

// Tiles along the tokens; with ids the most there can be (a tile holds tokens of
// one variant, ids out of range being one more).
template <int BM>
int64_t token_tiles(int64_t m, int32_t variants)
{
    return variants ? m / BM + (m < variants + 1 ? m : variants + 1) : (m + BM - 1) / BM;
}

struct Plan {
    bool tall;      // tiles of 128 tokens, or of 64
    int splits;
};

// Sums of all splits' tiles; never more than kMostParts.
constexpr size_t kMostParts = (size_t)1 << 28;
size_t part_bytes(bool tall, int64_t m, int64_t d_out, int splits, bool delta, int32_t variants)
{
    const int64_t rows = tall ? token_tiles<128>(m, variants) * 128 : token_tiles<64>(m, variants) * 64;
    return splits == 1 ? 0 : (size_t)(rows * ((d_out + kBN - 1) / kBN) * kBN * splits) * (delta ? 8 : 4);
}

// By what the two tiles take, in us: 512 workgroups of the tall tile fit the card
// at once and 768 of the other; a step of 128 columns takes them 1.25 and 1.0
// without a delta, 2.1 and 1.5 with one (8192 x 8192, 512 to 2048 tokens), so that
// full rounds go 20 % faster through the tall tile and a part of one through the
// other.  Split columns cost a second launch and the sums' way through memory at
// 4 TB/s.  With ids, a variant in four is taken to have no tile of its own.
//   tokens (8192 x 8192, one delta)   64 tall, best split   128 tall, best split
//     128                              40 (4)                43 (4)
//     512                              83 (1)                93 (2)
//    1024                             166 (1)               140 (1)
//   14 variants, 512                  184 (1)               234 (1)
//                2048                 379 (1)               375 (1)
// On 1024, 10240 and 28672 x 8192 and 8192 x 28672, with 128 to 2048 tokens, what this
// picks takes at most 7 % longer than the best of both tiles and 1, 2, 4 or 8 splits, but
// for 128 tokens through 1024 x 8192 (20 %), 2048 through 10240 x 8192 and 1024 through
// 28672 x 8192 with one delta (13 and 10 %).
Plan plan_of(int64_t m, int64_t d_out, int64_t d_in, bool delta, int32_t variants)
{
    const int64_t steps = (d_in + kStep - 1) / kStep, n_tiles = (d_out + kBN - 1) / kBN;
    Plan best = {false, 1};
    double least = 0;
    for (int tall = 0; tall < 2; ++tall) {
        const int64_t bm = tall ? 128 : 64, slots = tall ? 512 : 768;
        const int64_t tiles = ((m + bm - 1) / bm + (variants < m ? variants : m) * 3 / 4) * n_tiles;
        const double us = tall ? (delta ? 2.1 : 1.25) : (delta ? 1.5 : 1.0);
        for (int splits = 1; splits <= 16 && (splits == 1 || steps / splits >= 4); splits *= 2) {
            double cost = (double)((tiles * splits + slots - 1) / slots * ((steps + splits - 1) / splits)) * us;
            if (splits > 1) {
                if (part_bytes(tall, m, d_out, splits, delta, variants) > kMostParts)
                    break;
                cost += 4 + (double)(tiles * splits * bm) * kBN * (delta ? 8 : 4) * 2 / 4e6;
            }
            if ((!tall && splits == 1) || cost < least) {
                least = cost;
                best = {tall != 0, splits};
            }
        }
    }
    return best;
}

template <int BM, bool DELTA, bool GATHER>
hipError_t tiles(const TileArgs &a, int splits, void *workspace, hipStream_t s)
{
    const int64_t m_tiles = token_tiles<BM>(a.m, GATHER ? a.n_variants : 0), n_tiles = (a.d_out + kBN - 1) / kBN;
    int32_t *table = static_cast<int32_t *>(workspace);
    i32x4 *partial = static_cast<i32x4 *>(workspace);
    if constexpr (GATHER) {
        const hipError_t e = launch_bucket_tokens(a.ids, a.m, a.n_variants, BM, table, s);
        if (e != hipSuccess)
            return e;
        partial += table_bytes(a.m, a.n_variants) / 16;
    }
    // neighbours share the larger operand
    const bool n_fast = !GATHER && a.d_out < a.m;
    const dim3 grid((unsigned)(m_tiles * n_tiles * splits));
    int8_tiles<BM, DELTA, GATHER><<<grid, kWaves * 64, 0, s>>>(a, m_tiles, n_tiles, n_fast, splits, table, partial);
    if (splits > 1) {
        const dim3 joins((unsigned)(m_tiles * n_tiles * (BM / 8)));
        int8_tiles_join<BM, DELTA, GATHER><<<joins, kWaves * 64, 0, s>>>(a, m_tiles, n_tiles, n_fast, splits, table, partial);
    }
    return hipGetLastError();
}

template <bool DELTA, bool GATHER>
hipError_t planned(const TileArgs &a, void *workspace, hipStream_t s)
{
    const Plan p = plan_of(a.m, a.d_out, a.d_in, DELTA, GATHER ? a.n_variants : 0);
    return p.tall ? tiles<128, DELTA, GATHER>(a, p.splits, workspace, s) : tiles<64, DELTA, GATHER>(a, p.splits, workspace, s);
}

size_t partial_bytes(int64_t m, int64_t d_out, int64_t d_in, bool delta, int32_t variants)
{
    const Plan p = plan_of(m, d_out, d_in, delta, variants);
    return part_bytes(p.tall, m, d_out, p.splits, delta, variants);
}

int64_t whole(int64_t d_in) { return (d_in + 31) / 32 * 32; }

size_t sums_bytes(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    if (n_variants == 0)
        return partial_bytes(m, d_out, d_in, false, 0);
    // whether the call has ids is not known here
    const size_t one = partial_bytes(m, d_out, d_in, true, 0), many = partial_bytes(m, d_out, d_in, true, n_variants);
    return table_bytes(m, n_variants) + (one > many ? one : many);
}

// Whether rows that end inside 32 columns are copied for the tiles: the copy of all
// variants' signs has to be paid for by the tokens (333 tokens of 3 variants through
// 1000 x 4104: by the kernel for 64 tokens 60 us, copied 33), and stays below 2^28 bytes.
// A row of 8 columns is less than a chunk, which so would begin in front of w (4096 tokens
// through 8192 x 8 192 us by the kernel for 64 tokens, rows of 16 columns 71).
size_t pad_bytes(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    return (size_t)(m * whole(d_in) + n_variants * (d_out * (whole(d_in) / 8)) + 31) / 16 * 16;
}
bool pads(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    return d_in % 32 != 0 && d_in > 8 && n_variants <= m / 4 && pad_bytes(m, n_variants, d_out, d_in) <= (size_t)1 << 28;
}

}  // namespace

bool int8_tiles_take(const Int8Args &a)
{
    // a launch takes fewer than 2^32 threads
    const int64_t most = token_tiles<64>(a.m, a.ids ? a.n_variants : 0) * ((a.d_out + kBN - 1) / kBN);
    const bool rows = a.d_in % 32 == 0 ? ((uintptr_t)a.signs & 3) == 0 : pads(a.m, a.n_variants, a.d_out, a.d_in);
    return rows && most < (1 << 23);
}

size_t int8_tiles_workspace_bytes(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    return sums_bytes(m, n_variants, d_out, whole(d_in)) +
           (pads(m, n_variants, d_out, d_in) ? pad_bytes(m, n_variants, d_out, d_in) : 0);
}

hipError_t launch_int8_tiles(const Int8Args &args, void *workspace, hipStream_t s)
{
    TileArgs a{args, args.d_in};
    if (a.d_in % 32 != 0) {
        a.d_in = whole(a.d_in);
        const int64_t G = a.w_stride / 8, padded = a.d_in / 8;
        uint8_t *copies = static_cast<uint8_t *>(workspace) + sums_bytes(a.m, a.n_variants, a.d_out, a.d_in);
        uint64_t *q_to = reinterpret_cast<uint64_t *>(copies);
        uint32_t *signs_to = reinterpret_cast<uint32_t *>(copies + a.m * a.d_in);
        const int64_t q_units = a.m * padded, sign_units = a.n_variants * a.d_out * (padded / 4);
        int8_pad<<<(unsigned)((q_units + sign_units + 255) / 256), 256, 0, s>>>(
            reinterpret_cast<const uint64_t *>(a.q), q_to, (uint32_t)q_units, a.signs, signs_to, (uint32_t)sign_units, (uint32_t)G,
            (uint32_t)padded);
        a.q = reinterpret_cast<const int8_t *>(q_to);
        if (a.signs)
            a.signs = reinterpret_cast<const uint8_t *>(signs_to);
    }
    if (!a.signs)
        return planned<false, false>(a, workspace, s);
    return a.ids ? planned<true, true>(a, workspace, s) : planned<true, false>(a, workspace, s);
}

}  // namespace bd
