// Product of int8 rows with an int8 base and 1-bit deltas, few tokens
// (bitdelta_linear_int8):
//
//   y[i,r] = s_i (c_r sum_k q[i,k] w[r,k] + alpha_v[r] sum_k q[i,k] sign_v[r,k])
//
// Both sums are of whole numbers and exact in int32 (|sum| <= 131064 * 2^14 <
// 2^31), so they may be cut in any way.  Bound by reading w and the signs.
#include <type_traits>

#include "int8_device.h"
#include "int8_tiles.h"

namespace bd {
namespace {

constexpr int kRange = 512;       // columns a wave takes at a time
constexpr int kXcds = 8;

// lane p: the token at place p of the order by variant, and its variant
struct Order {
    int token, variant;
};

// Of the `group` (at most 64) tokens from t0 on, as numbers from t0; variants outside are n_variants.
__device__ __forceinline__ Order order_by_variant(const Int8Args &a, int64_t t0, int group)
{
    const int lane = threadIdx.x & 63;
    Order o{lane, 0};
    if (!a.ids)
        return o;
    const int id = lane < group ? a.ids[t0 + lane] : 0x7FFFFFFF;
    const bool known = (unsigned)id < (unsigned)a.n_variants;
    const int key = lane < group ? (known ? id : a.n_variants) : 0x7FFFFFFF;
    int place = 0;
    for (int i = 0; i < group; ++i) {
        const int other = __builtin_amdgcn_readlane(key, i);
        place += other < key || (other == key && i < lane) ? 1 : 0;
    }
    place = lane < group ? place : lane;
    o.token = __builtin_amdgcn_ds_permute(place * 4, lane);
    o.variant = __builtin_amdgcn_ds_permute(place * 4, key);
    return o;
}

// The signs of a range as one load brings them (16 bytes of a lane group) to the
// dwords that twice_sign_bytes takes: of the 128 signs of lane group g, halfwords p and
// 4 + p go to group p's dword g.
__device__ __forceinline__ void to_groups(const u32x4 &s, uint32_t (&e)[4])
{
    e[0] = __builtin_amdgcn_perm(s[2], s[0], 0x05040100u);
    e[1] = __builtin_amdgcn_perm(s[2], s[0], 0x07060302u);
    e[2] = __builtin_amdgcn_perm(s[3], s[1], 0x05040100u);
    e[3] = __builtin_amdgcn_perm(s[3], s[1], 0x07060302u);
    auto swap32 = [](uint32_t &p, uint32_t &q) {
        const auto o = __builtin_amdgcn_permlane32_swap(p, q, false, false);
        p = o[0], q = o[1];
    };
    auto swap16 = [](uint32_t &p, uint32_t &q) {
        const auto o = __builtin_amdgcn_permlane16_swap(p, q, false, false);
        p = o[0], q = o[1];
    };
    swap32(e[0], e[2]);
    swap32(e[1], e[3]);
    swap16(e[0], e[1]);
    swap16(e[2], e[3]);
}

// How rows are read: of whole 128 or 64 columns (signs by 16 or 8 bytes), or of any
// eights (signs by dwords, at any alignment).  Then no access is partly past a
// buffer's end, and each loads as often whatever the place, so that the loads of
// several variants can be on their way together.
enum Rows { kBy128, kBy64, kByEights };

// Signs of variant v (one that does not exist: zeros), rows n0 + lane % 16, the range from column k0 on.
template <Rows R, int CACHE>
__device__ __forceinline__ u32x4 load_signs(const Int8Args &a, int v, int64_t n0, int64_t k0)
{
    const int col = threadIdx.x & 15, quad = (threadIdx.x & 63) >> 4;
    const int64_t N = a.d_out, G = a.d_in >> 3;
    const bool known = (unsigned)v < (unsigned)a.n_variants;
    const uint8_t *base = a.signs + (known ? v : 0) * N * G;
    // signs may start on any byte: a buffer of whole dwords from the one that holds the first
    const uint32_t slip = R == kByEights ? (uint32_t)((uintptr_t)base & 3) : 0;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(base - slip, (N * G + slip + 3) & ~(int64_t)3);
    const uint32_t in_row = (uint32_t)(k0 >> 3) + quad * 16;
    const uint32_t at = known ? (uint32_t)((n0 + col) * G) + in_row + slip : kInvalidOffset;
    if constexpr (R == kBy128)
        return __builtin_amdgcn_raw_buffer_load_b128(rs, in_row < G ? at : kInvalidOffset, 0, CACHE);
    if constexpr (R == kBy64) {
        const auto lo = __builtin_amdgcn_raw_buffer_load_b64(rs, in_row < G ? at : kInvalidOffset, 0, CACHE);
        const auto hi = __builtin_amdgcn_raw_buffer_load_b64(rs, in_row + 8 < G ? at + 8 : kInvalidOffset, 0, CACHE);
        return (u32x4){lo[0], lo[1], hi[0], hi[1]};
    }
    uint32_t d[5];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        d[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, in_row < G ? (at & ~3u) + 4 * i : kInvalidOffset, 0, 0);
    u32x4 s;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = __builtin_amdgcn_alignbyte(d[i + 1], d[i], at & 3);
    return s;
}

// y of 16 channels from n0 on and 16 T tokens (from place 16 block on) from the sums that a wave holds:
// number c of lane l is row 4 (l / 16) + c of a block, channel l % 16.
template <int T, bool DELTA>
__device__ __forceinline__ void finish(const Int8Args &a, int64_t t0, int count, int64_t n0, const Order &order, int block,
                                       const i32x4 (&acc)[T], const i32x4 (&accd)[T])
{
    const int lane = threadIdx.x & 63;
    const int64_t n = n0 + (lane & 15), N = a.d_out;
    const float c = n < N ? a.w_scale[n] : 0.0f;
#pragma unroll
    for (int b = 0; b < T; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int place = 16 * (block + b) + (lane >> 4) * 4 + i;
            const int token = DELTA ? __shfl(order.token, place) : place, v = DELTA ? __shfl(order.variant, place) : 0;
            if (place >= count || n >= N)
                continue;
            const int64_t t = t0 + token;
            float y = 0.0f;
            if (!DELTA || (unsigned)v < (unsigned)a.n_variants)
                y = combine(a.q_scale[t], c, acc[b][i], DELTA ? a.alpha[a.per_matrix ? v : v * N + n] : 0.0f, accd[b][i]);
            if (a.f32)
                static_cast<float *>(a.y)[t * N + n] = y;
            else
                static_cast<uint16_t *>(a.y)[t * N + n] = to_bf16(y);
        }
}

// Up to 16 tokens.  One workgroup: 16 channels, NW waves, each with every NW-th
// range of the columns.  Of a range the 16 rows of w go straight into the wave's
// part of LDS, 512 contiguous bytes of a row at a time; chunk c (16 bytes) of row r
// stands at c ^ r there, so that the operands' reads meet all banks.  The tokens'
// numbers are read into registers, and of each variant's signs 64 bytes of every row
// in one load.  Lane group p (lanes 16 p ..) of the four holds, of 128 columns,
// 16 p .. and 64 + 16 p ..: two 16-byte operands of w and q, and as one dword their
// signs, which a 4 x 4 transpose over the lane groups brings there.
//
// The tokens are ordered by variant; a variant's product is formed for all 16 and
// kept for its own.
// MANY: with variant ids.
// One token through 8192 x 8192 with one delta 15.7 us, 4.8 TB/s; 16 of 14 variants
// through 10240 x 8192 50 us, 3.5 TB/s, between the variants' 64-byte pieces of rows.
template <int NW, bool DELTA, bool MANY, Rows R>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4)))
void int8_stream(Int8Args a)
{
    __shared__ __attribute__((aligned(16))) uint8_t tiles[NW][16 * kRange];
    __shared__ int32_t token_s[16], variant_s[16];

    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16, K = a.d_in, N = a.d_out;
    const int count = (int)a.m;
    const Order order = DELTA ? order_by_variant(a, 0, count) : Order{lane, 0};
    if (wave == 0 && lane < 16) {
        token_s[lane] = order.token;
        variant_s[lane] = order.variant;
    }
    const uint32_t qoff = col < count ? (uint32_t)(__shfl(order.token, col) * K) : kInvalidOffset;
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.q, a.m * K), rw = make_rsrc(a.w, N * K);
    // Columns k .. k + 15 of a row at byte `off` of a buffer.  No access is
    // partly past a buffer's end: with rows of whole 16 columns none can be,
    // other rows are read by eights.
    const bool eights = R == kByEights && K % 16 != 0;
    auto sixteen = [&](__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t k) -> u32x4 {
        if (!eights)
            return __builtin_amdgcn_raw_buffer_load_b128(r, k < K ? off + k : kInvalidOffset, 0, 0);
        const auto lo = __builtin_amdgcn_raw_buffer_load_b64(r, k < K ? off + k : kInvalidOffset, 0, 0);
        const auto hi = __builtin_amdgcn_raw_buffer_load_b64(r, k + 8 < K ? off + k + 8 : kInvalidOffset, 0, 0);
        return (u32x4){lo[0], lo[1], hi[0], hi[1]};
    };

    // rows 2 i and 2 i + 1 of w, chunk lane % 32 of a row in LDS; the range's columns
    // go into the scalar offset, which is not checked, so a chunk past the row's end
    // and a row that does not exist have lane offsets out of range (zeros)
    uint8_t *const tile = tiles[wave];
    uint32_t woff[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 2 * i + (lane >> 5);
        woff[i] = n0 + row < N ? (uint32_t)((n0 + row) * K) + ((lane & 31) ^ row) * 16 : kInvalidOffset;
    }
    auto load_w = [&](int64_t k0) {
        const int64_t left = K - k0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 2 * i + (lane >> 5), at = ((lane & 31) ^ row) * 16;
            if (!eights)
                copy16<kStream>(rw, tile + i * 1024, at < left ? woff[i] : kInvalidOffset, (uint32_t)k0);
            else
                *reinterpret_cast<u32x4 *>(tile + i * 1024 + lane * 16) =
                    sixteen(rw, n0 + row < N ? (uint32_t)((n0 + row) * K) : kInvalidOffset, (uint32_t)k0 + at);
        }
    };
    auto operand = [&](int j) { return *reinterpret_cast<const u32x4 *>(tile + col * kRange + (((4 * j + quad) ^ col) * 16)); };
    // past the row's end the tokens are zero, whatever the signs' bytes hold there
    u32x4 x[8];
    auto load_x = [&](int64_t k0) {
        if (R != kByEights && k0 + kRange <= K) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __builtin_amdgcn_raw_buffer_load_b128(rq, qoff + (uint32_t)k0 + quad * 16 + j * 64, 0, 0);
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = sixteen(rq, qoff, (uint32_t)k0 + j * 64 + quad * 16);
    };
    // the places where another variant's tokens begin
    uint64_t heads = 1;
    if (DELTA && a.ids) {
        const int before = __shfl(order.variant, lane ? lane - 1 : 0);
        heads = __ballot(lane < count && (lane == 0 || order.variant != before));
    }
    i32x4 acc = {0, 0, 0, 0}, accd = {0, 0, 0, 0};
    int64_t k0 = (int64_t)wave * kRange;
    u32x4 one;
    load_w(k0);
    if (DELTA && !MANY)
        one = load_signs<R, kStream>(a, 0, n0, k0);
    for (; k0 < K; k0 += NW * kRange) {
        load_x(k0);
        // The signs of the variants: of many, kAhead are on their way; of one, the next range's.
        constexpr int kAhead = MANY ? 4 : 0;
        struct Signs {
            u32x4 s;
            int begin, end;
        } ring[kAhead + 1];
        uint64_t left = heads;
        auto fetch = [&](Signs &r) {
            // past the last variant: nothing, loaded all the same
            r.begin = left ? __builtin_ctzll(left) : 0;
            const int v = left ? __builtin_amdgcn_readlane(order.variant, r.begin) : -1;
            left &= left - 1;
            r.end = v < 0 ? 0 : left ? __builtin_ctzll(left) : count;
            r.s = load_signs<R, kStream>(a, v, n0, k0);
        };
        if constexpr (MANY) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                fetch(ring[i]);
        }
        // the tile's copies are older than the loads of x, which are needed now too
        wait_vmcnt_lgkm0<0>();
        __builtin_amdgcn_sched_barrier(0);
        // with a delta the sums of 2 b - 1: the -1 here, 2 b below
        const u32x4 minus_ones = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            acc = mfma16(x[j], operand(j), acc);
            if constexpr (DELTA)
                accd = mfma16(x[j], minus_ones, accd);
        }
        wait_lgkm0();      // the operands are read: the next range's rows may go where they were
        __builtin_amdgcn_sched_barrier(0);
        load_w(k0 + NW * kRange);     // past the last range: zeros
        __builtin_amdgcn_sched_barrier(0);
        // d and the product of x and a variant's sign bits, twice
        auto product = [&](const u32x4 &signs, i32x4 d) {
            uint32_t e[4];
            to_groups(signs, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u32x4 b;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    b[c] = twice_sign_bytes(e[j >> 1], (j & 1) * 4 + c);
                d = mfma16(x[j], b, d);
            }
            return d;
        };
        if constexpr (DELTA) {
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                to_sign_order(x[j], x[j + 1]);
        }
        if constexpr (MANY) {
            bool more = true;
            while (more) {
#pragma unroll
                for (int i = 0; i <= kAhead; ++i) {
                    fetch(ring[(i + kAhead) % (kAhead + 1)]);
                    const Signs &r = ring[i];
                    if (r.begin == r.end) {
                        more = false;
                        break;
                    }
                    const i32x4 d = product(r.s, (i32x4){0, 0, 0, 0});
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        accd[c] += (unsigned)(quad * 4 + c - r.begin) < (unsigned)(r.end - r.begin) ? d[c] : 0;
                }
            }
        } else if constexpr (DELTA) {
            const u32x4 signs = one;
            one = load_signs<R, kStream>(a, 0, n0, k0 + NW * kRange);
            accd = product(signs, accd);
        }
    }
    // the waves' sums, each where its rows of w were: the last copies must have landed
    wait_vmcnt_lgkm0<0>();
    reinterpret_cast<i32x4 *>(tile)[lane] = acc;
    if constexpr (DELTA)
        reinterpret_cast<i32x4 *>(tile)[64 + lane] = accd;
    __syncthreads();
    // number c of lane l: row 4 (l / 16) + c, channel l % 16
    for (int at = threadIdx.x; at < 256; at += NW * 64) {
        const int row = at >> 4, ch = at & 15, from = (row >> 2) * 16 + ch;
        int A = 0, B = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const i32x4 *other = reinterpret_cast<const i32x4 *>(tiles[w]);
            A += other[from][row & 3];
            if constexpr (DELTA)
                B += other[64 + from][row & 3];
        }
        const int64_t n = n0 + ch;
        if (row >= count || n >= N)
            continue;
        const int64_t t = DELTA ? token_s[row] : row;
        const int v = DELTA ? variant_s[row] : 0;
        float y = 0.0f;
        if (!DELTA || (unsigned)v < (unsigned)a.n_variants)
            y = combine(a.q_scale[t], a.w_scale[n], A, DELTA ? a.alpha[a.per_matrix ? v : v * N + n] : 0.0f, B);
        if (a.f32)
            static_cast<float *>(a.y)[t * N + n] = y;
        else
            static_cast<uint16_t *>(a.y)[t * N + n] = to_bf16(y);
    }
}

// The same for more tokens: 64 channels (four waves of 16) and 16 T tokens a
// workgroup, which takes every `splits`-th range of the columns: neighbouring
// ranges, which share lines of signs, are read on one die at a time.  All waves
// work on one range and share the tokens' numbers in LDS; the signs of the
// following variants, the next range's among them, are on their way while one is used.
// 32 tokens through 50257 x 8192 without a delta 94 us, 4.4 TB/s; 61 tokens of 14
// variants through 8192 x 28672 210 us with the join, 3.0 TB/s: signs are spread to bytes
// by vector instructions (the waves' cycles: 41 % issue, 25 % wait to, 33 % wait for data),
// two waves a SIMD hide little, and lines of signs are fetched twice (0.90 GB for 0.62).
constexpr int kMidWaves = 4;

template <int T, bool DELTA, bool MANY, Rows R>
__global__ __launch_bounds__(kMidWaves * 64) __attribute__((amdgpu_waves_per_eu(2, 2)))
void int8_mid(Int8Args a, int splits, i32x4 *__restrict__ partial)
{
    __shared__ __attribute__((aligned(16))) uint8_t xs[16 * T * kRange], ws[kMidWaves][16 * kRange];

    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t K = a.d_in, N = a.d_out;
    // blocks of tokens that meet the same rows of w on one die, near in time
    const unsigned across = (unsigned)((a.m + 16 * T - 1) / (16 * T)) * splits;
    const unsigned turn = blockIdx.x / (kXcds * across), in_turn = blockIdx.x % (kXcds * across);
    const int64_t group_n = (int64_t)turn * kXcds + in_turn % kXcds, n0 = group_n * 64 + wave * 16;
    if (group_n * 64 >= N)
        return;
    const int split = (int)(in_turn / kXcds % splits), block = (int)(in_turn / kXcds / splits);
    const int64_t t0 = (int64_t)block * (16 * T);
    const int count = (int)(a.m - t0 < 16 * T ? a.m - t0 : 16 * T);
    const Order order = DELTA ? order_by_variant(a, t0, count) : Order{lane, 0};

    const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.q, a.m * K), rw = make_rsrc(a.w, N * K);
    const bool eights = R == kByEights && K % 16 != 0;
    auto sixteen = [&](__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t k) -> u32x4 {
        const auto lo = __builtin_amdgcn_raw_buffer_load_b64(r, k < K ? off + k : kInvalidOffset, 0, 0);
        const auto hi = __builtin_amdgcn_raw_buffer_load_b64(r, k + 8 < K ? off + k + 8 : kInvalidOffset, 0, 0);
        return (u32x4){lo[0], lo[1], hi[0], hi[1]};
    };
    // copies of two rows each, as in int8_stream; the waves share the tokens' rows
    uint8_t *const tile = ws[wave];
    uint32_t woff[8], xoff[2 * T];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 2 * i + (lane >> 5);
        woff[i] = n0 + row < N ? (uint32_t)((n0 + row) * K) : kInvalidOffset;
    }
#pragma unroll
    for (int i = 0; i < 2 * T; ++i) {
        const int row = 2 * (wave * 2 * T + i) + (lane >> 5);
        const int token = DELTA ? __shfl(order.token, row) : row;
        xoff[i] = row < count ? (uint32_t)((t0 + token) * K) : kInvalidOffset;
    }
    auto load = [&](int64_t k0) {
        const int64_t left = K - k0;
        auto rows = [&](__amdgpu_buffer_rsrc_t r, uint8_t *to, uint32_t off, int first) {
            const int at = ((lane & 31) ^ ((first + (lane >> 5)) & 15)) * 16;
            if (eights)
                *reinterpret_cast<u32x4 *>(to + lane * 16) = sixteen(r, off, (uint32_t)k0 + at);
            else
                copy16(r, to, at < left ? off + at : kInvalidOffset, (uint32_t)k0);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i)
            rows(rw, tile + i * 1024, woff[i], 2 * i);
#pragma unroll
        for (int i = 0; i < 2 * T; ++i)
            rows(rq, xs + (wave * 2 * T + i) * 1024, xoff[i], 2 * (wave * 2 * T + i));
    };

    i32x4 acc[T], accd[T];
#pragma unroll
    for (int b = 0; b < T; ++b)
        acc[b] = accd[b] = (i32x4){0, 0, 0, 0};
    uint64_t heads = 1;
    if (DELTA && a.ids) {
        const int before = __shfl(order.variant, lane ? lane - 1 : 0);
        heads = __ballot(lane < count && (lane == 0 || order.variant != before));
    }
    const unsigned all = (unsigned)((K + kRange - 1) / kRange);

    // A stream of signs over variants and ranges, kAhead of them on their way (more
    // cost registers: 61 tokens of 14 variants through 8192 x 28672 209 us with one or
    // two, 233 with three, 245 with five); a range's variants are filled up to whole
    // turns of the ring with empty ones.
    constexpr int kAhead = T == 4 ? 1 : 2;
    struct Signs {
        u32x4 s;
        int begin, end;
    } ring[kAhead + 1];
    const int turns = (__builtin_popcountll(heads) + kAhead) / (kAhead + 1);
    uint64_t left = heads;
    int fetched = 0;
    unsigned range = split;
    auto fetch = [&](Signs &r) {
        const bool real = left && range < all;
        r.begin = real ? __builtin_ctzll(left) : 0;
        const int v = real ? __builtin_amdgcn_readlane(order.variant, r.begin) : -1;
        left &= left - 1;
        r.end = !real ? 0 : left ? __builtin_ctzll(left) : count;
        r.s = load_signs<R, kStream>(a, v, n0, (int64_t)range * kRange);
        if (++fetched == turns * (kAhead + 1)) {
            fetched = 0;
            left = heads;
            range += splits;
        }
    };
    if ((unsigned)split < all)
        load((int64_t)split * kRange);
    u32x4 one;          // of one variant for all: the next range's signs
    if constexpr (MANY) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            fetch(ring[i]);
    } else if constexpr (DELTA) {
        one = load_signs<R, kStream>(a, 0, n0, (int64_t)split * kRange);
    }
    for (unsigned i = split; i < all; i += splits) {
        wait_vmcnt_lgkm0<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const u32x4 minus_ones = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
        u32x4 x[MANY ? T : 1][MANY ? 8 : 1];
        if constexpr (!MANY) {
            // one variant at most: base and delta from the same reading of the tokens
            uint32_t e[4] = {0, 0, 0, 0};
            if constexpr (DELTA) {
                to_groups(one, e);
                one = load_signs<R, kStream>(a, 0, n0, (int64_t)(i + splits) * kRange);
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const int at0 = col * kRange + (((4 * j + quad) ^ col) * 16), at1 = col * kRange + (((4 * j + 4 + quad) ^ col) * 16);
                const u32x4 w0 = *reinterpret_cast<const u32x4 *>(tile + at0), w1 = *reinterpret_cast<const u32x4 *>(tile + at1);
                u32x4 b0, b1;
                if constexpr (DELTA)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        b0[c] = twice_sign_bytes(e[j >> 1], c);
                        b1[c] = twice_sign_bytes(e[j >> 1], 4 + c);
                    }
#pragma unroll
                for (int b = 0; b < T; ++b) {
                    u32x4 x0 = *reinterpret_cast<const u32x4 *>(xs + b * 16 * kRange + at0);
                    u32x4 x1 = *reinterpret_cast<const u32x4 *>(xs + b * 16 * kRange + at1);
                    acc[b] = mfma16(x0, w0, acc[b]);
                    acc[b] = mfma16(x1, w1, acc[b]);
                    if constexpr (DELTA) {
                        accd[b] = mfma16(x0, minus_ones, accd[b]);
                        accd[b] = mfma16(x1, minus_ones, accd[b]);
                        to_sign_order(x0, x1);
                        accd[b] = mfma16(x0, b0, accd[b]);
                        accd[b] = mfma16(x1, b1, accd[b]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = col * kRange + (((4 * j + quad) ^ col) * 16);
                const u32x4 w = *reinterpret_cast<const u32x4 *>(tile + at);
#pragma unroll
                for (int b = 0; b < T; ++b)
                    x[b][j] = *reinterpret_cast<const u32x4 *>(xs + b * 16 * kRange + at);
#pragma unroll
                for (int b = 0; b < T; ++b) {
                    acc[b] = mfma16(x[b][j], w, acc[b]);
                    accd[b] = mfma16(x[b][j], minus_ones, accd[b]);
                }
            }
        }
        wait_lgkm0();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load((int64_t)(i + splits) * kRange);     // past the last range: zeros
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MANY) {
#pragma unroll
            for (int b = 0; b < T; ++b)
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    to_sign_order(x[b][j], x[b][j + 1]);
            for (int u = 0; u < turns; ++u)
#pragma unroll
                for (int slot = 0; slot <= kAhead; ++slot) {
                    fetch(ring[(slot + kAhead) % (kAhead + 1)]);
                    Signs &r = ring[slot];
                    if (r.begin == r.end)
                        continue;
                    uint32_t e[4];
                    to_groups(r.s, e);
                    u32x4 bytes[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            bytes[j][c] = twice_sign_bytes(e[j >> 1], (j & 1) * 4 + c);
#pragma unroll
                    for (int b = 0; b < T; ++b)
                        if (r.begin < 16 * b + 16 && r.end > 16 * b) {
                            // two chains, as one waits for its own sums
                            i32x4 d0 = {0, 0, 0, 0}, d1 = {0, 0, 0, 0};
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                d0 = mfma16(x[b][j], bytes[j], d0);
                                d1 = mfma16(x[b][j + 1], bytes[j + 1], d1);
                            }
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int place = 16 * b + quad * 4 + c;
                                accd[b][c] += (unsigned)(place - r.begin) < (unsigned)(r.end - r.begin) ? d0[c] + d1[c] : 0;
                            }
                        }
                }
        }
    }
    // copies still on their way must land before the workgroup's LDS is released
    __builtin_amdgcn_s_waitcnt(0);
    if (splits > 1) {
        const int64_t blocks = (a.m + 16 * T - 1) / (16 * T), channels = (N + 15) / 16;
        i32x4 *out = partial + (((int64_t)split * blocks + block) * channels + (n0 >> 4)) * (T * (DELTA ? 2 : 1) * 64);
        if (n0 < N)
#pragma unroll
            for (int b = 0; b < T; ++b) {
                out[b * 64 + lane] = acc[b];
                if constexpr (DELTA)
                    out[(T + b) * 64 + lane] = accd[b];
            }
        return;
    }
    finish<T, DELTA>(a, t0, count, n0, order, 0, acc, accd);
}

// Adds up the splits' sums of int8_mid: a wave for 16 channels and 16 tokens.
template <int T, bool DELTA>
__global__ __launch_bounds__(256) void int8_join(Int8Args a, int splits, const i32x4 *__restrict__ partial)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t blocks = (a.m + 16 * T - 1) / (16 * T), channels = (a.d_out + 15) / 16;
    const int64_t at = (int64_t)blockIdx.x * 4 + wave;
    if (at >= blocks * channels * T)
        return;
    const int b = (int)(at % T);
    const int64_t block = at / T / channels, channel = at / T % channels, t0 = block * (16 * T);
    const int count = (int)(a.m - t0 < 16 * T ? a.m - t0 : 16 * T);
    if (16 * b >= count)
        return;
    constexpr int kSums = T * (DELTA ? 2 : 1) * 64;
    const i32x4 *in = partial + (block * channels + channel) * kSums + b * 64 + lane;
    i32x4 acc[1] = {{0, 0, 0, 0}}, accd[1] = {{0, 0, 0, 0}};
    for (int split = 0; split < splits; ++split, in += blocks * channels * kSums) {
        acc[0] += in[0];
        if constexpr (DELTA)
            accd[0] += in[T * 64];
    }
    finish<1, DELTA>(a, t0, count, channel * 16, DELTA ? order_by_variant(a, t0, count) : Order{lane, 0}, b, acc, accd);
}

// Splits of a call's columns: as many as give each CU two workgroups, of two ranges
// at least, or one where each range meets many variants' signs.
//   us, 64 tokens x 8192 columns, ranges at least    4      2      1
//     1024 channels, none                           18.2   16.5   17.0
//                    one delta                      20.1   17.6   18.7
//                    4 variants                     31.3   26.0   26.4
//                   14                              48.2   34.7   30.8
//     2048 channels, none                           16.4   16.1   17.4
//                    one delta                      21.0   20.3   22.7
//                   14                              49.7   37.3   34.3
template <int T>
int mid_splits(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    const int64_t groups = (d_out + 63) / 64 * ((m + 16 * T - 1) / (16 * T)), ranges = (d_in + kRange - 1) / kRange;
    int64_t s = 1;
    while (groups * s < 512 && ranges / (s + 1) >= (n_variants >= 8 ? 1 : 2) && s < 16)
        ++s;
    return (int)s;
}

Rows rows_of(const Int8Args &a)
{
    if (((uintptr_t)a.signs & 3) != 0)
        return kByEights;
    return a.d_in % 128 == 0 ? kBy128 : a.d_in % 64 == 0 ? kBy64 : kByEights;
}

template <int T, bool DELTA, bool MANY>
hipError_t mid(const Int8Args &a, void *workspace, hipStream_t s)
{
    const int64_t groups = ((a.d_out + 63) / 64 + kXcds - 1) / kXcds * kXcds, blocks = (a.m + 16 * T - 1) / (16 * T);
    const int splits = mid_splits<T>(a.m, a.n_variants, a.d_out, a.d_in);
    i32x4 *partial = static_cast<i32x4 *>(workspace);
    const dim3 grid((unsigned)(groups * blocks * splits));
    switch (rows_of(a)) {
    case kBy128: int8_mid<T, DELTA, MANY, kBy128><<<grid, kMidWaves * 64, 0, s>>>(a, splits, partial); break;
    case kBy64: int8_mid<T, DELTA, MANY, kBy64><<<grid, kMidWaves * 64, 0, s>>>(a, splits, partial); break;
    default: int8_mid<T, DELTA, MANY, kByEights><<<grid, kMidWaves * 64, 0, s>>>(a, splits, partial); break;
    }
    if (splits > 1) {
        const dim3 joins((unsigned)((blocks * ((a.d_out + 15) / 16) * T + 3) / 4));
        int8_join<T, DELTA><<<joins, 256, 0, s>>>(a, splits, partial);
    }
    return hipGetLastError();
}

template <int T>
size_t mid_workspace(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    const int splits = mid_splits<T>(m, n_variants, d_out, d_in);
    return splits == 1 ? 0 : (size_t)(splits * ((m + 16 * T - 1) / (16 * T)) * ((d_out + 15) / 16)) * (T * (n_variants ? 2 : 1) * 64 * 16);
}

template <int NW, bool DELTA, bool MANY>
hipError_t stream(const Int8Args &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.d_out + 15) / 16));
    switch (rows_of(a)) {
    case kBy128: int8_stream<NW, DELTA, MANY, kBy128><<<grid, NW * 64, 0, s>>>(a); break;
    case kBy64: int8_stream<NW, DELTA, MANY, kBy64><<<grid, NW * 64, 0, s>>>(a); break;
    default: int8_stream<NW, DELTA, MANY, kByEights><<<grid, NW * 64, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

// Whether more than 64 tokens of many variants go in lots of 64: a tile has one
// variant's tokens, few of its rows, and reads all of the base's for them, a lot
// reads the base and its variants' signs once.
//   us                        tiles   lots          tiles   lots          tiles   lots
//                             128 tokens            192 tokens            256 tokens
//   8192 x 8192, 4 variants      80     76            107    106             96    106
//               14              154    113            158    173            159    191
//               38              253    160            289    264            298    312
//   1024 x 8192, 14              40     37             42     47             46     43
//               38               59     41             68     57             73     55
//   28672 x 8192, 14            420    413            437    579            454    688
//               38              815    604            936    867            985   1103
bool in_lots(const Int8Args &a)
{
    const int64_t lots = (a.m + 63) / 64;
    return a.ids && 3 * lots * lots <= (a.n_variants < a.m ? a.n_variants : a.m);
}

}  // namespace

// Up to 16 tokens the waves of a workgroup share the columns, up to 64 they share
// the tokens; from there on the tiles are used.  8192 x 8192, one delta: 16 tokens
// 21 us, 17 tokens 25, 64 tokens 33, 65 tokens 41 (the base from memory each time).
constexpr int64_t kMidFrom = 17, kTilesFrom = 65;

// Where the tiles do not take more than kSlice tokens they go by slices: a launch
// has fewer than 2^32 threads.
constexpr int64_t kSlice = 1 << 20;

size_t linear_int8_workspace_bytes(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    if (m < kMidFrom)
        return 0;
    size_t most = m < kTilesFrom ? 0 : int8_tiles_workspace_bytes(m, n_variants, d_out, d_in);
    if (m > kSlice) {
        for (const int64_t slice : {kSlice, m % kSlice}) {
            const size_t bytes = linear_int8_workspace_bytes(slice, n_variants, d_out, d_in);
            most = most > bytes ? most : bytes;
        }
        return most;
    }
    const size_t mid = m <= 32 ? mid_workspace<2>(m, n_variants, d_out, d_in)
                               : mid_workspace<4>(m, n_variants, d_out, d_in);
    return mid > most ? mid : most;
}

hipError_t launch_linear_int8(const Int8Args &a, void *workspace, hipStream_t s)
{
    if (a.m >= kTilesFrom && !in_lots(a) && int8_tiles_take(a))
        return launch_int8_tiles(a, workspace, s);
    if (a.m > kSlice) {
        for (int64_t t = 0; t < a.m; t += kSlice) {
            Int8Args part = a;
            part.m = a.m - t < kSlice ? a.m - t : kSlice;
            part.q += t * a.d_in;
            part.q_scale += t;
            if (a.ids)
                part.ids += t;
            part.y = static_cast<char *>(a.y) + t * a.d_out * (a.f32 ? 4 : 2);
            const hipError_t e = launch_linear_int8(part, workspace, s);
            if (e != hipSuccess)
                return e;
        }
        return hipSuccess;
    }
    if (a.m < kMidFrom)
        return a.ids ? stream<8, true, true>(a, s) : a.signs ? stream<8, true, false>(a, s) : stream<8, false, false>(a, s);
    if (a.m <= 32)
        return a.ids ? mid<2, true, true>(a, workspace, s) : a.signs ? mid<2, true, false>(a, workspace, s) : mid<2, false, false>(a, workspace, s);
    return a.ids ? mid<4, true, true>(a, workspace, s) : a.signs ? mid<4, true, false>(a, workspace, s) : mid<4, false, false>(a, workspace, s);
}

}  // namespace bd
