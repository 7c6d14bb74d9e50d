// Causal attention over a paged cache, with shared prefixes
// (bitdelta_attention).
//
// All kernels keep the running maximum m, sum l and weighted value o of each
// row (a token and query head) over the keys seen so far,
//   m' = max(m, s);  l = l 2^(m - m') + sum 2^(s - m');  o likewise with v,
// s = log2(e) scale q.k, in fp32; the weights 2^(s - m') enter the product
// with v rounded to bf16 (half a step, 2^-8 relative), as the matrix
// instructions take them, and l sums the rounded ones in fp32.  Keys that a row does
// not see have s = -inf.  States over parts of the keys are joined by the
// same formula (attention_join).
//
// Scores are formed transposed, S' = K Q', so that a lane holds several keys
// of one row: the maximum and the sum are mostly inside the lane, and the
// weights are already where the second product O' = V' P' wants its right
// operand.  The order of the keys in that product is free as long as V' uses
// the same, so no weight moves between lanes; V' fragments are read from
// row-major V in LDS by the transposing LDS load.
//
// attention_schedule.h says which kernel takes which rows and keys.
#include <limits.h>

#include <type_traits>

#include "attention_schedule.h"
#include "bd_device.h"
#include "decoder_launch.h"

namespace bd {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f;

struct AttnArgs {
    Sched s;
    const uint16_t *q;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    uint16_t *out;
    int64_t *cut;       // what the join has to know: key tiles of a split, units of a workgroup, first unit of each sequence
    float *part_o;      // partial states: [rows][head_dim], slots first, then planes
    float2 *part_ml;    // their m and l
    int64_t q_stride;
    float scale;
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8 as_bf16x8(uint4 w) { return __builtin_bit_cast(bf16x8, w); }

// Eight weights as the bf16 operand of the second product; l sums what the
// product takes, the rounded weights, so that they add up to one.
__device__ __forceinline__ bf16x8 weights(const float *e, float &l)
{
    const uint4 w = make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                               pack_bf16x2(e[6], e[7]));
    constexpr uint32_t ones = 0x3F803F80u;
    l = dot2(w.x, ones, l);
    l = dot2(w.y, ones, l);
    l = dot2(w.z, ones, l);
    l = dot2(w.w, ones, l);
    return as_bf16x8(w);
}

// Four e4m3 numbers as four bf16 (exact).
__device__ __forceinline__ u32x2 e4m3_to_bf16(uint32_t w)
{
    u32x2 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
    return r;
}
__device__ __forceinline__ uint4 e4m3x8_to_bf16(uint32_t a, uint32_t b)
{
    const u32x2 x = e4m3_to_bf16(a), y = e4m3_to_bf16(b);
    return make_uint4(x[0], x[1], y[0], y[1]);
}

// Row strides of bf16 tiles in LDS, in numbers: the padding shifts a row
// against the one before by 4 banks (K: 16 rows' 16-byte pieces of one column
// block), 16 banks (V of the tiled kernel: four rows' 64 bytes) or 8 banks (V
// of the streaming kernel: eight rows' 32 bytes), so that one access touches
// every bank equally often; a fixed stride keeps all addresses of a tile at
// one register plus constants.
template <int D>
struct Stride {
    static constexpr int k = D + 8, v = D + 32, v_stream = D + 16;
};

// Transposing LDS read: 16 lanes give the addresses of a 4-row, 16-column
// block (lane t: row t / 4, columns 4 (t % 4)..), lane t gets column t.
__device__ __forceinline__ u32x2 read_tr(const uint16_t *p)
{
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p));
}

// Keeps LDS accesses of one wave in program order for the compiler; the LDS
// itself serves a wave's accesses in order.
__device__ __forceinline__ void lds_order()
{
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// The wave's number in the workgroup, as a value the compiler knows to be the
// same in all of its lanes.
__device__ __forceinline__ int wave_of_thread() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

// The larger of lane l's and lane l ^ 32's value.
__device__ __forceinline__ float max_of_halves(float x)
{
    const uint32_t b = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Scores are masked and compared before they are scaled, which needs a factor
// above zero.  What else an 8-bit cache's scale gives goes into the row's q: the
// sign, or a zero, which leaves there what is not finite as a NaN.
template <typename Q>
__device__ __forceinline__ float positive_factor(float sc, Q &q)
{
    if (sc <= 0.0f) {
        const float f = sc < 0.0f ? -1.0f : 0.0f;
        for (auto &block : q)
            for (auto &k : block)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    k[i] = (__bf16)((float)k[i] * f);
        sc = sc < 0.0f ? -sc : 1.0f;
    }
    return sc;
}

// Waits for this wave's LDS accesses.
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Where a column of V holds a number that is not finite, a weight of zero does
// not keep it out of the rows that do not see its key.  In tiles that some of
// the rows see only in part such numbers are therefore taken out of V and added
// afterwards to the rows that do see them.  This takes them out of eight bf16
// numbers and returns where they were; what they were stays in their place: an
// infinity a zero of its sign, a NaN the least number (e4m3 has only NaN).
template <bool E4M3>
__device__ __forceinline__ uint32_t take_nonfinite(uint4 &w)
{
    uint32_t bits = 0;
    const auto look = [&](uint32_t x, int i) {
        bits |= (x & 0x7F80u) == 0x7F80u ? 1u << (2 * i) : 0u;
        bits |= (x & 0x7F800000u) == 0x7F800000u ? 2u << (2 * i) : 0u;
    };
    look(w.x, 0), look(w.y, 1), look(w.z, 2), look(w.w, 3);
    if (__builtin_expect(__any(bits != 0), 0)) {
        const auto take = [&](uint32_t &x) {
            if ((x & 0x7F80u) == 0x7F80u)
                x = E4M3 ? x & 0xFFFF0000u : (x & 0xFFFF8000u) | ((x & 0x7Fu) != 0);
            if ((x & 0x7F800000u) == 0x7F800000u)
                x = E4M3 ? x & 0xFFFFu : (x & 0x8000FFFFu) | ((x & 0x7F0000u) != 0) << 16;
        };
        take(w.x), take(w.y), take(w.z), take(w.w);
    }
    return bits;
}

// x with the number added that take_nonfinite left as p.
template <bool E4M3>
__device__ __forceinline__ float add_taken(float x, uint32_t p)
{
    return E4M3 || (p & 0x7FFFu) ? NAN : x + (p ? -INFINITY : INFINITY);
}

// The lowest n bits (none for n < 0, all from 64 on).
__device__ __forceinline__ uint64_t first_bits64(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Exclusive prefix sum over the workgroup's threads, and the total.
struct Scan {
    int64_t wave[kWaves];
};
__device__ __forceinline__ int64_t scan_block(int64_t v, Scan &sh, int64_t &total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t y = __shfl_up(x, o);
        x += lane >= o ? y : 0;
    }
    __syncthreads();
    if (lane == 63)
        sh.wave[w] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        before += i < w ? sh.wave[i] : 0;
        total += sh.wave[i];
    }
    return before + x - v;
}

// Sums of two values over the workgroup's threads.
__device__ __forceinline__ void sum_block(int64_t &x, int64_t &y, Scan &sx, Scan &sy)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        x += __shfl_xor(x, o), y += __shfl_xor(y, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        sx.wave[threadIdx.x >> 6] = x, sy.wave[threadIdx.x >> 6] = y;
    __syncthreads();
    x = y = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        x += sx.wave[i], y += sy.wave[i];
}

// a / b for a >= 0, b > 0: nearly always within 32 bits, where it is far cheaper
// (in the schedule's sums, once a thread, it costs more registers than it saves time:
// chunk of 1021 tokens beside 31 decodes 115 us with it there, 111 without).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Fills the group table.
__device__ __forceinline__ void fill_groups(const Sched &s, Groups &gr)
{
    static_assert(kThreads >= BD_MAX_GROUPS, "a thread per group");
    if ((int)threadIdx.x < s.p.b.n_groups)
        fill_group(s, gr, threadIdx.x);
    if (s.p.b.n_groups)
        __syncthreads();
}

// A list of segments whose sizes are laid end to end: thread i sums the
// sizes of segments [i * per, (i + 1) * per).
struct Located {
    int first;        // a segment at or before the one that holds the position
    int64_t base;     // where `first` begins
    Segment segment;  // segment `first`, as its thread read it
};
template <typename Read, typename Size>
struct Listing {
    int n, per;
    int64_t mine, before, total;
    Segment head;     // the thread's first segment
    __device__ __forceinline__ Listing(int n_, const Read &read, const Size &size, Scan &sh)
    {
        n = n_, per = (n + kThreads - 1) / kThreads;
        mine = 0;
        const int i0 = threadIdx.x * per;
        for (int i = i0; i < min(n, i0 + per); ++i) {
            const Segment g = read(i);
            if (i == i0)
                head = g;
            mine += size(g);
        }
        before = scan_block(mine, sh, total);
    }
    // position in [0, total), the same in all threads
    __device__ __forceinline__ Located locate(int64_t position, Located *sh) const
    {
        __syncthreads();
        if (before <= position && position < before + mine)
            *sh = {(int)threadIdx.x * per, before, head};
        __syncthreads();
        return *sh;
    }
};

// ------------------------------------------------------------ few rows: stream
//
// Decode: memory bound.  Each wave streams its own 32-key tiles (every fourth
// of the workgroup's) straight into registers, K as the fragments that the
// matrix instruction takes, V by whole rows and on through the wave's own
// piece of LDS; no barrier until the workgroup's run of one key head ends and
// the four waves' states are joined.  Eight waves a CU with 16 KB each on the
// way cover the memory latency (twelve with 8 KB of an 8-bit cache).  64 users
// with up to 16000 keys each, 64 query heads over 8 of 128: 340 us, 6.2 TB/s
// (V through the caches like K: 380); one user's 200003 keys 140 us, 5.9 TB/s
// (152); 96 users on an 8-bit cache 74 us, 6.0 TB/s (95); one user's 1531 keys
// 9 us: four memory latencies and a launch.
// Workgroups of it that fit a CU, by their registers.
constexpr int stream_per_cu(int d, bool e4m3, int nb) { return nb == 1 && (e4m3 || d == 64) ? 3 : 2; }

template <int D, int NB>
struct StreamLds {
    static constexpr int kJoin = kWaves * 16 * NB * (D + 4) * 4, kStage = kWaves * kStreamKeys * Stride<D>::v_stream * 2;
    __attribute__((aligned(16))) uint8_t tiles[kJoin > kStage ? kJoin : kStage];
    uint8_t bad[kWaves][kStreamKeys][D / 8];
    float2 wave_ml[kWaves][16 * NB];
    Scan scan;
    Located found;
    Groups groups;
};

template <int D, bool E4M3, int NB>
__device__ __forceinline__ void stream_body(const AttnArgs &a, StreamLds<D, NB> &sh, int block)
{
    constexpr int R = 16 * NB, KS = D / 32, DB = D / 16;
    constexpr int ES = E4M3 ? 1 : 2;                 // bytes of a cached number
    constexpr int NK = KS * ES / 2;                  // 16-byte loads of a lane for 16 keys
    constexpr int LPR = D * ES / 16;                 // lanes that load a row of V
    constexpr int NV = kStreamKeys * LPR / 64, RPI = 64 / LPR;
    constexpr int VS = Stride<D>::v_stream;
    constexpr int OROW = D + 4;                      // padded row of the join
    auto &bad = sh.bad;
    auto &wave_ml = sh.wave_ml;
    auto &groups = sh.groups;

    const Sched &s = a.s;
    const Paged &p = s.p;
    const int lane = threadIdx.x & 63, wave = wave_of_thread(), col = lane & 15, quad = lane >> 4;
    fill_groups(s, groups);
    const auto read = [&](int i) { return sequence(s, groups, i); };
    const auto size = [&](const Segment &g) { return stream_units(s, g); };
    const Listing list(p.b.n_seqs, read, size, sh.scan);
    const int64_t chunk = stream_chunk(s, list.total);
    int64_t at = block * chunk;
    const int64_t end = min(list.total, at + chunk);
    if (block == 0) {
        if (threadIdx.x == 0)
            a.cut[1] = chunk;
        int64_t b = list.before;
        for (int i = threadIdx.x * list.per; i < min(list.n, (int)(threadIdx.x + 1) * list.per); ++i) {
            a.cut[2 + i] = b;
            b += list.per > 1 ? size(read(i)) : 0;
        }
    }
    if (at >= end)
        return;
    const Located loc = list.locate(at, &sh.found);
    int seq = loc.first;
    int64_t base = loc.base;
    Segment g = loc.segment;
    uint16_t *vt = reinterpret_cast<uint16_t *>(sh.tiles) + wave * kStreamKeys * VS;
    float *oj = reinterpret_cast<float *>(sh.tiles);

    while (at < end) {
        for (int64_t units; base + (units = stream_units(s, g)) <= at;) {
            if (++seq >= p.b.n_seqs)
                return;      // only where the lengths changed under the call
            base += units;
            g = read(seq);
        }
        const int tiles = key_tiles(g, kStreamKeys), pre_tiles = (int)cdiv(g.pre, kStreamKeys);
        const int64_t row_tiles = stream_row_tiles(s, g), rows = rows_of(s, g);
        const int len = stream_run(g);
        const int64_t run = quotient(at - base, len);
        const int from = (int)((at - base) - run * len), to = (int)min((int64_t)len, from + (end - at));
        const int t0 = max(from - kRunCost, 0), t1 = to - kRunCost;
        at += to - from;
        if (t0 >= t1)
            continue;
        const int head = (int)quotient(run, row_tiles);
        const int row0 = (int)(run - head * row_tiles) * R;
        const int32_t *own_table = p.b.page_table + (int64_t)seq * p.b.max_pages;
        const int32_t *pre_table = g.pre ? p.b.prefix_table + (int64_t)g.group * p.b.max_prefix_pages : own_table;

        bf16x8 q[NB][KS];
        int seen[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int row = row0 + n * 16 + col, tok = row / s.group;
            seen[n] = row < rows ? own_seen(g, tok) : 0;
            const uint16_t *src = a.q + (g.tok0 + (int64_t)tok) * a.q_stride +
                                  (int64_t)(head * s.group + row - tok * s.group) * D;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                // the columns of a K fragment: those of the lane's 16-byte loads
                const int c = E4M3 ? (k >> 1) * 64 + quad * 16 + (k & 1) * 8 : k * 32 + quad * 8;
                q[n][k] = as_bf16x8(row < rows ? *reinterpret_cast<const uint4 *>(src + c) : make_uint4(0, 0, 0, 0));
            }
        }
        const int least = own_seen(g, row0 / s.group);   // own keys that the first row sees: the fewest

        f32x4 o[NB][DB];
        float m[NB], l[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            m[n] = -INFINITY, l[n] = 0.0f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
                o[n][d] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }
        float sc = a.scale * kLog2e * (E4M3 && a.k_scale ? a.k_scale[head] : 1.0f);

        // lane l: the cell of the tile's key l % 32
        const auto cells = [&](int t) {
            const bool own = t >= pre_tiles;
            const int j = (own ? t - pre_tiles : t) * kStreamKeys + (lane & 31);
            return j < (own ? g.own : g.pre) ? cell_of(p, own ? own_table : pre_table, head, j) : -1;
        };
        uint4 kr[2][NK], vr[NV];
        uint32_t v_held = 0;
        // a key without a cell reads cell 0: its score is masked, its value cleared
        const auto load = [&](int cell) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint8_t *src = a.k + (uint64_t)max(__shfl(cell, b * 16 + col), 0) * (D * ES) + quad * 16;
#pragma unroll
                for (int k = 0; k < NK; ++k)
                    kr[b][k] = *reinterpret_cast<const uint4 *>(src + k * 64);
            }
            v_held = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = __shfl(cell, i * RPI + lane / LPR);
                // whole lines, read once: past the caches (K, whose loads take half lines, through them)
                vr[i] = ld_stream16(a.v + (uint64_t)max(c, 0) * (D * ES) + lane % LPR * 16);
                v_held |= c >= 0 ? 1u << i : 0u;
            }
        };
        int t = t0 + wave, cell = -1, next = -1;
        if (t < t1) {
            cell = cells(t);
            load(cell);
        }
        if (t + kWaves < t1)
            next = cells(t + kWaves);
        if (E4M3)
            sc = positive_factor(sc, q);
        for (; t < t1; t += kWaves) {
            const uint32_t held = (uint32_t)__ballot(cell >= 0);
            const bool own = t >= pre_tiles;
            const int j0 = own ? (t - pre_tiles) * kStreamKeys : 0;
            const bool masked = held != 0xFFFFFFFFu || (own && j0 + kStreamKeys > least);
            uint32_t any_bad = 0;
            lds_order();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int r = i * RPI + lane / LPR, c = lane % LPR * (E4M3 ? 2 : 1);
                uint4 w[2] = {vr[i], vr[i]};
                if (E4M3)
                    w[0] = e4m3x8_to_bf16(vr[i].x, vr[i].y), w[1] = e4m3x8_to_bf16(vr[i].z, vr[i].w);
#pragma unroll
                for (int e = 0; e < (E4M3 ? 2 : 1); ++e) {
                    if (masked) {
                        if (!((v_held >> i) & 1u))
                            w[e] = make_uint4(0, 0, 0, 0);
                        const uint32_t bits = take_nonfinite<E4M3>(w[e]);
                        bad[wave][r][c + e] = (uint8_t)bits;
                        any_bad |= bits;
                    }
                    *reinterpret_cast<uint4 *>(vt + r * VS + (c + e) * 8) = w[e];
                }
            }
            f32x4 x[NB][2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    x[n][b] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint4 w = kr[b][E4M3 ? k >> 1 : k];
                    const bf16x8 kf = as_bf16x8(!E4M3 ? w : k & 1 ? e4m3x8_to_bf16(w.z, w.w) : e4m3x8_to_bf16(w.x, w.y));
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        x[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[n][k], x[n][b], 0, 0, 0);
                }
            }
            // the next tile is on its way while this one is weighed
            cell = next;
            if (t + kWaves < t1)
                load(cell);
            if (t + 2 * kWaves < t1)
                next = cells(t + 2 * kWaves);

            bf16x8 pf[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if (masked) {
                    const uint32_t ok = (held & (uint32_t)first_bits64(own ? seen[n] - j0 : INT_MAX)) >> quad * 4;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            x[n][b][r] = (ok >> (b * 16 + r)) & 1u ? x[n][b][r] : -INFINITY;
                }
                float mx = -INFINITY;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        mx = fmaxf(mx, x[n][b][r]);
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32)) * sc;
                const float mn = fmaxf(m[n], mx), mu = mn == -INFINITY ? 0.0f : mn;
                const float keep = exp2_(m[n] - mu);
                m[n] = mn;
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    e[i] = exp2_(fmaf(x[n][i >> 2][i & 3], sc, -mu));
                l[n] *= keep;
                pf[n] = weights(e, l[n]);
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[n][d] *= keep;
            }
            lds_order();
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                // keys 4 quad + 0..3 and 16 + 4 quad + 0..3 of column 16 d + col
                const uint16_t *src = vt + (quad * 4 + (col >> 2)) * VS + d * 16 + (col & 3) * 4;
                const u32x2 lo = read_tr(src), hi = read_tr(src + 16 * VS);
                const bf16x8 vf = as_bf16x8(make_uint4(lo[0], lo[1], hi[0], hi[1]));
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[n], o[n][d], 0, 0, 0);
            }
            if (masked && __builtin_expect(__any(any_bad != 0), 0)) {
#pragma unroll 1
                for (int key = 0; key < kStreamKeys; ++key)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const int bits = bad[wave][key][2 * d + (quad >> 1)] >> (quad & 1) * 4 & 15;
                        if (!bits)
                            continue;
                        const u32x2 was = *reinterpret_cast<const u32x2 *>(vt + key * VS + d * 16 + quad * 4);
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (((bits >> r) & 1) && (!own || key < seen[n] - j0))
                                    o[n][d][r] = add_taken<E4M3>(o[n][d][r], was[r >> 1] >> 16 * (r & 1) & 0xFFFFu);
                    }
            }
        }

        // join the four waves' states
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            l[n] += __shfl_xor(l[n], 16);
            l[n] += __shfl_xor(l[n], 32);
            if (quad == 0)
                wave_ml[wave][n * 16 + col] = make_float2(m[n], l[n]);
#pragma unroll
            for (int d = 0; d < DB; ++d)
                *reinterpret_cast<f32x4 *>(oj + (wave * R + n * 16 + col) * OROW + d * 16 + quad * 4) = o[n][d];
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles;
        const int64_t slot = 2 * (int64_t)block + (t0 == 0 ? 1 : 0);
        const float vs = E4M3 && a.v_scale ? a.v_scale[head] : 1.0f;
        for (int u = threadIdx.x; u < R * (D / 4); u += kThreads) {
            const int r = u / (D / 4), c = u % (D / 4) * 4, row = row0 + r;
            if (row >= rows)
                continue;
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                mm = fmaxf(mm, wave_ml[w][r].x);
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float2 ml = wave_ml[w][r];
                if (ml.x == -INFINITY && !(ml.y != ml.y))
                    continue;
                const float e = exp2_(ml.x - mm);
                ll = fmaf(ml.y, e, ll);
                acc += *reinterpret_cast<const f32x4 *>(oj + (w * R + r) * OROW + c) * e;
            }
            acc *= vs;
            const int tok = row / s.group;
            const int64_t cell_out = (g.tok0 + (int64_t)tok) * s.n_heads + head * s.group + row - tok * s.group;
            if (whole && !g.shared) {
                const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
                u32x2 w;
                w[0] = pack_bf16x2(acc[0] * inv, acc[1] * inv);
                w[1] = pack_bf16x2(acc[2] * inv, acc[3] * inv);
                *reinterpret_cast<u32x2 *>(a.out + cell_out * D + c) = w;
            } else {
                const int64_t pr = whole ? 2 * (int64_t)s.stream_wgs * R + cell_out : slot * R + r;
                *reinterpret_cast<f32x4 *>(a.part_o + pr * D + c) = acc;
                if (c == 0)
                    a.part_ml[pr] = make_float2(mm, ll);
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------- many rows: tiles
//
// Prompts and shared prefixes: matrix bound.  A workgroup holds 128 rows, 32
// a wave (256 and 64 at 64 columns), and walks 64-key tiles of K and V that all
// four waves read from LDS; a tile's loads are in registers one step ahead, and
// LDS holds two tiles, so a step has one barrier.  Prompts of up to 4097 tokens,
// 64 heads over 8 of 128: 424 us, 811 TFLOP/s of the causal work (a large bf16
// product reaches 1398 here).  A wave's step of 128 columns is 413 instructions,
// 32 of them matrix instructions of 32 cycles, and takes 5060 cycles beside the
// SIMD's other wave (4500 alone): 37% issuing, 38% ready but behind the other
// wave or the matrix unit, 25% waiting for loads, LDS or the barrier, with one
// tile on its way in one set of registers.  The matrix units are busy 40% of the
// cycles; leaving out all exponentials saves 5%, three quarters of the second
// product 10%, any one kind of LDS read 2-4%.  Measured and dropped: eight waves that share
// a tile, also half a step apart (430 us), 64 rows a wave at 128 columns, one
// wave a SIMD (640 us), K fragments read ahead over the barrier (435 us), steps
// of 32 keys (465 us), with them a third wave a SIMD (510 us, registers spilled).
// As built the kernels at 256 registers spill 4 of them at 128 columns in bf16, 2
// to 6 at 64 columns, and 45 to 70 scalars, once an item; no step touches scratch.
template <int D>
struct TiledLds {
    __attribute__((aligned(16))) uint16_t kt[2][kTileKeys * Stride<D>::k], vt[2][kTileKeys * Stride<D>::v];
    uint8_t key_held[2][kTileKeys], bad[2][kTileKeys][D / 8];
    int hole[2][kWaves], any_bad[2][kWaves], holes;
    Scan scan, scan2;
    Located found;
    Groups groups;
};

template <int D, bool E4M3>
__device__ __forceinline__ void tiled_body(const AttnArgs &a, TiledLds<D> &sh, int block, int blocks)
{
    constexpr int KS = D / 16, DB = D / 32;
    constexpr int ES = E4M3 ? 1 : 2;
    constexpr int NR = tile_rows(D) / (32 * kWaves);
    constexpr int NL = D * ES / 64;   // loads of a thread, K and V each: four threads a key, 64 bytes a load
    static_assert(kThreads == 4 * kTileKeys, "four threads a key");
    constexpr int KR = Stride<D>::k, VR = Stride<D>::v;
    auto &kt = sh.kt;
    auto &vt = sh.vt;
    auto &key_held = sh.key_held;
    auto &bad = sh.bad;
    auto &any_bad = sh.any_bad;
    auto &hole = sh.hole;
    auto &groups = sh.groups;

    const Sched &s = a.s;
    const Paged &p = s.p;
    const int lane = threadIdx.x & 63, wave = wave_of_thread(), col = lane & 31, half = lane >> 5;
    const int n_seg = p.b.n_seqs + p.b.n_groups;
    int64_t depth = INT_MAX;
    fill_groups(s, groups);
    if (s.splits > 1) {
        int64_t work = 0, items = 0;
        for (int i = threadIdx.x; i < n_seg; i += kThreads) {
            const Segment g = tiled_segment(s, groups, i);
            if (g.ntok) {
                work += tiled_work(s, g);
                items += p.n_kv * tiled_row_tiles(s, g);
            }
        }
        sum_block(work, items, sh.scan, sh.scan2);
        // lane k - 1 tries k
        float best = lane < s.splits && items > 0 ? tiled_time(items, work, lane + 1) : INFINITY;
        const float mine = best;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            best = fminf(best, __shfl_xor(best, o));
        depth = tiled_depth(items, work, __ffsll(__ballot(mine == best)));
    }
    if (block == 0 && threadIdx.x == 0)
        a.cut[0] = depth;
    const auto read = [&](int i) { return tiled_segment(s, groups, i); };
    const auto size = [&](const Segment &g) { return tiled_items(s, g, depth); };
    const Listing list(n_seg, read, size, sh.scan);

    // Tiles are numbered over all items of the workgroup.  A wave that stages
    // keys without a cell, or values that are not finite, leaves the tile's
    // number in its flag; nothing is written for the other tiles.  `holes` stays
    // set from the first tile with such keys on.
    if (threadIdx.x == 0)
        sh.holes = 0;
    if (threadIdx.x < 2 * kWaves)
        (&hole[0][0])[threadIdx.x] = (&any_bad[0][0])[threadIdx.x] = -1;
    int number = 0;

    for (int64_t item = block; item < list.total; item += blocks) {
        const Located loc = list.locate(item, &sh.found);
        int seg = loc.first;
        int64_t base = loc.base;
        Segment g = loc.segment;
        for (int64_t n; item >= base + (n = size(g));) {
            if (++seg >= n_seg)
                return;      // only where the lengths changed under the call
            base += n;
            g = read(seg);
        }
        // heads fastest, then splits, then row tiles from the last (the longest) to the first
        const int64_t idx = item - base;
        const int splits = tiled_splits(s, g, depth);
        const int64_t idx2 = quotient(idx, p.n_kv), idx3 = quotient(idx2, splits);
        const int head = (int)(idx - idx2 * p.n_kv), split = (int)(idx2 - idx3 * splits);
        const int64_t rows = rows_of(s, g);
        const int row0 = (int)(tiled_row_tiles(s, g) - 1 - idx3) * tile_rows(D);
        const int rows_here = (int)min((int64_t)tile_rows(D), rows - row0);
        const int pre_tiles = (int)cdiv(g.pre, kTileKeys);
        const bool is_prefix = seg >= p.b.n_seqs;
        // tiles up to the last row's own key; a split's share is that of the whole segment
        const int last_seen = is_prefix ? 0 : own_seen(g, (row0 + rows_here - 1) / s.group);
        const int per = (int)cdiv(key_tiles(g, kTileKeys), splits);
        const int t0 = split * per, t1 = min(t0 + per, pre_tiles + (int)cdiv(last_seen, kTileKeys));
        const int32_t *own_table = is_prefix ? nullptr : p.b.page_table + (int64_t)seg * p.b.max_pages;
        const int32_t *pre_table = g.pre ? p.b.prefix_table + (int64_t)g.group * p.b.max_prefix_pages : nullptr;

        // the wave's rows: NR blocks of 32, a lane's row in block n is rowi[n]
        int tok[NR], seen[NR];
        int64_t cell_out[NR];
        bf16x8 q[NR][KS];
        const int wave_row = row0 + wave * 32 * NR, wave_rows = min(rows_here - wave * 32 * NR, 32 * NR);   // may be negative
        const int least = own_seen(g, wave_row / s.group);               // own keys of the wave's first row: the fewest
        const int least_all = own_seen(g, row0 / s.group);
        const int most = wave_rows <= 0 ? 0 : own_seen(g, (wave_row + wave_rows - 1) / s.group);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int row = wave_row + n * 32 + col;
            const bool live = row < rows;
            tok[n] = live ? row / s.group : -1;
            const int h = live ? head * s.group + row - tok[n] * s.group : 0;
            seen[n] = live ? own_seen(g, tok[n]) : 0;
            cell_out[n] = (g.tok0 + (int64_t)tok[n]) * s.n_heads + h;
            const uint16_t *from = a.q + (g.tok0 + (int64_t)max(tok[n], 0)) * a.q_stride + (int64_t)h * D + half * 8;
#pragma unroll
            for (int k = 0; k < KS; ++k)
                q[n][k] = as_bf16x8(live ? *reinterpret_cast<const uint4 *>(from + k * 16) : make_uint4(0, 0, 0, 0));
        }
        f32x16 o[NR][DB];
        float m[NR], l[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            m[n] = -INFINITY, l[n] = 0.0f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    o[n][d][r] = 0.0f;
        }
        float sc = a.scale * kLog2e * (E4M3 && a.k_scale ? a.k_scale[head] : 1.0f);

        // One set of registers carries K of the next tile until the scores of
        // this one are done, then its V.  A key without a cell reads cell 0: its
        // score is masked, its value cleared.
        int page = 0, cell = -1;
        const uint8_t *src = nullptr;
        struct Loads {
            uint4 at[NL];
        } in;
        // Four threads a key, so a key's cell and address are formed once.  The
        // 16 keys of a wave are dealt so that 16 neighbouring threads, four keys,
        // write to different banks under both row strides.
        const int part = threadIdx.x & 3, k4 = (lane >> 2) & 3;
        const int ldr = wave * 16 + k4 * 4 + ((k4 + (lane >> 4)) & 3);
        const auto read_page = [&](int t) {
            const bool own = t >= pre_tiles;
            const int j = (own ? t - pre_tiles : t) * kTileKeys + ldr;
            page = (own ? own_table : pre_table)[min(j, (own ? g.own : g.pre) - 1) >> p.page_shift];
        };
        const auto load = [&](const uint8_t *from) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                in.at[i] = *reinterpret_cast<const uint4 *>(from + i * 64);
        };
        const auto load_k = [&](int t) {
            const bool own = t >= pre_tiles;
            const int j = (own ? t - pre_tiles : t) * kTileKeys + ldr;
            cell = j < (own ? g.own : g.pre) && (unsigned)page < (unsigned)p.n_pages
                       ? ((page * p.n_kv + head) << p.page_shift) + (j & ((1 << p.page_shift) - 1)) : -1;
            const uint64_t off = (uint64_t)max(cell, 0) * (D * ES) + part * 16;
            src = a.v + off;
            load(a.k + off);
        };
        // some row of the workgroup does not see all of tile t's keys that others see
        const auto partial = [&](int t) { return t >= pre_tiles && (t - pre_tiles + 1) * kTileKeys > least_all; };
        const int ldc = part * (E4M3 ? 2 : 1);                     // first of a load's 8-column pieces
        constexpr int PIECES = E4M3 ? 2 : 1, STEP = 4 * PIECES;
        const int num0 = number - t0;                              // tile t has number num0 + t
        const auto put = [&](uint16_t *tile, int stride) {
            uint4 *dst = reinterpret_cast<uint4 *>(tile + ldr * stride + ldc * 8);
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (E4M3) {
                    dst[i * STEP] = e4m3x8_to_bf16(in.at[i].x, in.at[i].y);
                    dst[i * STEP + 1] = e4m3x8_to_bf16(in.at[i].z, in.at[i].w);
                } else {
                    dst[i * STEP] = in.at[i];
                }
        };
        const auto stage_k = [&](int t) {
            put(kt[t & 1], KR);
            if (__any(cell < 0)) {
                key_held[t & 1][ldr] = cell >= 0;
                hole[t & 1][wave] = num0 + t;
                sh.holes = 1;
            }
        };
        const auto stage_v = [&](int t, auto plain) {
            const int buf = t & 1;
            if ((decltype(plain)::value || !partial(t)) && !__any(cell < 0)) {
                put(vt[buf], VR);
                return;
            }
            uint4 *dst = reinterpret_cast<uint4 *>(vt[buf] + ldr * VR + ldc * 8);
            uint32_t found_bad = 0;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                uint4 v[2] = {in.at[i], in.at[i]};
                if (E4M3)
                    v[0] = e4m3x8_to_bf16(in.at[i].x, in.at[i].y), v[1] = e4m3x8_to_bf16(in.at[i].z, in.at[i].w);
#pragma unroll
                for (int e = 0; e < PIECES; ++e) {
                    if (cell < 0)
                        v[e] = make_uint4(0, 0, 0, 0);
                    if (partial(t)) {
                        const uint32_t bits = take_nonfinite<E4M3>(v[e]);
                        bad[buf][ldr][ldc + i * STEP + e] = (uint8_t)bits;
                        found_bad |= bits;
                    }
                    dst[i * STEP + e] = v[e];
                }
            }
            if (__any(found_bad != 0))
                any_bad[buf][wave] = num0 + t;
        };
        // q has to be there before the loop: its wait inside would be one for all loads in flight
        wait_vmcnt<0>();
        if (E4M3)
            sc = positive_factor(sc, q);
        if (t0 < t1) {
            // past the end the last tile is read once more, and dropped
            read_page(t0);
            load_k(t0);
            stage_k(t0);
            load(src);
            read_page(min(t0 + 1, t1 - 1));
            stage_v(t0, std::false_type());
            load_k(min(t0 + 1, t1 - 1));
            read_page(min(t0 + 2, t1 - 1));
        }
        __syncthreads();
        // One step.  A wave issues an instruction every 8 cycles at best and two
        // waves share a SIMD, so what a step costs is its number of instructions;
        // PLAIN steps, whose keys (and the next tile's) are in range and seen by
        // all rows, leave out what only the others need, and reads are waited for
        // by the group.
        const auto step = [&](int t, auto plain) {
            constexpr bool PLAIN = decltype(plain)::value;
            const int buf = t & 1, now = num0 + t;
            const bool own = t >= pre_tiles;
            const int j0 = own ? (t - pre_tiles) * kTileKeys : 0;
            const bool active = wave_rows > 0 && (PLAIN || !(own && j0 >= most)), more = PLAIN || t + 1 < t1;
            f32x16 x[NR][2];
            uint64_t held = ~0ull;
            if (active) {
                // the scheduling fences keep the compiler from drawing a read to its use
                constexpr int kAhead = KS;
                const uint16_t *kl = kt[buf] + col * KR + half * 8;
                bf16x8 kf[kAhead];
                const auto read_k = [&](int i) {
                    kf[i % kAhead] = as_bf16x8(*reinterpret_cast<const uint4 *>(kl + (i & 1) * 32 * KR + (i >> 1) * 16));
                };
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    read_k(i);
                const int holes = sh.holes;
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            x[n][b][r] = 0.0f;
                __builtin_amdgcn_s_setprio(1);
                wait_lgkm0();
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 2 * KS; ++i) {
                    if (i == kAhead)
                        wait_lgkm0();
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        x[n][i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i % kAhead], q[n][i >> 1], x[n][i & 1],
                                                                              0, 0, 0);
                    if (i + kAhead < 2 * KS)
                        read_k(i + kAhead);
                    __builtin_amdgcn_sched_barrier(0);
                }
                __builtin_amdgcn_s_setprio(0);
                if (__builtin_amdgcn_readfirstlane(holes)) {
                    const int4 flags = *reinterpret_cast<const int4 *>(hole[buf]);
                    held = __ballot(key_held[buf][lane] != 0) | (flags.x == now ? 0 : 0xFFFFull) |
                           (flags.y == now ? 0 : 0xFFFFull << 16) | (flags.z == now ? 0 : 0xFFFFull << 32) |
                           (flags.w == now ? 0 : 0xFFFFull << 48);
                }
            }
            if (more) {
                wait_vmcnt<1>();          // K of the next tile; the page number after it may still be on its way
                stage_k(t + 1);
                load(src);
            }
            if (active) {
                // keys 16 i + 4 half + 0..3 and + 8 of column 32 d + col
                const uint16_t *vl = vt[buf] + (half * 4 + ((lane & 15) >> 2)) * VR + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
                bf16x8 vf[2][DB];
                const auto read_v = [&](int i, int d) {
                    const uint16_t *from = vl + i * 16 * VR + d * 32;
                    const u32x2 lo = read_tr(from), hi = read_tr(from + 8 * VR);
                    vf[i & 1][d] = as_bf16x8(make_uint4(lo[0], lo[1], hi[0], hi[1]));
                };
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    read_v(0, d);
                __builtin_amdgcn_sched_barrier(0);
                if (held != ~0ull || (!PLAIN && own && j0 + kTileKeys > least)) {
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const uint64_t ok = (held & first_bits64(own ? seen[n] - j0 : INT_MAX)) >> half * 4;
                        const uint32_t word[2] = {(uint32_t)ok, (uint32_t)(ok >> 32)};
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                x[n][b][r] = (word[b] >> ((r >> 2) * 8 + (r & 3))) & 1u ? x[n][b][r] : -INFINITY;
                    }
                }
                float mx[NR], mu[NR];
                bool grown = false;
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    mx[n] = -INFINITY;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            mx[n] = fmaxf(mx[n], x[n][b][r]);
                    mx[n] = max_of_halves(mx[n]) * sc;
                    grown |= mx[n] > m[n] + 8.0f;
                }
                // the maximum follows only where it grew by more than 2^8: weights
                // up to 2^8 are as exact, and most tiles need no rescaling
                if (__any(grown)) {
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        // row by row, so that no row's bits depend on another's scores
                        const bool follows = mx[n] > m[n] + 8.0f;
                        const float keep = follows ? exp2_(m[n] - mx[n]) : 1.0f;
                        m[n] = follows ? mx[n] : m[n];
                        l[n] *= keep;
#pragma unroll
                        for (int d = 0; d < DB; ++d)
                            o[n][d] *= keep;
                    }
                }
                float e[NR][8];
                bf16x8 pf[2][NR];
                const auto weigh = [&](int i, int n, int r) {
                    e[n][r] = exp2_(fmaf(x[n][i >> 1][(i & 1) * 8 + r], sc, -mu[n]));
                };
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    mu[n] = m[n] == -INFINITY ? 0.0f : m[n];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        weigh(0, n, r);
                    pf[0][n] = weights(e[n], l[n]);
                }
                // the weights of the next 16 keys are formed, and their values read,
                // between the matrix instructions of these
                constexpr int kSlots = NR * DB, kPer = 8 * NR / kSlots;
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    wait_lgkm0();
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int c = 0; c < kSlots; ++c) {
                        const int d = c / NR, n = c % NR;
                        o[n][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[i & 1][d], pf[i & 1][n], o[n][d], 0, 0, 0);
                        if (i < 3) {
                            if (n == 0)
                                read_v(i + 1, d);
#pragma unroll
                            for (int w = c * kPer; w < (c + 1) * kPer; ++w)
                                weigh(i + 1, w >> 3, w & 7);
                            if ((c + 1) * kPer % 8 == 0)
                                pf[(i + 1) & 1][(c + 1) * kPer / 8 - 1] =
                                    weights(e[(c + 1) * kPer / 8 - 1], l[(c + 1) * kPer / 8 - 1]);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
                __builtin_amdgcn_s_setprio(0);
                bool some = false;
                if (!PLAIN && partial(t))
#pragma unroll
                    for (int w = 0; w < kWaves; ++w)
                        some |= any_bad[buf][w] == now;
                if (__builtin_expect(some, 0)) {
#pragma unroll 1
                    for (int key = 0; key < kTileKeys; ++key)
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            const int bits = any_bad[buf][key >> 4] == now ? bad[buf][key][c] >> half * 4 & 15 : 0;
                            if (!bits)
                                continue;
                            const u32x2 was = *reinterpret_cast<const u32x2 *>(vt[buf] + key * VR + c * 8 + half * 4);
#pragma unroll
                            for (int n = 0; n < NR; ++n)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    if (((bits >> r) & 1) && key < seen[n] - j0)
                                        o[n][c >> 2][(c & 3) * 4 + r] = add_taken<E4M3>(
                                            o[n][c >> 2][(c & 3) * 4 + r], was[r >> 1] >> 16 * (r & 1) & 0xFFFFu);
                        }
                }
            }
            if (more) {
                wait_vmcnt<0>();
                stage_v(t + 1, plain);
                load_k(PLAIN ? t + 2 : min(t + 2, t1 - 1));
                read_page(min(t + 3, t1 - 1));
            }
            __syncthreads();
        };
        // plain tiles end with the last whole one that all rows see, and the last
        // of the prefix is whole or not
        const int whole_pre = g.pre / kTileKeys, whole_own = min(g.own, least_all) / kTileKeys;
        const int plain_end = min(t1, pre_tiles > whole_pre && t0 < pre_tiles ? whole_pre : pre_tiles + whole_own) - 1;
        int t = t0;
        for (; t < plain_end - 1; ++t)
            step(t, std::true_type());
        for (; t < t1; ++t)
            step(t, std::false_type());
        number += max(t1 - t0, 0);

        const float vs = E4M3 && a.v_scale ? a.v_scale[head] : 1.0f;
        const bool whole = splits == 1 && !g.shared;
        const int64_t plane = is_prefix ? s.splits + split : split;
        const int64_t plane_row = 2 * (int64_t)s.stream_wgs * s.stream_rows + plane * s.p.b.n_tokens * s.n_heads;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            l[n] += __shfl_xor(l[n], 32);
            if (tok[n] < 0)
                continue;
            const float f = whole ? (l[n] == 0.0f ? 0.0f : vs / l[n]) : vs;
            const int64_t pr = plane_row + cell_out[n];
            if (!whole && half == 0)
                a.part_ml[pr] = make_float2(m[n], l[n]);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int c = d * 32 + r * 8 + half * 4;
                    const f32x4 w = {o[n][d][4 * r] * f, o[n][d][4 * r + 1] * f, o[n][d][4 * r + 2] * f,
                                     o[n][d][4 * r + 3] * f};
                    if (whole) {
                        u32x2 b;
                        b[0] = pack_bf16x2(w[0], w[1]);
                        b[1] = pack_bf16x2(w[2], w[3]);
                        *reinterpret_cast<u32x2 *>(a.out + cell_out[n] * D + c) = b;
                    } else {
                        *reinterpret_cast<f32x4 *>(a.part_o + pr * D + c) = w;
                    }
                }
        }
    }
}

// ---------------------------------------------------------------------- kernels

template <int D, bool E4M3, int NB>
__global__ __launch_bounds__(kThreads, stream_per_cu(D, E4M3, NB)) void attention_stream(AttnArgs a)
{
    __shared__ StreamLds<D, NB> sh;
    stream_body<D, E4M3, NB>(a, sh, blockIdx.x);
}

// Both at once where a call may have work for both: the streaming workgroups
// come first, one for each CU, and the tiled ones fill the other half, so that
// the one's loads run under the other's matrix instructions (128 users behind
// three prefixes: 74 us in two launches, 67 in one).
template <int D, bool E4M3, int NB>
__global__ __launch_bounds__(kThreads, 2) void attention_mixed(AttnArgs a)
{
    __shared__ union {
        StreamLds<D, NB> stream;
        TiledLds<D> tiled;
    } sh;
    const int block = blockIdx.x, streaming = a.s.stream_wgs;
    if (block < streaming)
        stream_body<D, E4M3, NB>(a, sh.stream, block);
    else
        tiled_body<D, E4M3>(a, sh.tiled, block - streaming, gridDim.x - streaming);
}

// ------------------------------------------------------------------------ join
//
// Joins the partial states of a token's heads and writes the zero rows of
// tokens that see nothing; finished rows are left alone.  Latency bound: 16
// lanes take a head, so a wave has four heads' states on the way, and where
// BY_PARTS (few tokens, perhaps many states a head) the four waves share the
// states of the same four heads: 6 us for one token's 64 heads of 13 states
// each, 11 us of 64 (one wave a head and state after state: 10 and 35 us).
template <int D, bool BY_PARTS>
__global__ __launch_bounds__(kThreads) void attention_join(AttnArgs a, int tokens)
{
    constexpr int N = D / 64;      // 16-byte pieces of a lane, 64 columns apart
    __shared__ Groups groups;
    __shared__ float2 wave_ml[kWaves][4];
    __shared__ f32x4 wave_o[kWaves][4][D / 4];
    const Sched &s = a.s;
    const Paged &p = s.p;
    const int lane = threadIdx.x & 63, wave = wave_of_thread(), sub = lane & 15, grp = lane >> 4;
    const int64_t slots = 2 * (int64_t)s.stream_wgs * s.stream_rows, plane = p.b.n_tokens * s.n_heads;

    const int64_t tok0 = (int64_t)blockIdx.x * tokens;
    const int64_t depth = s.tiled ? a.cut[0] : 1, chunk = a.cut[1];
    fill_groups(s, groups);
    int seq = seq_of(p, tok0);
    for (int64_t tok = tok0; tok < min(tok0 + tokens, p.b.n_tokens); ++tok) {
    if (seq < 0 || tok >= seq_begin(p, seq + 1))
        seq = tok == tok0 ? seq : seq_of(p, tok);
    // parts of own keys: planes [0, own_parts), or the slots of workgroups first_wg .. where `slotted`
    int own_parts = 0, prefix_parts = 0, tiles = 0;
    bool by_stream = false;
    Segment g;
    int64_t units0 = 0;
    if (seq >= 0) {
        g = sequence(s, groups, seq);
        by_stream = streamed(s, g);
        units0 = a.cut[2 + seq];
        tiles = key_tiles(g, kStreamKeys);
        if (!by_stream) {
            own_parts = tiled_splits(s, g, depth);
            if (own_parts == 1 && !g.shared) {
                // finished, and so are the sequence's other tokens
                tok = (int64_t)g.tok0 + g.ntok - 1;
                continue;
            }
        }
        if (g.shared)
            prefix_parts = tiled_splits(s, prefix(s, groups, g.group), depth);
    }
    constexpr int kHeads = BY_PARTS ? 4 : 4 * kWaves;      // heads of a workgroup at a time
    for (int h0 = blockIdx.y * kHeads; h0 < s.n_heads; h0 += gridDim.y * kHeads) {
        const int h = h0 + (BY_PARTS ? 0 : wave * 4) + grp;
        bool mine = h < s.n_heads;
        const int64_t cell_out = tok * s.n_heads + h;
        int64_t first_wg = 0;
        int parts = own_parts, row_in = 0;
        bool slotted = false;
        if (by_stream && tiles && mine) {
            const int head = h / s.group, row = (int)(tok - g.tok0) * s.group + h - head * s.group;
            const int64_t u0 = units0 + kRunCost +
                               (head * stream_row_tiles(s, g) + row / s.stream_rows) * stream_run(g);
            first_wg = quotient(u0, chunk);
            parts = (int)(quotient(u0 + tiles - 1, chunk) - first_wg) + 1;
            slotted = parts > 1;
            row_in = row % s.stream_rows;
            mine = slotted || g.shared;
        }
        const int total = mine ? parts + prefix_parts : 0;
        int most = total;
        most = max(most, __shfl_xor(most, 16));
        most = max(most, __shfl_xor(most, 32));
        float m = -INFINITY, l = 0.0f;
        f32x4 o[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        // lane `sub` holds a part's m and l, then the 16 lanes add the parts' values
        for (int b = BY_PARTS ? wave * 16 : 0; b < most; b += BY_PARTS ? 16 * kWaves : 16) {
            const int i = b + sub;
            int64_t pr = 0;
            float2 ml = make_float2(-INFINITY, 0.0f);
            if (i < total) {
                if (i >= parts)
                    pr = slots + (s.splits + i - parts) * plane + cell_out;
                else if (slotted)
                    pr = (2 * (first_wg + i) + (i == 0 ? 1 : 0)) * s.stream_rows + row_in;
                else
                    pr = slots + i * plane + cell_out;
                ml = a.part_ml[pr];
            }
            float mx = ml.x;
#pragma unroll
            for (int w = 8; w > 0; w >>= 1)
                mx = fmaxf(mx, __shfl_xor(mx, w));
            const float mn = fmaxf(m, mx);
            // a part without keys has m = -inf and l = 0 (NaN where its scores were)
            const bool none = ml.x == -INFINITY && !(ml.y != ml.y);
            const float e = none ? 0.0f : exp2_(ml.x - mn), keep = m == -INFINITY ? 0.0f : exp2_(m - mn);
            float sum = none ? 0.0f : e * ml.y;
#pragma unroll
            for (int w = 8; w > 0; w >>= 1)
                sum += __shfl_xor(sum, w);
            l = l * keep + sum;
            m = mn;
#pragma unroll
            for (int c = 0; c < N; ++c)
                o[c] *= keep;
            for (int j0 = 0; j0 < min(16, most - b); j0 += 4)
#pragma unroll
                for (int j4 = 0; j4 < 4; ++j4) {
                    const int from = (lane & 48) + j0 + j4;
                    const float ej = __shfl(e, from);
                    const int64_t row = __shfl(pr, from);     // row 0 where there is no such part
                    const bool skip = __shfl((int)none, from);
#pragma unroll
                    for (int c = 0; c < N; ++c) {
                        const f32x4 v = *reinterpret_cast<const f32x4 *>(a.part_o + row * D + c * 64 + sub * 4);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            o[c][r] += skip ? 0.0f : ej * v[r];
                    }
                }
        }
        if (BY_PARTS) {
            if (sub == 0)
                wave_ml[wave][grp] = make_float2(m, l);
#pragma unroll
            for (int c = 0; c < N; ++c)
                wave_o[wave][grp][c * 16 + sub] = o[c];
            __syncthreads();
            float mm = -INFINITY;
            l = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                mm = fmaxf(mm, wave_ml[w][grp].x);
#pragma unroll
            for (int c = 0; c < N; ++c)
                o[c] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float2 ml = wave_ml[w][grp];
                if (ml.x == -INFINITY && !(ml.y != ml.y))
                    continue;
                const float e = exp2_(ml.x - mm);
                l += e * ml.y;
#pragma unroll
                for (int c = 0; c < N; ++c)
                    o[c] += wave_o[w][grp][c * 16 + sub] * e;
            }
            __syncthreads();
        }
        if (mine && (!BY_PARTS || wave == 0)) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int c = 0; c < N; ++c) {
                u32x2 w;
                w[0] = pack_bf16x2(o[c][0] * inv, o[c][1] * inv);
                w[1] = pack_bf16x2(o[c][2] * inv, o[c][3] * inv);
                *reinterpret_cast<u32x2 *>(a.out + cell_out * D + c * 64 + sub * 4) = w;
            }
        }
    }
    }
}

// ------------------------------------------------------------------------ host

// Workgroups of a launch, so that their threads stay below 2^32; more items go round.
constexpr int64_t kMaxItems = 1 << 23;

struct Plan {
    Sched s;
    int64_t grid, rows;     // workgroups, rows of partial states
};

size_t cut_bytes(const bd_batch &b) { return (size_t)(2 + b.n_seqs + 1) / 2 * 16; }

Plan make_plan(int32_t n_heads, const bd_kv_cache &c, const bd_batch &b)
{
    Plan pl;
    Sched &s = pl.s;
    s.p = {b, c.n_pages, c.n_kv_heads, __builtin_ctz((unsigned)c.page_size)};
    s.n_heads = n_heads, s.group = n_heads / c.n_kv_heads;
    const int64_t T = b.n_tokens;
    // 32 rows a streaming tile; 16 where the hint says that no sequence has more
    const int64_t most = b.max_new > 0 ? (int64_t)b.max_new * s.group : T > b.n_seqs ? INT_MAX : s.group;
    s.tiled = b.n_groups > 0 || most > 32;
    s.stream_rows = most <= 16 ? 16 : 32;
    s.few = s.tiled ? 32 : INT_MAX;
    s.stream_wgs = 256 * (s.tiled ? 1 : stream_per_cu(c.head_dim, c.dtype == BD_KV_E4M3, s.stream_rows / 16));
    s.tile_rows = tile_rows(c.head_dim);
    // enough splits that row tiles x key heads x splits fill the chip twice
    const int64_t tiles = cdiv(T * s.group, s.tile_rows) * c.n_kv_heads;
    const int64_t want = cdiv(2 * kTiledSlots, tiles);
    s.splits = s.tiled ? (int32_t)(want < 1 ? 1 : want > 64 ? 64 : want) : 1;
    const int64_t planes = b.n_groups > 0 ? 2 * s.splits : s.splits > 1 ? s.splits : 0;
    pl.rows = 2 * (int64_t)s.stream_wgs * s.stream_rows + planes * T * n_heads;
    // a workgroup per item; where items are split they are few, and the bound is loose
    const int64_t full = T * s.group / s.tile_rows;
    const int64_t row_tiles = full + (b.n_seqs < T ? b.n_seqs : T) + (b.n_groups > 0 ? full + b.n_groups : 0);
    const int64_t items = row_tiles * c.n_kv_heads * s.splits, cap = s.splits > 1 ? 2 * kTiledSlots : kMaxItems;
    const int64_t tiled_wgs = items < s.stream_wgs ? s.stream_wgs : items < cap ? items : cap;
    pl.grid = s.stream_wgs + (s.tiled ? tiled_wgs : 0);
    return pl;
}

template <int D, bool E4M3>
void start(const AttnArgs &a, const Plan &pl, hipStream_t st)
{
    const Sched &s = a.s;
    const dim3 grid((unsigned)pl.grid);
    if (s.tiled && s.stream_rows == 16)
        attention_mixed<D, E4M3, 1><<<grid, kThreads, 0, st>>>(a);
    else if (s.tiled)
        attention_mixed<D, E4M3, 2><<<grid, kThreads, 0, st>>>(a);
    else if (s.stream_rows == 16)
        attention_stream<D, E4M3, 1><<<grid, kThreads, 0, st>>>(a);
    else
        attention_stream<D, E4M3, 2><<<grid, kThreads, 0, st>>>(a);
    // a workgroup for every four heads where tokens are few, for sixteen, for a
    // token (1052 tokens of 40 heads: 116 us with it, 120 by sixteen), for 16
    // tokens where most are finished ones of prompts
    const unsigned T = (unsigned)s.p.b.n_tokens, heads = (unsigned)s.n_heads;
    if (T <= 64)
        attention_join<D, true><<<dim3(T, (heads + 3) / 4), kThreads, 0, st>>>(a, 1);
    else if (T <= 512)
        attention_join<D, false><<<dim3(T, (heads + 15) / 16), kThreads, 0, st>>>(a, 1);
    else if (T <= 2048)
        attention_join<D, false><<<dim3(T), kThreads, 0, st>>>(a, 1);
    else {
        const unsigned each = T <= 16 * kTokensAcross ? 16 : (unsigned)cdiv(T, kTokensAcross);
        attention_join<D, false><<<dim3((unsigned)cdiv(T, each)), kThreads, 0, st>>>(a, (int)each);
    }
}

}  // namespace

size_t attention_workspace_bytes(int32_t n_heads, const bd_kv_cache &c, const bd_batch &b)
{
    if (b.n_tokens == 0)
        return 0;
    return cut_bytes(b) + (size_t)make_plan(n_heads, c, b).rows * (c.head_dim * 4 + 8);
}

hipError_t launch_attention(const uint16_t *q, int64_t q_stride, int32_t n_heads, float scale, const bd_kv_cache &c,
                            const bd_batch &b, uint16_t *out, void *workspace, hipStream_t st)
{
    const Plan pl = make_plan(n_heads, c, b);
    AttnArgs a;
    a.s = pl.s;
    a.q = q, a.q_stride = q_stride, a.out = out, a.scale = scale;
    a.k = static_cast<const uint8_t *>(c.k), a.v = static_cast<const uint8_t *>(c.v);
    a.k_scale = c.k_scale, a.v_scale = c.v_scale;
    a.cut = static_cast<int64_t *>(workspace);
    a.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + cut_bytes(b));
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + pl.rows * c.head_dim);
    const bool e4m3 = c.dtype == BD_KV_E4M3;
    if (c.head_dim == 64) {
        if (e4m3)
            start<64, true>(a, pl, st);
        else
            start<64, false>(a, pl, st);
    } else {
        if (e4m3)
            start<128, true>(a, pl, st);
        else
            start<128, false>(a, pl, st);
    }
    return hipGetLastError();
}

}  // namespace bd
