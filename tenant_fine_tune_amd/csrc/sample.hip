// One token from each row of logits (bitdelta_sample).
//
// In the order of the logits, largest first, every limit keeps a beginning of
// the row, and the token drawn is where the running sum of weights passes a
// number.  So no row is sorted: a histogram over logits finds the few tokens
// next to each border, and only those are put in order.
//
//   sample_bins  a part of a row is read once and held in registers: its largest
//                logit, then for each of 2048 bins the tokens in it and the sum of
//                their weights.
//   sample_draw  one workgroup a row adds the parts' bins up.  The sums in front of
//                the bins tell which bins can hold a border (top-k, top-p, min-p, the
//                draw); the row is read a second time, from the caches, for the
//                tokens in those, and every border is found among them.  Where they
//                are too many (nearly flat rows), border by border through smaller bins.
//
// Bins are d = 2^e wide, T / 64 < d <= T / 32, at multiples of d, so the parts' bins
// are the same ones; 2048 of them reach exp(-32) below the part's largest logit, and
// what lies deeper has no weight.  In a bin with lower edge L the weight relative to
// it, exp((l - L) / T), exceeds one by exp(1/32) - 1 at most; that excess, held in units of
// 2^-36, and the count share a 64-bit number, so that one LDS addition serves both,
// and all sums are of whole numbers: exact, in any order, cut in any way.
//
// sample_bins is bound by its vector instructions and LDS additions, one of 64 bits a
// logit: 512 rows of 131071 bf16 logits 51 us (2.6 TB/s), one of 32000 4.2.  sample_draw
// is bound by its stages, each waiting for the one before: one row 14 us, of which the
// row's reading takes 2; 512 rows 52 to 57, of which 15 are the reading from the caches.
#include "bd_device.h"
#include "sample_launch.h"
#include "sample_scale.h"

namespace bd {
namespace {

constexpr int kBinThreads = 1024;            // of sample_bins
constexpr uint32_t kWithoutExponents = 0x9DA1u;   // inverse of 1 + 0x433 * 2^5 of 2^17
constexpr int kFew = 128;

typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight logits as loaded; the ones that do not exist are -inf.
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
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (2 * i < n ? p[2 * i] : 0xFF80u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] : 0xFF80u) << 16;
    }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? hi_f32(w[i >> 1]) : lo_f32(w[i >> 1]); }
};

template <>
struct Eight<float> {
    u32x4 a, b;
    __device__ __forceinline__ void load(const float *p, int n)
    {
        if (n == 8) {
            a = *reinterpret_cast<const u32x4a4 *>(p);
            b = *reinterpret_cast<const u32x4a4 *>(p + 4);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            (i < 4 ? a : b)[i & 3] = i < n ? __float_as_uint(p[i]) : 0xFF800000u;
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i < 4 ? a[i] : b[i - 4]); }
};

__device__ __forceinline__ float one_of(const uint16_t *p, int i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ float one_of(const float *p, int i) { return p[i]; }

__device__ __forceinline__ bool greedy(float t) { return !(t > 0.0f); }

// What sample_bins leaves of a part: the largest logit and, for rows that take
// it, the first token that has it; then kBins packed bins.
struct Part {
    float top;
    int32_t first;
    uint64_t pad;
    uint64_t bins[kBins];
};

// What lane's neighbour by a fixed move holds, `none` where there is no such lane
// or the move does not reach its row of 16.
constexpr int kUp1 = 0x111, kUp2 = 0x112, kUp4 = 0x114, kUp8 = 0x118;    // within a row
constexpr int kRow = 0x142, kRows = 0x143;       // from the last lane of the row, of the two rows, before
constexpr int kWave1 = 0x138;                    // one lane up, over the rows
template <int MOVE, int ROWS = 15>
__device__ __forceinline__ uint32_t moved(uint32_t v, uint32_t none)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, MOVE, ROWS, 15, false);
}
template <int MOVE, int ROWS = 15>
__device__ __forceinline__ unsigned long long moved(unsigned long long v, unsigned long long none)
{
    return (unsigned long long)moved<MOVE, ROWS>((uint32_t)(v >> 32), (uint32_t)(none >> 32)) << 32 |
           moved<MOVE, ROWS>((uint32_t)v, (uint32_t)none);
}
template <int MOVE, int ROWS = 15>
__device__ __forceinline__ double moved(double v, double none)
{
    return __longlong_as_double((long long)moved<MOVE, ROWS>((unsigned long long)__double_as_longlong(v),
                                                             (unsigned long long)__double_as_longlong(none)));
}

__device__ __forceinline__ float wave_max(float v)
{
    auto with = [&](uint32_t other) { v = fmaxf(v, __uint_as_float(other)); };
    with(moved<kUp1>(__float_as_uint(v), __float_as_uint(v)));
    with(moved<kUp2>(__float_as_uint(v), __float_as_uint(v)));
    with(moved<kUp4>(__float_as_uint(v), __float_as_uint(v)));
    with(moved<kUp8>(__float_as_uint(v), __float_as_uint(v)));
    with(moved<kRow, 10>(__float_as_uint(v), __float_as_uint(v)));
    with(moved<kRows, 12>(__float_as_uint(v), __float_as_uint(v)));
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// G groups of eight logits a thread.
template <int G, typename T>
__global__ __launch_bounds__(kBinThreads)
void sample_bins(SampleArgs a, Part *__restrict__ parts, int32_t splits)
{
    __shared__ uint64_t bins[kBins];
    __shared__ float tops[kBinThreads / 64];
    __shared__ int32_t first;
    const int64_t row = blockIdx.x / (unsigned)splits;
    const int split = blockIdx.x % (unsigned)splits;
    const T *p = static_cast<const T *>(a.logits) + row * a.stride;
    const int at0 = split * (G * 8 * kBinThreads) + threadIdx.x * 8;
    Eight<T> l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int at = at0 + g * 8 * kBinThreads;
        l[g].load(p + at, min(max(a.vocab - at, 0), 8));
    }
    const float t = a.temperature ? a.temperature[row] : a.temperature_all;
    for (int i = threadIdx.x; i < kBins; i += kBinThreads)
        bins[i] = 0;
    if (threadIdx.x == 0)
        first = 0x7FFFFFFF;
    float top = -INFINITY;       // a maximum passes NaN over
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = fmaxf(top, l[g].get(i));
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0)
        tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = wave_max(tops[threadIdx.x & (kBinThreads / 64 - 1)]);

    Part &out = parts[blockIdx.x];
    if (threadIdx.x == 0)
        out.top = top;
    if (greedy(t)) {
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int g = G - 1; g >= 0; --g)
#pragma unroll
            for (int i = 7; i >= 0; --i)
                if (l[g].get(i) == top)
                    at = at0 + g * 8 * kBinThreads + i;
        if (at != 0x7FFFFFFF)
            atomicMin(&first, at);
        __syncthreads();
        if (threadIdx.x == 0)
            out.first = first;
        return;
    }
    Scale s;
    s.set(t, top);
    if (s.alone) {
        int n = 0;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                n += l[g].get(i) == top;
        if (n)
            atomicAdd((unsigned long long *)&bins[0], (unsigned long long)n << kCountShift);
    } else {
        const float first_byte = 8.0f * s.top_bin;
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = ldexpf(l[g].get(i), s.shift), at = fmaf(floorf(a), -8.0f, first_byte);
                if (at < 8.0f * kBins)
                    atomicAdd((unsigned long long *)((uint8_t *)bins + (int)at), (unsigned long long)s.raw_excess(a));
            }
            __builtin_amdgcn_sched_barrier(0);      // one group's temporaries at a time
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kBinThreads) {
        // n exponents, 0x433 from bit 52 on, are in the sum too: the bits from the
        // count's on are n (1 + 0x433 * 2^5) of 2^17, which an odd factor takes back
        const uint64_t v = bins[i];
        const uint32_t n = s.alone ? (uint32_t)(v >> kCountShift) : (uint32_t)(v >> kCountShift) * kWithoutExponents & 0x1FFFFu;
        out.bins[i] = (uint64_t)n << kCountShift | (v & kExcess);
    }
}

// Sum of v over the wave's lanes up to this one.
template <typename V>
__device__ __forceinline__ V wave_scan(V v)
{
    v += moved<kUp1>(v, V(0));
    v += moved<kUp2>(v, V(0));
    v += moved<kUp4>(v, V(0));
    v += moved<kUp8>(v, V(0));
    v += moved<kRow, 10>(v, V(0));
    v += moved<kRows, 12>(v, V(0));
    return v;
}

// Number i of a thread's N stands at place i * TH + its own: their sums over the places in
// front, `total` over all of them.
template <int TH, int N, typename V>
__device__ __forceinline__ void scan(const V (&v)[N], V *part, V (&before)[N], V &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    V s[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        s[i] = wave_scan(v[i]);
    __syncthreads();          // part may still be read from the scan before
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane == 63)
            part[i * (TH / 64) + wave] = s[i];
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        before[i] = 0;
#pragma unroll
    for (int w = 0; w < N * (TH / 64); ++w) {
        const V x = part[w];
#pragma unroll
        for (int i = 0; i < N; ++i)
            before[i] += w < i * (TH / 64) + wave ? x : V(0);
        total += x;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        before[i] += moved<kWave1>(s[i], V(0));
}
template <int TH, typename V>
__device__ __forceinline__ V scan(V v, V *part, V &total)
{
    const V mine[1] = {v};
    V before[1];
    scan<TH>(mine, part, before, total);
    return before[0];
}

// The first of n <= 4096 places that is right, n - 1 if no other is: `right` turns
// from false to true once.  All lanes of a wave look at places 64 apart, then at those between.
template <typename F>
__device__ __forceinline__ int first_of(int n, F right)
{
    const int lane = threadIdx.x & 63;
    int from = 0;
    if (n > 64) {
        const uint64_t far = __ballot(right(min(lane * 64 + 63, n - 1)));
        from = far ? (int)__builtin_ctzll(far) * 64 : 63 * 64;
    }
    const uint64_t near = __ballot(right(min(from + lane, n - 1)));
    return min(near ? from + (int)__builtin_ctzll(near) : n - 1, n - 1);
}

// What is looked for in a bin, in the order of its tokens: the first one with at
// least `count` tokens and `weight` of their weights (whole numbers, both from the
// bin's beginning, the token included), or the last one.
struct Query {
    uint32_t count;
    uint64_t weight;
};
struct Found {
    uint64_t entry;        // ~key and token, as they stand in the list
    uint64_t weight;       // from the bin's beginning, the token included
};

// Ranges of bins, each an interval of the sums in front of the bins.
struct Ranges {
    int lo[4], hi[4], n, read;
    float from[4], to[4];    // logits
};

// TH threads a row.
template <int TH, typename T>
struct Draw {
    // tokens put in order at a time: as many as LDS holds for one workgroup of 1024 or two of 512 a CU
    static constexpr int kList = TH == 1024 ? 4096 : 2560;
    static constexpr int kPicked = 2 * kList;

    struct Shared {
        uint64_t work[2 * kList];        // the list and its sums; smaller bins
        double wpre[kBins + 1];          // weights and tokens in front of a bin
        uint32_t cpre[kBins + 1];
        double part_d[kBins / 128];
        unsigned long long part_u[TH / 64];
        uint32_t part_c[kBins / 128];
        uint32_t guess[kList / 2];       // two 16-bit numbers each
        uint32_t n, passed;
        int32_t hit;
        uint32_t hit_n, hit_count;
        uint64_t hit_weight, entry;
        Ranges r;
        uint32_t listed;
        int32_t least_lo, least_hi;
        int32_t at[3], place[3];         // bins of top-k, top-p and the draw (-1: not known yet), of their tokens in the list,
        double edge[3], units[3];        // their edges' weights, units of a bin in a weight of one
    };
    Shared &sh;
    const SampleArgs &a;
    const T *row;
    uint64_t *list, *upto;               // ~key and index of tokens, in order once order() was called; their weights added up
    Scale s;

    // Calls f(token, logit) for every token whose logit is in [lo, hi].
    template <typename F>
    __device__ __forceinline__ void each(float lo, float hi, F f)
    {
#pragma unroll 1
        for (int at = threadIdx.x * 8; at < a.vocab; at += TH * 8) {
            Eight<T> l;
            l.load(row + at, min(a.vocab - at, 8));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = l.get(i);
                if (x >= lo && x <= hi)
                    f(at + i, x);
            }
        }
    }

    // Puts the tokens whose logits are within one of N ranges [lo, hi] into
    // picked(), in any order, as far as they fit; sh.n counts them.
    template <int N>
    __device__ __forceinline__ void pick(const float *lo, const float *hi)
    {
        constexpr int kBatch = 4, kSpan = TH * 8;     // loads on their way together
        float from[N], to[N];
#pragma unroll
        for (int r = 0; r < N; ++r)
            from[r] = lo[r], to[r] = hi[r];
#pragma unroll 1
        for (int base = threadIdx.x * 8; base < a.vocab; base += kBatch * kSpan) {
            Eight<T> l[kBatch];
#pragma unroll
            for (int g = 0; g < kBatch; ++g)
                l[g].load(row + base + g * kSpan, min(max(a.vocab - base - g * kSpan, 0), 8));
            uint32_t hits = 0;
#pragma unroll
            for (int i = 0; i < kBatch * 8; ++i) {
                const float x = l[i >> 3].get(i & 7);
                bool hit = false;
#pragma unroll
                for (int r = 0; r < N; ++r)
                    hit |= x >= from[r] && x <= to[r];
                hits = hits + hits + (hit ? 1u : 0u);
            }
            while (hits) {
                const int i = __builtin_clz(hits);
                hits &= ~(0x80000000u >> i);
                const uint32_t n = atomicAdd(&sh.n, 1u);
                if (n < kPicked)
                    picked()[n] = (uint32_t)(base + (i >> 3) * kSpan + (i & 7));
            }
        }
    }
    __device__ __forceinline__ uint32_t *picked() const { return reinterpret_cast<uint32_t *>(upto); }

    // Puts the list's n entries in order and adds their weights up.  Where an entry
    // will stand is guessed from its place in its bin (r: the list's bins; none: all
    // entries are of one bin, with keys from klo to khi); entries of one guess count
    // those before them among themselves.
    __device__ __forceinline__ void order(int n, const Ranges *r, uint32_t klo, uint32_t khi)
    {
        if (n <= kFew) {
            uint64_t e = 0;
            int before = 0;
            if ((int)threadIdx.x < n) {
                e = list[threadIdx.x];
                for (int i = 0; i < n; ++i)
                    before += list[i] < e;
            }
            __syncthreads();
            if ((int)threadIdx.x < n)
                list[before] = e;
        } else {
            constexpr int per = kList / TH;
            for (int i = threadIdx.x; i < kList / 2; i += TH)
                sh.guess[i] = 0;
            __syncthreads();
            uint64_t e[per];
            uint32_t at[per], place[per];
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const int j = threadIdx.x + i * TH;
                at[i] = place[i] = 0;
                e[i] = ~0ull;
                if (j < n) {
                    e[i] = list[j];
                    const uint32_t key = ~(uint32_t)(e[i] >> 32);
                    if (r) {
                        const float l = logit_of(key);
                        const int b = (int)s.bin(l);
                        const uint32_t held = sh.cpre[b + 1] - sh.cpre[b];
                        for (int q = 0; q < r->n; ++q)
                            at[i] += sh.cpre[min(max(b, r->lo[q]), r->hi[q] + 1)] - sh.cpre[r->lo[q]];
                        at[i] += s.guess(l, sizeof(T) == 2, (uint32_t)e[i], a.vocab, held);
                    } else {
                        at[i] = (uint32_t)(((uint64_t)(khi - key) * (uint32_t)n) / ((uint64_t)(khi - klo) + 1));
                    }
                    const int half = 16 * (at[i] & 1);
                    place[i] = atomicAdd(&sh.guess[at[i] >> 1], 1u << half) >> half & 0xFFFFu;
                }
            }
            __syncthreads();
            uint32_t have[per], mine = 0, all;
            uint16_t *guess = reinterpret_cast<uint16_t *>(sh.guess);
#pragma unroll
            for (int i = 0; i < per; ++i)
                mine += have[i] = guess[threadIdx.x * per + i];
            uint32_t before = scan<TH>(mine, sh.part_c, all);
#pragma unroll
            for (int i = 0; i < per; ++i) {
                guess[threadIdx.x * per + i] = (uint16_t)before;
                before += have[i];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < per; ++i)
                if (threadIdx.x + i * TH < (unsigned)n)
                    upto[guess[at[i]] + place[i]] = e[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < per; ++i)
                if (threadIdx.x + i * TH < (unsigned)n) {
                    const int from = guess[at[i]], to = at[i] + 1 < (unsigned)kList ? (int)guess[at[i] + 1] : n;
                    int rank = from;
                    for (int j = from; j < to; ++j)
                        rank += upto[j] < e[i];
                    list[rank] = e[i];
                }
        }
        __syncthreads();
        constexpr int per = kList / TH;
        const int from = threadIdx.x * per;
        unsigned long long w[per], mine = 0, all;
#pragma unroll
        for (int i = 0; i < per; ++i) {
            w[i] = from + i < n ? s.weight(logit_of(~(uint32_t)(list[from + i] >> 32))) : 0;
            mine += w[i];
        }
        uint64_t sum = scan<TH>(mine, sh.part_u, all);
#pragma unroll
        for (int i = 0; i < per; ++i) {
            sum += w[i];
            upto[from + i] = sum;
        }
        __syncthreads();
    }

    // The query's token among the list's entries from .. from + n - 1, which are in
    // order, with count0 tokens and weight0 in front of them.
    __device__ __forceinline__ Found among(int from, int n, uint32_t count0, uint64_t weight0, Query q) const
    {
        const uint64_t base = from ? upto[from - 1] : 0;
        // the last one has what is asked for
        const int at = first_of(n, [&](int i) { return count0 + i + 1 >= q.count && weight0 + upto[from + i] - base >= q.weight; });
        return {list[from + at], weight0 + upto[from + at] - base};
    }

    // The query's token of bin b, which holds n, however many they are.
    __device__ Found search(int b, uint32_t n, Query q)
    {
        float from, to;
        s.span(b, b, from, to);
        uint32_t klo = key_of(from), khi = key_of(to);
        uint32_t count0 = 0;         // tokens and weight of the bin in front of [klo, khi]
        uint64_t weight0 = 0;
        while (n > kList && klo < khi) {
            // 2048 smaller bins over the keys, from the largest on
            int shift = 0;
            while ((khi - klo) >> shift >= kBins)
                ++shift;
            static_assert(kBins / 2 + kBins <= 2 * kList, "counts and sums");
            uint32_t *counts = reinterpret_cast<uint32_t *>(sh.work);
            uint64_t *sums = sh.work + kBins / 2;
            __syncthreads();
            for (int i = threadIdx.x; i < kBins; i += TH)
                counts[i] = 0, sums[i] = 0;
            __syncthreads();
            each(logit_of(klo), logit_of(khi), [&](int, float x) {
                if (within(x, klo, khi) && s.bin(x) == b) {
                    const uint32_t i = (khi - key_of(x)) >> shift;
                    atomicAdd(&counts[i], 1u);
                    atomicAdd((unsigned long long *)&sums[i], (unsigned long long)s.weight(x));
                }
            });
            __syncthreads();
            constexpr int per = kBins / TH;
            const int i0 = threadIdx.x * per;
            uint32_t c = 0, call;
            unsigned long long w = 0, wall;
#pragma unroll
            for (int i = 0; i < per; ++i)
                c += counts[i0 + i], w += sums[i0 + i];
            uint32_t cs = count0 + scan<TH>(c, sh.part_c, call);
            uint64_t wsum = weight0 + scan<TH>(w, sh.part_u, wall);
            q.weight = min(q.weight, weight0 + (uint64_t)wall);      // roundings may ask for more than there is
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const uint32_t cn = counts[i0 + i];
                const uint64_t wn = sums[i0 + i];
                if ((cs < q.count || wsum < q.weight) && cs + cn >= q.count && wsum + wn >= q.weight) {
                    sh.hit = i0 + i;
                    sh.hit_n = cn;
                    sh.hit_count = cs;
                    sh.hit_weight = wsum;
                }
                cs += cn;
                wsum += wn;
            }
            __syncthreads();
            n = sh.hit_n, count0 = sh.hit_count, weight0 = sh.hit_weight;
            khi -= (uint32_t)sh.hit << shift;
            const uint32_t span = (1u << shift) - 1;
            klo = khi - klo > span ? khi - span : klo;
            __syncthreads();
        }
        if (n > kList) {
            // equal logits alone: the one at its place among them, by index
            const float l = logit_of(khi);
            const uint64_t w = s.weight(l);
            uint64_t need = q.count > count0 ? q.count - count0 : 1;
            if (q.weight > weight0) {
                const uint64_t by_weight = (q.weight - weight0 + w - 1) / w;
                need = min(by_weight > need ? by_weight : need, (uint64_t)n);
            }
            // each thread's share is a stretch of the row here
            const int per = (a.vocab + TH - 1) / TH, first = min((int)threadIdx.x * per, a.vocab);
            const int last = min(first + per, a.vocab);
            uint32_t mine = 0, all;
            for (int i = first; i < last; ++i)
                mine += one_of(row, i) == l;
            uint32_t before = scan<TH>(mine, sh.part_c, all);
            if (before < need && before + mine >= need)
                for (int i = first; i < last; ++i)
                    if (one_of(row, i) == l && ++before == need)
                        sh.entry = (uint64_t)~khi << 32 | (uint32_t)i;
            __syncthreads();
            const Found f{sh.entry, weight0 + need * w};
            __syncthreads();
            return f;
        }
        if (threadIdx.x == 0)
            sh.n = 0;
        __syncthreads();
        each(logit_of(klo), logit_of(khi), [&](int at, float x) {
            if (within(x, klo, khi) && s.bin(x) == b)
                list[min(atomicAdd(&sh.n, 1u), (uint32_t)kList - 1)] = (uint64_t)~key_of(x) << 32 | (uint32_t)at;
        });
        __syncthreads();
        order((int)min(sh.n, (uint32_t)kList), nullptr, klo, khi);
        const Found f = among(0, (int)n, count0, weight0, q);
        __syncthreads();
        return f;
    }
};

// A border: the last kept token, or the one drawn.
struct Border {
    double weight;       // of the tokens up to it and with it
    int bin;
    Found f;             // within the bin; its entry only where it is looked for
};

template <int TH, typename T>
__global__ __launch_bounds__(TH) __attribute__((amdgpu_waves_per_eu(4, 4)))
void sample_draw(SampleArgs a, const Part *__restrict__ parts, int32_t splits)
{
    constexpr int kList = Draw<TH, T>::kList;
    __shared__ typename Draw<TH, T>::Shared sh;
    const int64_t row = blockIdx.x;
    parts += row * splits;
    const float t = a.temperature ? a.temperature[row] : a.temperature_all;
    float top = -INFINITY;
    for (int i = threadIdx.x & 63; i < splits; i += 64)
        top = fmaxf(top, parts[i].top);
    top = wave_max(top);
    if (top == -INFINITY || greedy(t)) {
        if (threadIdx.x == 0) {
            int32_t first = -1;
            for (int i = splits - 1; i >= 0 && top != -INFINITY; --i)
                if (parts[i].top == top)
                    first = parts[i].first;
            a.tokens[row] = first;
            if (a.logprobs)
                a.logprobs[row] = first < 0 ? -INFINITY : 0.0f;
        }
        return;
    }
    Draw<TH, T> d{sh, a, static_cast<const T *>(a.logits) + row * a.stride, sh.work, sh.work + kList, {}};
    Scale &s = d.s;
    s.set(t, top);

    // The row's bins, and the sums of counts and weights in front of them.  Two bins of a pair are
    // added up first and the pairs stand as the places of 1024 threads do, however many there
    // are: the weights' sums, which are rounded, are the same ones.
    constexpr int per = kBins / TH, kPairs = per / 2;
    auto bin_at = [&](int i) { return ((i >> 1) * TH + (int)threadIdx.x) * 2 + (i & 1); };
    uint64_t count[per], excess[per];
#pragma unroll
    for (int i = 0; i < per; ++i)
        count[i] = excess[i] = 0;
    constexpr int kTogether = 4;         // parts whose loads are on their way together
    for (int p = 0; p < splits; p += kTogether) {
        float first[kTogether];
        uint64_t v[kTogether][per];
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
            first[q] = p + q < splits ? s.bin(parts[p + q].top) : INFINITY;      // the part's first bin among the row's
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int i = 0; i < per; ++i) {
                v[q][i] = 0;
                if (first[q] <= (float)bin_at(i))
                    v[q][i] = parts[p + q].bins[bin_at(i) - (int)first[q]];
            }
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int i = 0; i < per; ++i) {
                count[i] += v[q][i] >> kCountShift;
                excess[i] += v[q][i] & kExcess;
            }
    }
    uint32_t counts[kPairs], cs[kPairs], all;
    double weight[per], weights[kPairs], ws[kPairs], total;
#pragma unroll
    for (int i = 0; i < per; ++i) {
#pragma clang fp contract(off)
        const uint64_t w = count[i] * (uint64_t)kOne + excess[i];
        weight[i] = w ? (double)w * (1.0 / kOne) * s.edge_weight(bin_at(i)) : 0.0;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        counts[i] = (uint32_t)count[2 * i] + (uint32_t)count[2 * i + 1];
        weights[i] = weight[2 * i] + weight[2 * i + 1];
    }
    scan<TH>(counts, sh.part_c, cs, all);
    scan<TH>(weights, sh.part_d, ws, total);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int b = bin_at(2 * i);
        sh.cpre[b] = cs[i];
        sh.wpre[b] = ws[i];
        sh.cpre[b + 1] = cs[i] + (uint32_t)count[2 * i];
        sh.wpre[b + 1] = ws[i] + weight[2 * i];
    }
    if (threadIdx.x == TH - 1) {
        sh.cpre[kBins] = cs[kPairs - 1] + counts[kPairs - 1];
        sh.wpre[kBins] = ws[kPairs - 1] + weight[per - 2] + weight[per - 1];
    }
    if (threadIdx.x == 0)
        sh.n = sh.passed = 0;
    __syncthreads();

    // the first bin with c tokens, or w of the weights (`past`: more), up to its end; the last one with any where there is none
    auto bin_of = [&](uint32_t c, double w, bool past) {
        int b = first_of(kBins, [&](int i) {
            const double x = sh.wpre[i + 1];
            return sh.cpre[i + 1] >= c && (past ? x > w : x >= w);
        });
        // roundings of the sums may end at a bin without tokens: the next one with any, or the last
        if (sh.cpre[b + 1] == sh.cpre[b]) {
            const uint32_t next = min(sh.cpre[b] + 1, all);
            b = first_of(kBins, [&](int i) { return sh.cpre[i + 1] >= next; });
        }
        return b;
    };

    // Which bins hold a border, and between what the kept weight lies.
    const float p = a.top_p ? a.top_p[row] : a.top_p_all;
    const float least = a.min_p ? a.min_p[row] : a.min_p_all;
    // no token weighs more than one: a limit above that leaves the first alone
    const int32_t k = least > 1.0f ? 1 : a.top_k ? a.top_k[row] : a.top_k_all;
    const bool by_k = k > 0 && (uint32_t)k < all, by_p = p < 1.0f, by_least = least > 0.0f && least <= 1.0f && !s.alone && !s.flat;
    constexpr double kLess = 1.0 - 0x1p-45, kMore = 1.0 + 0x1p-45;     // roundings of the sums
    const float u = a.u[row] > 0.0f ? a.u[row] : 0.0f;
    // below the kept weight whatever u
    auto target = [&](double kept) { return fmin((double)u * kept, kept * (1.0 - 0x1p-52)); };
    if (threadIdx.x < 64) {
        // the borders' ranges of bins: top-k, top-p, min-p, the draw; from..to -1 where there is none
        int from[4], to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            from[i] = kBins, to[i] = -1;
        double wlo = total * kLess, whi = total * kMore;
        int last_bin = kBins - 1, least_lo = kBins;
        // the weight kept ends in the bins lo .. hi, and within [least, most]
        auto kept_within = [&](int i, int lo, int hi, double least, double most) {
            from[i] = lo;
            to[i] = hi;
            last_bin = hi;
            wlo = fmin(wlo, fmax(sh.wpre[lo], least) * kLess);
            whi = fmin(whi, fmin(sh.wpre[hi + 1], most) * kMore);
        };
        // A bin's tokens differ by exp(1/32) at most, the heaviest stand first: what the
        // first of them weigh in the mean, at least and at most.  With bounds as near as
        // this the next border is in one bin nearly always, and all borders' tokens fit the list.
        constexpr double kLightest = 1.0 - 0x1p-30, kHeaviest = 1.04;
        auto mean_of = [&](int b) { return (sh.wpre[b + 1] - sh.wpre[b]) / (double)max(sh.cpre[b + 1] - sh.cpre[b], 1u); };
        // the bins of the weights w0 and w1 >= w0
        auto bins_of = [&](double w0, double w1, bool past, int &lo, int &hi) {
            lo = hi = bin_of(1, w0, past);
            const double x = sh.wpre[lo + 1];
            if (!(past ? x > w1 : x >= w1))
                hi = bin_of(1, w1, past);
        };
        int at[3] = {-1, -1, -1};        // the bins of top-k, top-p and the draw, where they are known already
        if (by_k) {
            at[0] = bin_of((uint32_t)k, 0.0, false);
            const double first = (double)((uint32_t)k - sh.cpre[at[0]]) * mean_of(at[0]);
            kept_within(0, at[0], at[0], sh.wpre[at[0]] + first * kLightest, sh.wpre[at[0]] + first * kHeaviest);
        }
        if (by_p) {
            const double w0 = p > 0.0f ? (double)p * wlo : 0.0, w1 = p > 0.0f ? (double)p * whi : 0.0;
            int lo, hi;
            bins_of(w0, w1, false, lo, hi);
            at[1] = lo == hi && hi <= last_bin ? lo : -1;
            lo = min(lo, last_bin);
            // up to one token past what is asked for
            kept_within(1, lo, min(hi, last_bin), w0, w1 + mean_of(lo) * kHeaviest);
        }
        if (by_least) {
            // exp((l - top) / T) >= min_p from top + T ln(min_p) on, give or take the roundings
            const double z = s.t * log((double)least), off = 1e-13 * (fabs((double)top) + fabs(z) + s.t);
            const double lo = (double)s.top_bin - floor(ldexp((double)top + z + off, s.shift));
            const double hi = (double)s.top_bin - floor(ldexp((double)top + z - off, s.shift));
            const int first = (int)fmax(0.0, fmin(lo, (double)kBins));
            if (first <= last_bin) {
                least_lo = first;
                kept_within(2, first, min((int)fmin(hi, (double)kBins - 1), last_bin), 0.0, INFINITY);
                sh.least_hi = last_bin;
            }
        }
        int lo, hi;
        bins_of(target(wlo), target(whi), true, lo, hi);
        at[2] = lo == hi && hi <= last_bin ? lo : -1;
        to[3] = min(hi, last_bin);
        from[3] = min(lo, to[3]);
        // in the order of the bins, joined where they meet
#pragma unroll
        for (int pass = 0; pass < 3; ++pass)
#pragma unroll
            for (int i = 0; i < 3 - pass; ++i)
                if (from[i + 1] < from[i]) {
                    const int f = from[i], e = to[i];
                    from[i] = from[i + 1], to[i] = to[i + 1];
                    from[i + 1] = f, to[i + 1] = e;
                }
        // lane i: range i
        const int lane = threadIdx.x;
        int n = 0, mine_lo = 0, mine_hi = -1;
        {
            int f = from[0], e = to[0];
#pragma unroll
            for (int i = 1; i < 5; ++i) {
                const bool more = i < 4 && from[i < 4 ? i : 3] < kBins;
                if (more && from[i < 4 ? i : 3] <= e) {
                    e = max(e, to[i < 4 ? i : 3]);
                } else if (more || i == 4) {
                    if (lane == n)
                        mine_lo = f, mine_hi = e;
                    ++n;
                    if (more)
                        f = from[i < 4 ? i : 3], e = to[i < 4 ? i : 3];
                }
            }
        }
        const uint32_t first = sh.cpre[mine_lo], past = sh.cpre[mine_hi + 1];
        const uint32_t upto = wave_scan(lane < n ? past - first : 0u);
        const uint32_t listed = (uint32_t)__builtin_amdgcn_readlane((int)upto, 3);
        const uint32_t all_of = (uint32_t)__builtin_amdgcn_readlane((int)past, n - 1) - (uint32_t)__builtin_amdgcn_readlane((int)first, 0);
        const int read = ranges_read(n, listed, all_of, a.vocab, Draw<TH, T>::kPicked);
        Ranges &r = sh.r;
        if (lane < n) {
            r.lo[lane] = mine_lo;
            r.hi[lane] = mine_hi;
            s.span(mine_lo, mine_hi, r.from[lane], r.to[lane]);
        }
        if (read == 1 && lane == n - 1)
            r.from[0] = r.from[n - 1];
        uint32_t place[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
            place[i] = wave_scan(lane < n ? sh.cpre[min(max(at[i], mine_lo), mine_hi + 1)] - first : 0u);
        if (lane < 3) {
            const int b = lane == 0 ? at[0] : lane == 1 ? at[1] : at[2];
            sh.at[lane] = b;
            sh.edge[lane] = s.edge_weight(max(b, 0));
            sh.units[lane] = kOne / sh.edge[lane];
        }
        if (lane == 3) {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                sh.place[i] = (int)place[i];
        }
        r.n = n;
        r.read = read;
        sh.listed = listed;
        sh.least_lo = least_lo;
    }
    __syncthreads();
    const Ranges &r = sh.r;
    auto heavy = [&](float x) { return exp(((double)x - (double)top) / s.t) >= (double)least; };
    const uint32_t listed = sh.listed;
    const int least_lo = sh.least_lo;
    bool gathered = listed <= kList;
    if (gathered) {
        switch (r.read) {
        case 1: d.template pick<1>(r.from, r.to); break;
        case 2: d.template pick<2>(r.from, r.to); break;
        case 3: d.template pick<3>(r.from, r.to); break;
        default: d.template pick<4>(r.from, r.to); break;
        }
        __syncthreads();
        const uint32_t n = sh.n;
        gathered = n <= (uint32_t)Draw<TH, T>::kPicked;
        __syncthreads();
        if (threadIdx.x == 0)
            sh.n = 0;
        __syncthreads();
        for (uint32_t i = threadIdx.x; gathered && i < n; i += TH) {
            const uint32_t at = d.picked()[i];
            const float x = one_of(d.row, (int)at), b = s.bin(x);
            bool within = false;
            for (int j = 0; j < r.n; ++j)
                within |= b >= (float)r.lo[j] && b <= (float)r.hi[j];
            if (!within)
                continue;
            if (b >= (float)least_lo && heavy(x))
                atomicAdd(&sh.passed, 1u);
            d.list[min(atomicAdd(&sh.n, 1u), (uint32_t)kList - 1)] = (uint64_t)~key_of(x) << 32 | at;
        }
        __syncthreads();
        if (gathered)
            d.order((int)min(sh.n, (uint32_t)kList), &r, 0, 0);
    }
    if (!gathered && least_lo < kBins) {
        float lo, hi;
        s.span(least_lo, sh.least_hi, lo, hi);
        d.each(lo, hi, [&](int, float x) {
            const float b = s.bin(x);
            if (b >= (float)least_lo && b <= (float)sh.least_hi && heavy(x))
                atomicAdd(&sh.passed, 1u);
        });
        __syncthreads();
    }
    // what is left is one wave's work, as long as the list has what is looked for
    if (gathered && threadIdx.x >= 64)
        return;

    // Where the kept tokens end; nothing is looked for past it.
    Border cap{total, kBins, {0, 0}};
    // which: 0 top-k, 1 top-p, 2 the draw, 3 min-p
    auto border = [&](int which, uint32_t c, double w, bool past) -> Border {
        const bool known = which < 3 && sh.at[which < 3 ? which : 0] >= 0;
        int b = known ? sh.at[which] : bin_of(c, w, past);
        if (b > cap.bin) {
            if (!past)
                return cap;
            b = cap.bin;
        }
        const uint32_t before = sh.cpre[b], n = sh.cpre[b + 1] - before;
        if (c == before + n && !(w > 0.0) && !past)
            return {sh.wpre[b + 1], b, {0, ~0ull}};      // the bin's end, of whatever tokens
        const bool prepared = known && b == sh.at[which];
        const double wb = sh.wpre[b], edge = prepared ? sh.edge[which] : s.edge_weight(b);
        // whole units of the bin's weight that the token has to reach, of those that the limits keep
        double units = (w - wb) * (prepared ? sh.units[which] : kOne / edge);
        units = past ? floor(units) + 1.0 : ceil(units);
        Query q;
        q.count = c > before ? c - before : 0;
        q.weight = units > 0 ? (uint64_t)fmin(units, 0x1p62) : 0;
        if (b == cap.bin && q.weight > cap.f.weight)
            q.weight = cap.f.weight;
        if (q.count == 0 && q.weight == 0)
            q.count = 1;
        Found f;
        int at = prepared ? sh.place[which] : 0;     // of the bin's tokens in the list
        bool within = prepared;
        for (int i = 0; i < (prepared ? 0 : r.n); ++i) {
            at += (int)(sh.cpre[min(max(b, r.lo[i]), r.hi[i] + 1)] - sh.cpre[r.lo[i]]);
            within |= b >= r.lo[i] && b <= r.hi[i];
        }
        if (gathered && within)
            f = d.among(at, (int)n, 0, 0, q);
        else if (!gathered)
            f = d.search(b, n, q);
        else
            f = {d.list[listed - 1], ~0ull};      // not met: the ranges allow for the sums' roundings
        return {wb + (double)f.weight * (1.0 / kOne) * edge, b, f};
    };
    const uint32_t passed = least_lo < kBins ? sh.cpre[least_lo] + sh.passed : all;
    uint64_t entry = 0;
    double kept = 0;
#pragma unroll 1
    for (int stage = 0; stage < 4; ++stage) {
        uint32_t c = 1;
        double w = 0.0;
        if (stage == 0) {
            if (!by_k)
                continue;
            c = (uint32_t)k;
        } else if (stage == 1) {
            if (!by_p)
                continue;
            w = p > 0.0f ? (double)p * cap.weight : 0.0;
        } else if (stage == 2) {
            if (passed >= all)
                continue;
            c = passed;
        } else {
            kept = cap.weight;
            w = target(kept);
            if (u >= 1.0f) {
                // the last kept token, which may weigh less than a rounding of the sums
                if (cap.bin < kBins && cap.f.weight != ~0ull) {
                    entry = cap.f.entry;
                    continue;
                }
                c = sh.cpre[min(cap.bin, kBins - 1) + 1];
                w = 0.0;
            }
        }
        const Border e = border(stage == 2 ? 3 : min(stage, 2), c, w, stage == 3);
        if (stage == 3)
            entry = e.f.entry;
        else if (e.bin < cap.bin || (e.bin == cap.bin && e.f.weight < cap.f.weight))
            cap = e;
    }
    if (threadIdx.x == 0) {
        a.tokens[row] = (int32_t)entry;
        if (a.logprobs) {
#pragma clang fp contract(off)
            // from the weight as it stands in the sums, rounded alike: what else is kept is so right next to a
            // probability of one too, and nothing where the token is kept alone
            const float l = logit_of(~(uint32_t)(entry >> 32));
            const double w = (double)s.weight(l) * (1.0 / kOne) * s.edge_weight((int)s.bin(l));
            a.logprobs[row] = (float)(0.0 - log1p(fmax(kept - w, 0.0) / w));
        }
    }
}

// Groups of eight logits a thread of sample_bins: as many as leave two
// workgroups a CU, up to what fits the registers of 32 waves a CU.
int groups(int64_t m, int64_t vocab)
{
    int g = 4;
    while (g > 1 && m * ((vocab + g * 8 * kBinThreads - 1) / (g * 8 * kBinThreads)) < 512)
        g /= 2;
    return g;
}

int parts_of(int64_t m, int64_t vocab)
{
    const int64_t part = (int64_t)groups(m, vocab) * 8 * kBinThreads;
    return (int)((vocab + part - 1) / part);
}

template <typename T>
void start(const SampleArgs &a, Part *parts, hipStream_t s)
{
    const int splits = parts_of(a.m, a.vocab);
    const dim3 grid((unsigned)(a.m * splits));
    switch (groups(a.m, a.vocab)) {
    case 4: sample_bins<4, T><<<grid, kBinThreads, 0, s>>>(a, parts, splits); break;
    case 2: sample_bins<2, T><<<grid, kBinThreads, 0, s>>>(a, parts, splits); break;
    default: sample_bins<1, T><<<grid, kBinThreads, 0, s>>>(a, parts, splits); break;
    }
    // up to a row a CU the wider form is faster; of more rows one is at its borders while another is read
    // (512 rows of 131071 bf16 logits 103 us, by the wider form 113), as long as the shorter list holds the
    // tokens of three full bins (264 rows of 250000, each with limits of its own: 258 us, 114 by the wider
    // form; 400000: 532 and 301; where few tokens are at the borders the wider form takes 3 to 15 % longer)
    if (a.m <= 256 || a.vocab > 150000)
        sample_draw<1024, T><<<(unsigned)a.m, 1024, 0, s>>>(a, parts, splits);
    else
        sample_draw<512, T><<<(unsigned)a.m, 512, 0, s>>>(a, parts, splits);
}

// Rows go by slices whose bins take 2^28 bytes and a little.
int64_t slice_rows(int64_t vocab)
{
    return ((1 << 28) / (int64_t)sizeof(Part)) / ((vocab + 4 * 8 * kBinThreads - 1) / (4 * 8 * kBinThreads));
}

}  // namespace

size_t sample_workspace_bytes(int64_t m, int64_t vocab)
{
    const int64_t slice = slice_rows(vocab), first = m < slice ? m : slice, last = m < slice ? m : m % slice;
    const int64_t most = first * parts_of(first, vocab), tail = last * parts_of(last, vocab);
    return (size_t)(most > tail ? most : tail) * sizeof(Part);
}

hipError_t launch_sample(const SampleArgs &args, void *workspace, hipStream_t s)
{
    Part *parts = static_cast<Part *>(workspace);
    const int64_t slice = slice_rows(args.vocab);
    for (int64_t row = 0; row < args.m; row += slice) {
        SampleArgs a = args;
        a.m = args.m - row < slice ? args.m - row : slice;
        a.logits = static_cast<const char *>(args.logits) + row * args.stride * (args.f32 ? 4 : 2);
        a.u += row;
        a.tokens += row;
        a.temperature = args.temperature ? args.temperature + row : nullptr;
        a.top_k = args.top_k ? args.top_k + row : nullptr;
        a.top_p = args.top_p ? args.top_p + row : nullptr;
        a.min_p = args.min_p ? args.min_p + row : nullptr;
        a.logprobs = args.logprobs ? args.logprobs + row : nullptr;
        if (a.f32)
            start<float>(a, parts, s);
        else
            start<uint16_t>(a, parts, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace bd
