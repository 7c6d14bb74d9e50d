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
//   sample_draw  one workgroup a row adds the parts' bins up, finds the bin of each
//                border (top-k, top-p, min-p, the draw), and the place within it.
//
// Bins are d = 2^e wide, T / 64 < d <= T / 32, at multiples of d, so the parts' bins
// are the same ones; 2048 of them reach exp(-32) below the part's largest logit, and
// what lies deeper has no weight.  In a bin with upper edge E the weight relative to
// it, exp((l - E) / T), is within 1/32 of one; what is missing to one, held in units
// of 2^-36, and the count share a 64-bit number, so that one LDS addition serves
// both, and all sums are of whole numbers: exact, in any order, cut in any way.
#include "bd_device.h"
#include "sample_launch.h"

namespace bd {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kCountShift = 47;              // of a packed bin: below it 65536 tokens' missing weight, each below 2^31
constexpr uint64_t kMissing = (1ull << kCountShift) - 1;
constexpr double kOne = 0x1p36;              // weight of a token at its bin's upper edge
constexpr int kList = 4096;                  // tokens put in order at a time

typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

// Logits as they count: NaN is never drawn, like -inf, and the zeros are equal.
__device__ __forceinline__ float counted(float l) { return l == l ? l + 0.0f : -INFINITY; }

__device__ __forceinline__ void load8(const uint16_t *p, int n, float *l)
{
    if (n == 8) {
        const u32x4 w = *reinterpret_cast<const u32x4a2 *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            l[i] = counted(i & 1 ? hi_f32(w[i >> 1]) : lo_f32(w[i >> 1]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        l[i] = i < n ? counted(__uint_as_float((uint32_t)p[i] << 16)) : -INFINITY;
}

__device__ __forceinline__ void load8(const float *p, int n, float *l)
{
    if (n == 8) {
        const u32x4 a = *reinterpret_cast<const u32x4a4 *>(p), b = *reinterpret_cast<const u32x4a4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            l[i] = counted(__uint_as_float(a[i])), l[4 + i] = counted(__uint_as_float(b[i]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        l[i] = i < n ? counted(p[i]) : -INFINITY;
}

// Numbers that order as the logits do, and back.
__device__ __forceinline__ uint32_t key_of(float l)
{
    const uint32_t b = __float_as_uint(l);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t k)
{
    return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

// The bins of a row, counted downwards from the one of `top`.
struct Scale {
    double to_bin, width, top_bin;    // 1/d, d/T, floor(top / d)
    float top;
    bool flat, drawn_max;             // T = +inf: all tokens of weight one; top = +inf: those alone

    __device__ __forceinline__ void set(float temperature, float largest)
    {
        top = largest;
        flat = temperature == INFINITY;
        drawn_max = largest == INFINITY;
        int e;
        frexp((double)temperature, &e);                       // T in [2^(e-1), 2^e)
        to_bin = flat ? 0.0 : ldexp(1.0, 6 - e);              // d = 2^(e-6): T / 64 < d <= T / 32
        width = flat ? 0.0 : ldexp(1.0, e - 6) / (double)temperature;
        top_bin = drawn_max || flat ? 0.0 : floor((double)largest * to_bin);
    }
    // Bin of l (kBins: none), and how far below the bin's upper edge it lies, in bins.
    __device__ __forceinline__ int bin(float l, double &below) const
    {
        below = 0.0;
        if (l == -INFINITY)
            return kBins;
        if (drawn_max)
            return l == INFINITY ? 0 : kBins;
        if (flat)
            return 0;
        const double a = (double)l * to_bin, b = floor(a), rel = top_bin - b;
        below = b + 1.0 - a;
        return rel < kBins ? (int)rel : kBins;
    }
    // 1 - exp(-x), x <= 1/32, in units of 2^-36: the series to x^6 is within 2^-47
    __device__ __forceinline__ uint64_t missing(double below) const
    {
        const double x = below * width;
        double s = fma(x, -1.0 / 720.0, 1.0 / 120.0);
        s = fma(x, s, -1.0 / 24.0);
        s = fma(x, s, 1.0 / 6.0);
        s = fma(x, s, -0.5);
        s = fma(x, s, 1.0);
        // adding 2^52 leaves the whole number in the low bits
        return (uint64_t)__double_as_longlong(fma(x * s, kOne, 0x1p52)) & kMissing;
    }
    // weight of the upper edge of bin b, relative to the largest logit
    __device__ __forceinline__ double edge(int b, double temperature) const
    {
        if (drawn_max || flat)
            return 1.0;
        return exp(((top_bin - b + 1.0) / to_bin - (double)top) / temperature);
    }
};

__device__ __forceinline__ bool greedy(float t) { return !(t > 0.0f); }

// What sample_bins leaves of a part: the largest logit and, for rows that take
// it, the first token that has it; then kBins packed bins.
struct Part {
    float top;
    int32_t first;
    uint64_t pad;
    uint64_t bins[kBins];
};

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

// G groups of eight logits a thread.
template <int G, typename T>
__global__ __launch_bounds__(kThreads) void sample_bins(SampleArgs a, Part *__restrict__ parts, int32_t splits)
{
    __shared__ uint64_t bins[kBins];
    __shared__ float tops[kThreads / 64];
    __shared__ int32_t first;
    const int64_t row = blockIdx.x / (unsigned)splits;
    const int split = blockIdx.x % (unsigned)splits;
    const T *p = static_cast<const T *>(a.logits) + row * a.stride;
    const int at0 = split * (G * 8 * kThreads) + threadIdx.x * 8;
    float l[G][8];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int at = at0 + g * 8 * kThreads;
        load8(p + at, min(max(a.vocab - at, 0), 8), l[g]);
    }
    const float t = a.temperature ? a.temperature[row] : a.temperature_all;
    for (int i = threadIdx.x; i < kBins; i += kThreads)
        bins[i] = 0;
    if (threadIdx.x == 0)
        first = 0x7FFFFFFF;
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = fmaxf(top, l[g][i]);
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0)
        tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = wave_max(tops[threadIdx.x & (kThreads / 64 - 1)]);

    Part &out = parts[blockIdx.x];
    if (greedy(t)) {
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int g = G - 1; g >= 0; --g)
#pragma unroll
            for (int i = 7; i >= 0; --i)
                if (l[g][i] == top)
                    at = at0 + g * 8 * kThreads + i;
        if (at != 0x7FFFFFFF)
            atomicMin(&first, at);
        __syncthreads();
        if (threadIdx.x == 0) {
            out.top = top;
            out.first = first;
        }
        return;
    }
    Scale s;
    s.set(t, top);
    if (top != -INFINITY)
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                double below;
                const int b = s.bin(l[g][i], below);
                if (b < kBins)
                    atomicAdd((unsigned long long *)&bins[b], (1ull << kCountShift) | s.missing(below));
            }
    __syncthreads();
    if (threadIdx.x == 0)
        out.top = top;
    for (int i = threadIdx.x; i < kBins; i += kThreads)
        out.bins[i] = bins[i];
}

// Sum of v over the threads before this one; `total` over all of them.
template <typename V>
__device__ __forceinline__ V scan(V v, V *part, V &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    V s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const V n = __shfl_up(s, o);
        s += lane >= o ? n : V(0);
    }
    __syncthreads();          // part may still be read from the scan before
    if (lane == 63)
        part[wave] = s;
    __syncthreads();
    V before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        const V x = part[w];
        before += w < wave ? x : V(0);
        total += x;
    }
    return before + s - v;
}

// What is looked for in a bin, in the order of its tokens: the first one with at
// least `count` tokens and `weight` of their weights (whole numbers, both from the
// bin's beginning, the token included).
struct Query {
    uint32_t count;
    uint64_t weight;
};
struct Found {
    int32_t token;
    uint32_t key;
    uint64_t weight;       // from the bin's beginning, the token included
};

template <typename T>
struct Draw {
    // LDS
    struct Shared {
        uint64_t list[kList];
        uint32_t counts[kBins];
        uint64_t sums[kBins];
        double part_d[kThreads / 64];
        unsigned long long part_u[kThreads / 64];
        uint32_t part_c[kThreads / 64];
        uint32_t n, klo, khi;
        int32_t token, bin;
        uint64_t weight;
        double before;
    };
    Shared &sh;
    const SampleArgs &a;
    const T *row;
    Scale s;

    // Calls f(token, logit) for every token of bin b whose key is within [klo, khi].
    template <typename F>
    __device__ __forceinline__ void each(int b, uint32_t klo, uint32_t khi, F f)
    {
        for (int at = threadIdx.x * 8; at < a.vocab; at += kThreads * 8) {
            float l[8];
            load8(row + at, min(a.vocab - at, 8), l);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                double below;
                const uint32_t k = key_of(l[i]);
                if (k >= klo && k <= khi && s.bin(l[i], below) == b)
                    f(at + i, l[i], k, below);
            }
        }
    }

    // The token of bin b that the query asks for; n of them are there.
    __device__ Found find(int b, uint32_t n, Query q)
    {
        // keys of the bin's edges, one step to the outside of their roundings
        uint32_t klo = 0, khi = 0xFFFFFFFFu;
        if (!s.flat && !s.drawn_max) {
            const float lo = (float)((s.top_bin - b) / s.to_bin), hi = (float)((s.top_bin - b + 1.0) / s.to_bin);
            klo = key_of(counted(lo)) - 1;
            khi = key_of(counted(hi)) + 1;
        }
        uint32_t count0 = 0;         // tokens and weight of the bin in front of [klo, khi]
        uint64_t weight0 = 0;
        while (n > kList && klo < khi) {
            // too many to put in order: 2048 smaller bins over the keys, from the largest on
            int shift = 0;
            while ((khi - klo) >> shift >= kBins)
                ++shift;
            uint32_t *counts = reinterpret_cast<uint32_t *>(sh.list);
            uint64_t *sums = sh.list + kBins / 2;
            __syncthreads();
            for (int i = threadIdx.x; i < kBins; i += kThreads)
                counts[i] = 0, sums[i] = 0;
            __syncthreads();
            each(b, klo, khi, [&](int, float, uint32_t k, double below) {
                atomicAdd(&counts[(khi - k) >> shift], 1u);
                atomicAdd((unsigned long long *)&sums[(khi - k) >> shift], (unsigned long long)((uint64_t)kOne - s.missing(below)));
            });
            __syncthreads();
            const int i0 = threadIdx.x * (kBins / kThreads);
            uint32_t c = 0, call;
            unsigned long long w = 0, wall;
            for (int i = 0; i < kBins / kThreads; ++i)
                c += counts[i0 + i], w += sums[i0 + i];
            uint32_t cs = count0 + scan(c, sh.part_c, call);
            unsigned long long wsum = weight0 + scan(w, sh.part_u, wall);
            if (threadIdx.x == 0)
                sh.bin = -1;
            __syncthreads();
            for (int i = 0; i < kBins / kThreads; ++i) {
                const uint32_t cn = counts[i0 + i];
                const uint64_t wn = sums[i0 + i];
                if (cn && (cs < q.count || wsum < q.weight) && cs + cn >= q.count && wsum + wn >= q.weight) {
                    sh.bin = i0 + i;
                    sh.n = cn;
                    sh.klo = cs;
                    sh.weight = wsum;
                }
                cs += cn;
                wsum += wn;
            }
            __syncthreads();
            const int hit = sh.bin;
            n = sh.n, count0 = sh.klo, weight0 = sh.weight;
            khi = khi - ((uint32_t)hit << shift);
            const uint32_t span = (1u << shift) - 1;
            klo = khi - klo > span ? khi - span : klo;
            __syncthreads();
        }
        if (n > kList) {
            // equal logits alone: the one at its place among them, by index
            const uint64_t one = (uint64_t)kOne;
            double below;
            s.bin(logit_of(khi), below);
            const uint64_t w = one - s.missing(below);
            uint64_t need = q.count > count0 ? q.count - count0 : 1;
            if (q.weight > weight0) {
                const uint64_t by_weight = (q.weight - weight0 + w - 1) / w;
                need = by_weight > need ? by_weight : need;
            }
            // each thread's share is a stretch of the row here
            const int per = (a.vocab + kThreads - 1) / kThreads, from = threadIdx.x * per;
            const int to = min(from + per, a.vocab);
            const float l = logit_of(khi);
            uint32_t mine = 0, all;
            for (int i = from; i < to; ++i)
                mine += one_of(i) == l;
            uint32_t before = scan(mine, sh.part_c, all);
            if (before < need && before + mine >= need)
                for (int i = from; i < to; ++i)
                    if (one_of(i) == l && ++before == need)
                        sh.token = i;
            __syncthreads();
            return {sh.token, khi, weight0 + need * w};
        }
        if (threadIdx.x == 0)
            sh.n = 0;
        __syncthreads();
        each(b, klo, khi, [&](int at, float, uint32_t k, double) {
            const uint32_t i = atomicAdd(&sh.n, 1u);
            if (i < kList)
                sh.list[i] = (uint64_t)~k << 32 | (uint32_t)at;
        });
        __syncthreads();
        const int held = min(sh.n, (uint32_t)kList);
        int size = 2;
        while (size < held)
            size *= 2;
        for (int i = held + threadIdx.x; i < size; i += kThreads)
            sh.list[i] = ~0ull;
        for (int k = 2; k <= size; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                __syncthreads();
                for (int i = threadIdx.x; i < size / 2; i += kThreads) {
                    const int x = (i / j) * 2 * j + i % j, y = x + j;
                    const uint64_t p = sh.list[x], r = sh.list[y];
                    if ((p > r) == ((x & k) == 0))
                        sh.list[x] = r, sh.list[y] = p;
                }
            }
        __syncthreads();
        constexpr int per = kList / kThreads;
        const int from = threadIdx.x * per;
        unsigned long long w[per], mine = 0, all;
#pragma unroll
        for (int i = 0; i < per; ++i) {
            w[i] = 0;
            if (from + i < held) {
                double below;
                s.bin(logit_of(~(uint32_t)(sh.list[from + i] >> 32)), below);
                w[i] = (uint64_t)kOne - s.missing(below);
            }
            mine += w[i];
        }
        uint64_t sum = weight0 + scan(mine, sh.part_u, all);
        if (threadIdx.x == 0) {
            // roundings of the border's place may ask for a little more than there is: the last one then
            sh.token = (int32_t)sh.list[held - 1];
            sh.klo = ~(uint32_t)(sh.list[held - 1] >> 32);
            sh.weight = weight0 + all;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < per; ++i) {
            const bool before = count0 + from + i < q.count || sum < q.weight;
            sum += w[i];
            if (from + i < held && before && count0 + from + i + 1 >= q.count && sum >= q.weight) {
                sh.token = (int32_t)sh.list[from + i];
                sh.klo = ~(uint32_t)(sh.list[from + i] >> 32);
                sh.weight = sum;
            }
        }
        __syncthreads();
        const Found f{sh.token, sh.klo, sh.weight};
        __syncthreads();
        return f;
    }

    __device__ __forceinline__ float one_of(int i) const
    {
        if constexpr (sizeof(T) == 2)
            return counted(__uint_as_float((uint32_t)row[i] << 16));
        else
            return counted(row[i]);
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_draw(SampleArgs a, const Part *__restrict__ parts, int32_t splits)
{
    __shared__ typename Draw<T>::Shared sh;
    const int64_t row = blockIdx.x;
    parts += row * splits;
    const double t = a.temperature ? a.temperature[row] : a.temperature_all;
    float top = -INFINITY;
    for (int i = 0; i < splits; ++i)
        top = fmaxf(top, parts[i].top);
    if (top == -INFINITY || greedy((float)t)) {
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
    Draw<T> d{sh, a, static_cast<const T *>(a.logits) + row * a.stride, {}};
    Scale &s = d.s;
    s.set((float)t, top);

    // the row's bins, and the sums of counts and weights in front of them
    constexpr int per = kBins / kThreads;
    const int b0 = threadIdx.x * per;
    uint32_t count[per], counts = 0, all;
    double weight[per], weights = 0, total;
#pragma unroll
    for (int i = 0; i < per; ++i) {
        uint64_t n = 0, missing = 0;
        for (int p = 0; p < splits; ++p) {
            double below;
            const float largest = parts[p].top;
            // the part's first bin among the row's
            const int shift = s.bin(largest, below), b = b0 + i - shift;
            if (b >= 0 && b < kBins && shift < kBins) {
                const uint64_t v = parts[p].bins[b];
                n += v >> kCountShift;
                missing += v & kMissing;
            }
        }
        count[i] = (uint32_t)n;
        sh.counts[b0 + i] = count[i];
        sh.sums[b0 + i] = n * (uint64_t)kOne - missing;
        weight[i] = n ? (double)sh.sums[b0 + i] * (1.0 / kOne) * s.edge(b0 + i, t) : 0.0;
        counts += count[i];
        weights += weight[i];
    }
    const uint32_t cbefore = scan(counts, sh.part_c, all);
    const double wbefore = scan(weights, sh.part_d, total);

    // The place of a border: the bin with the first token that has `c` tokens and
    // `w` of the weights up to and with it; then within the bin.
    struct Border {
        double weight;      // up to the token and with it
        Found f;
        int bin;
    };
    // where the kept tokens end; nothing is looked for past it
    Border cap{total, {}, kBins};
    auto border = [&](uint32_t c, double w, bool past) -> Border {
        __syncthreads();
        uint32_t cs = cbefore;
        double ws = wbefore;
        int mine = -1, last = -1;
        uint32_t cmine = 0;
        double wmine = 0;
#pragma unroll
        for (int i = 0; i < per; ++i) {
            if (count[i]) {
                const bool reached = cs + count[i] >= c && (past ? ws + weight[i] > w : ws + weight[i] >= w);
                if (reached && mine < 0)
                    mine = b0 + i, cmine = cs, wmine = ws;
                last = b0 + i;
            }
            cs += count[i];
            ws += weight[i];
        }
        // the first such bin; next to the end of all weights roundings may leave none, then the last one
        int hit = mine >= 0 ? mine : 0x7FFFFFFF;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            hit = min(hit, __shfl_xor(hit, o)), last = max(last, __shfl_xor(last, o));
        if ((threadIdx.x & 63) == 0)
            sh.part_c[threadIdx.x >> 6] = (uint32_t)hit, sh.part_u[threadIdx.x >> 6] = (unsigned long long)(last + 1);
        __syncthreads();
        for (int i = 0; i < kThreads / 64; ++i)
            hit = min(hit, (int)sh.part_c[i]), last = max(last, (int)sh.part_u[i] - 1);
        const bool none = hit == 0x7FFFFFFF;
        if (none)
            hit = last;
        if (hit > cap.bin)
            return cap;
        if (hit / per == (int)threadIdx.x) {
            if (hit != mine) {
                cmine = cbefore, wmine = wbefore;
                for (int i = 0; i < hit % per; ++i)
                    cmine += count[i], wmine += weight[i];
            }
            sh.n = cmine;
            sh.before = wmine;
        }
        __syncthreads();
        const uint32_t before = sh.n;
        const double wb = sh.before, edge = s.edge(hit, t);
        __syncthreads();
        // whole units of the bin's weight that the token has to reach
        double units = (w - wb) / edge * kOne;
        units = past ? floor(units) + 1.0 : ceil(units);
        Query q;
        q.count = c > before ? c - before : 0;
        // of what is there, and of what the limits keep
        q.weight = units > 0 ? min((uint64_t)units, hit == cap.bin ? cap.f.weight : sh.sums[hit]) : 0;
        if (q.count == 0 && q.weight == 0)
            q.count = 1;
        const Found f = d.find(hit, sh.counts[hit], q);
        return {wb + (double)f.weight * (1.0 / kOne) * edge, f, hit};
    };

    auto keep = [&](const Border &e) {
        if (e.bin < cap.bin || (e.bin == cap.bin && e.f.weight < cap.f.weight))
            cap = e;
    };
    const int32_t k = a.top_k ? a.top_k[row] : a.top_k_all;
    if (k > 0 && (uint32_t)k < all)
        keep(border((uint32_t)k, -1.0, false));
    const float p = a.top_p ? a.top_p[row] : a.top_p_all;
    if (p < 1.0f)
        keep(border(1, p > 0.0f ? (double)p * cap.weight : 0.0, false));
    const float least = a.min_p ? a.min_p[row] : a.min_p_all;
    if (least > 0.0f) {
        // how many tokens weigh at least min_p (one at most: the first token stays)
        const double floor_p = fmin((double)least, 1.0);
        uint32_t mine = 0, n;
        for (int at = threadIdx.x * 8; at < a.vocab; at += kThreads * 8) {
            float l[8];
            load8(d.row + at, min(a.vocab - at, 8), l);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                double below;
                if (s.bin(l[i], below) < kBins)
                    mine += s.drawn_max || s.flat || exp(((double)l[i] - (double)top) / t) >= floor_p ? 1 : 0;
            }
        }
        scan(mine, sh.part_c, n);
        if (n < all)
            keep(border(n, -1.0, false));
    }
    // below the kept sum whatever u
    const double kept = cap.weight;
    const float u = a.u[row];
    double target = u > 0.0f ? (double)u * kept : 0.0;
    if (!(target < kept))
        target = kept * (1.0 - 0x1p-52);
    const Found f = border(1, target, true).f;
    if (threadIdx.x == 0) {
        a.tokens[row] = f.token;
        if (a.logprobs) {
            const double z = s.drawn_max || s.flat ? 0.0 : ((double)logit_of(f.key) - (double)top) / t;
            a.logprobs[row] = (float)(z - log(kept));
        }
    }
}

// Logits a workgroup takes: as many as leave two workgroups a CU, at most 65536.
int groups(int64_t m, int64_t vocab)
{
    int g = 8;
    while (g > 1 && m * ((vocab + g * 8 * kThreads - 1) / (g * 8 * kThreads)) < 512)
        g /= 2;
    return g;
}

template <typename T>
void start(const SampleArgs &a, Part *parts, hipStream_t s)
{
    const int g = groups(a.m, a.vocab);
    const int splits = (a.vocab + g * 8 * kThreads - 1) / (g * 8 * kThreads);
    const dim3 grid((unsigned)(a.m * splits));
    switch (g) {
    case 8: sample_bins<8, T><<<grid, kThreads, 0, s>>>(a, parts, splits); break;
    case 4: sample_bins<4, T><<<grid, kThreads, 0, s>>>(a, parts, splits); break;
    case 2: sample_bins<2, T><<<grid, kThreads, 0, s>>>(a, parts, splits); break;
    default: sample_bins<1, T><<<grid, kThreads, 0, s>>>(a, parts, splits); break;
    }
    sample_draw<T><<<(unsigned)a.m, kThreads, 0, s>>>(a, parts, splits);
}

}  // namespace

size_t sample_workspace_bytes(int64_t m, int64_t vocab)
{
    const int64_t chunk = (int64_t)groups(m, vocab) * 8 * kThreads;
    return (size_t)(m * ((vocab + chunk - 1) / chunk)) * sizeof(Part);
}

hipError_t launch_sample(const SampleArgs &a, void *workspace, hipStream_t s)
{
    Part *parts = static_cast<Part *>(workspace);
    if (a.f32)
        start<float>(a, parts, s);
    else
        start<uint16_t>(a, parts, s);
    return hipGetLastError();
}

}  // namespace bd
