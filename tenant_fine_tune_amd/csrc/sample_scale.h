// The bins of a row's logits (sample.hip): which bin a logit is in, what a bin holds and
// weighs, and about where a token stands in it.  Plain arithmetic, which the host
// checks too.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace bd {
namespace {

constexpr int kBins = 2048;
constexpr int kCountShift = 47;              // of a packed bin: below it the excess of a part's tokens (32768 at most), each below 2^32
constexpr uint64_t kExcess = (1ull << kCountShift) - 1;
constexpr double kOne = 0x1p36;              // weight of a token at its bin's lower edge

// Numbers that order as the logits do (the zeros alike), and back.
__host__ __device__ __forceinline__ uint32_t key_of(float l)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__host__ __device__ __forceinline__ float logit_of(uint32_t k)
{
    return __builtin_bit_cast(float, k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
// Whether l's number is one of lo .. hi.  Compared as logits the zeros would be in the
// range below theirs too, whose last number stands for the negative zero.
__host__ __device__ __forceinline__ bool within(float l, uint32_t lo, uint32_t hi)
{
    return key_of(l) - lo <= hi - lo;
}

// How many ranges n ranges of candidates are read as.  Each costs a comparison with every
// logit, a token read in vain some more: one where few lie between, as long as all
// that it holds find room.
__host__ __device__ __forceinline__ int ranges_read(int n, uint32_t listed, uint32_t in_one, int32_t vocab, uint32_t room)
{
    return n > 1 && in_one - listed <= (uint32_t)vocab / 64 && in_one <= room ? 1 : n;
}

// The bins of a row, counted downwards from the one of its largest logit.
struct Scale {
    double c1, c2, c3, c4;       // excess(f) = f (c1 + f (c2 + f (c3 + f c4))), f = place in the bin
    double t;
    float top, top_bin;          // largest logit, floor(top / d)
    int shift;                   // d = 2^-shift
    bool alone;                  // only tokens at `top` have a weight (top = +inf, or so far above T that its neighbours have none)
    bool flat;                   // T = +inf: every token has weight one

    __host__ __device__ __forceinline__ void set(float temperature, float largest)
    {
        top = largest;
        t = temperature;
        flat = temperature == INFINITY;
        int e;
        frexp(t, &e);                             // T in [2^(e-1), 2^e)
        shift = flat ? -2000 : 6 - e;             // d = 2^(e-6): T / 64 < d <= T / 32
        // from 2^36 d on the next smaller logits are 2048 bins away
        alone = largest == INFINITY || fabs(ldexp((double)largest, shift)) >= 0x1p36;
        top_bin = floorf(ldexpf(largest, shift));
        // exp(x) - 1 for 0 <= x <= 1/32, as x times a polynomial through its four Chebyshev points: within 2^-38
        const double w = flat ? 0.0 : ldexp(1.0, -shift) / t;
        c1 = w * 0x1.ffffffff76092p-1 * kOne;
        c2 = w * w * 0x1.00000227c482ap-1 * kOne;
        c3 = w * w * w * 0x1.554ff31ff6e04p-3 * kOne;
        c4 = w * w * w * w * 0x1.59a176b303773p-5 * kOne;
    }
    // Bin of l as a number, at least kBins or NaN where it has none (l NaN or -inf).
    __host__ __device__ __forceinline__ float bin(float l) const
    {
        if (alone)
            return l == top ? 0.0f : INFINITY;
        return top_bin - floorf(ldexpf(l, shift));
    }
    // The excess of the logit a / to_bin in the low 47 bits of a double, and a count
    // of one above it: the sum 2^52 + 2^47 + excess is whole, so its bits are those
    // numbers under the exponent's.
    __device__ __forceinline__ uint64_t raw_excess(float a) const
    {
        const double f = __builtin_amdgcn_fract((double)a);
        return (uint64_t)__double_as_longlong(fma(f, fma(f, fma(f, fma(f, c4, c3), c2), c1), 0x1p52 + 0x1p47));
    }
    __device__ __forceinline__ uint64_t weight(float l) const
    {
        return (uint64_t)kOne + (alone ? 0 : raw_excess(ldexpf(l, shift)) & kExcess);
    }
    // lower edge of a bin, as a logit, and its weight relative to the largest logit
    __host__ __device__ __forceinline__ double edge(int b) const { return ldexp((double)top_bin - b, -shift); }
    __host__ __device__ __forceinline__ double edge_weight(int b) const
    {
        return alone || flat ? 1.0 : exp((edge(b) - (double)top) / t);
    }
    // Logits between which the bins' lo .. hi lie; bin() says of those at an end in which they are.
    __host__ __device__ __forceinline__ void span(int lo, int hi, float &from, float &to) const
    {
        if (alone) {
            from = to = top;
            return;
        }
        from = -__FLT_MAX__;
        to = top;
        if (flat)
            return;
        // the first logit from the lower edge on, the last one in front of the upper one
        const double e0 = edge(hi), e1 = edge(lo - 1);
        const float f0 = (float)e0, f1 = (float)e1;
        from = fmaxf((double)f0 < e0 ? logit_of(key_of(f0) + 1) : f0, from);
        // negative logits that scale to less than half the smallest number are in the bin from zero on
        if (e0 == 0.0)
            from = -ldexpf(1.0f, -150 - shift);
        if (lo > 0)
            to = fminf((double)f1 >= e1 ? logit_of(key_of(f1) - (f1 == 0.0f ? 2 : 1)) : f1, to);     // in front of zero: its negative is none
    }
    // About where a token of a bin that holds `held` stands among those, in their order: a
    // guess that puts none in front of one that comes before it.  Equal logits of 16
    // bits, of which a bin holds few different ones, are spread by their index over the
    // step below the next larger logit, which is half as far from a negative power of
    // two as its exponent says; of one weight for all (flat) the bin says nothing of a
    // logit's place.
    __host__ __device__ __forceinline__ uint32_t guess(float l, bool sixteen_bits, uint32_t index, int32_t vocab, uint32_t held) const
    {
        const uint32_t bits = __builtin_bit_cast(uint32_t, l);
        const int step = (int)(bits >> 23 & 255) - 134 + shift - (l < 0.0f && (bits & 0x7FFFFFu) == 0 ? 1 : 0);
        const float in_bin = ldexpf(l, shift);
        const float u = flat ? 0.0f : alone ? 1.0f : sixteen_bits ? fminf(ldexpf(1.0f, step), 1.0f) : 0.0f;
        const float f = flat ? 1.0f : alone ? 0.0f : fminf(in_bin - floorf(in_bin), 0x1.fffffep-1f);
        const float below = 1.0f - f - u + u * (float)index / (float)vocab;
        const uint32_t at = (uint32_t)(fmaxf(below, 0.0f) * (float)held);
        return at < held - 1 ? at : held - 1;
    }
};

}  // namespace
}  // namespace bd
