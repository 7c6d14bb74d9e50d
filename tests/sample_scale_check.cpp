// Walks the arithmetic of sample_scale.h on the host over all 16-bit logits and many
// of 32 bits, at temperatures from the smallest number to infinity.
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#include "../tenant_fine_tune_amd/csrc/sample_scale.h"

using namespace bd;

static int failures = 0;
#define EXPECT(c, ...)                                    \
    do {                                                  \
        if (!(c) && failures++ < 20) {                    \
            fprintf(stderr, "line %d: %s: ", __LINE__, #c); \
            fprintf(stderr, __VA_ARGS__);                 \
            fprintf(stderr, "\n");                        \
        }                                                 \
    } while (0)

static const float kTemperatures[] = {0x1p-149f, 1e-40f, 1e-30f, 1e-3f, 0.05f, 0.2f, 0.5f, 0.7f, 0.75f, 1.0f, 1.2f, 1.5f, 2.0f,
                                      4.0f, 30.0f, 63.9f, 64.0f, 100.0f, 128.0f, 1e4f, 1e10f, 1e20f, 1e30f, 3e38f, INFINITY};

// Every finite bf16 number, from the smallest on.
static std::vector<float> bf16_numbers()
{
    std::vector<float> v;
    for (uint32_t h = 0xFF7F; h > 0x8000; --h)      // the zeros have one key
        v.push_back(__builtin_bit_cast(float, h << 16));
    for (uint32_t h = 0; h <= 0x7F7F; ++h)
        v.push_back(__builtin_bit_cast(float, h << 16));
    return v;
}

// Numbers of 32 bits: single steps around powers of two and their multiples, and random ones.
static std::vector<float> f32_numbers()
{
    std::mt19937 r(1);
    std::vector<uint32_t> keys;
    for (int e = -149; e <= 127; ++e)
        for (float m : {1.0f, 1.5f, 1.25f, 1.984375f})
            for (float s : {-1.0f, 1.0f}) {
                const float l = s * ldexpf(m, e);
                if (l == 0.0f || !(fabsf(l) <= __FLT_MAX__))
                    continue;
                for (int d = -2; d <= 2; ++d)
                    keys.push_back(key_of(l) + d);
            }
    for (int i = 0; i < 20000; ++i)
        keys.push_back(r());
    for (int d = -4; d <= 4; ++d)
        keys.push_back(key_of(0.0f) + d);
    std::vector<float> v;
    for (uint32_t k : keys) {
        const float l = logit_of(k);
        if (fabsf(l) <= __FLT_MAX__)
            v.push_back(l);
    }
    std::sort(v.begin(), v.end());
    return v;
}

// A token's guessed place is never in front of that of one before it in the order:
// of a larger logit, or of an equal one with a lower index.
static void check_guesses(const std::vector<float> &v, bool sixteen)
{
    for (float t : kTemperatures) {
        Scale s;
        for (size_t i = 0; i + 1 < v.size(); ++i) {
            // bins lie at multiples of their width, whatever the largest logit is
            s.set(t, v[i + 1]);
            if (s.bin(v[i]) != s.bin(v[i + 1]) || s.alone)
                continue;
            for (int32_t vocab : {2, 50257, 131071, 1048576})
                for (uint32_t held : {2u, 3u, 129u, 582u, 4096u}) {
                    const uint32_t upper = s.guess(v[i + 1], sixteen, vocab - 1, vocab, held), lower = s.guess(v[i], sixteen, 0, vocab, held);
                    EXPECT(upper <= lower, "T=%g: %.9g at %u, %.9g at %u of %u", t, v[i + 1], upper, v[i], lower, held);
                    EXPECT(s.guess(v[i], sixteen, vocab / 2, vocab, held) >= lower, "T=%g: %.9g", t, v[i]);
                    EXPECT(s.guess(v[i], sixteen, vocab - 1, vocab, held) < held, "T=%g: %.9g", t, v[i]);
                }
        }
    }
}

// Every logit that is counted in a bin is among those that the bin's span names, as
// that of a range of bins too.
static void check_spans(const std::vector<float> &v)
{
    for (float t : kTemperatures) {
        Scale s;
        for (size_t i = 0; i < v.size(); ++i)
            for (size_t above : {(size_t)0, (size_t)1, (size_t)7, v.size() / 100, v.size() / 2}) {
                s.set(t, v[std::min(i + above, v.size() - 1)]);
                const float b = s.bin(v[i]);
                if (!(b < kBins))
                    continue;
                EXPECT(b >= 0, "T=%g: %.9g, largest %.9g: bin %g", t, v[i], s.top, b);
                for (int lo : {0, 1, 0x10000})
                    for (int hi : {0, 3}) {
                        float from, to;
                        s.span(std::max((int)b - lo, 0), std::min((int)b + hi, kBins - 1), from, to);
                        EXPECT(v[i] >= from && v[i] <= to, "T=%g: %.9g, largest %.9g: bin %g holds %.9g to %.9g", t, v[i], s.top, b, from, to);
                    }
            }
    }
}

// Of two neighbouring ranges of keys a logit is in one, wherever they meet.
static void check_ranges(const std::vector<float> &v)
{
    for (size_t i = 0; i < v.size(); ++i) {
        const uint32_t key = key_of(v[i]);
        EXPECT(logit_of(key) == v[i], "%.9g", v[i]);
        for (uint32_t meet : {key - 3, key - 1, key, key + 1, 0x7FFFFFFEu, 0x7FFFFFFFu, 0x80000000u})
            EXPECT(within(v[i], key_of(-__FLT_MAX__), meet) != within(v[i], meet + 1, key_of(INFINITY)), "%.9g, ranges meet at %08x", v[i], meet);
    }
}

// Ranges read as one find room, as they do one by one.
static void check_reading()
{
    for (uint32_t room : {5120u, 8192u})
        for (int32_t vocab : {2, 1000, 131071, 262144, 300000, 1048576})
            for (uint32_t listed : {2u, 100u, room / 2})
                for (uint32_t between : {0u, 100u, (uint32_t)vocab / 64, (uint32_t)vocab / 64 + 1, room / 2, room / 2 + 1, room})
                    for (int n : {1, 2, 4}) {
                        const int r = ranges_read(n, listed, listed + between, vocab, room);
                        EXPECT(r == n || (r == 1 && listed + between <= room), "%d ranges, %u and %u between, %d logits", n, listed, between, vocab);
                        EXPECT(n == 1 || between > 100 || vocab < 6400 || r == 1, "%d ranges, %u between, %d logits", n, between, vocab);
                    }
}

// The bin that ends at zero does not name the zeros, of which a row may have any number.
static void check_below_zero()
{
    for (float t : kTemperatures) {
        Scale s;
        s.set(t, 3.0f * t);
        if (s.alone || s.flat)
            continue;
        const int below = (int)s.bin(0.0f) + 1;
        float from, to;
        s.span(below, below, from, to);
        EXPECT(to < 0.0f && (from < 0.0f || t < 1e-44f), "T=%g: bin %d holds %.9g to %.9g", t, below, from, to);
    }
}

int main()
{
    check_guesses(bf16_numbers(), true);
    check_guesses(f32_numbers(), false);
    check_spans(bf16_numbers());
    check_spans(f32_numbers());
    check_ranges(f32_numbers());
    check_reading();
    check_below_zero();
    printf("sample scale: %d failures\n", failures);
    return failures != 0;
}
