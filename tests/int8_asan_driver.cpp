// The entries of bitdelta_int8.h and bitdelta_sample.h under AddressSanitizer and
// UndefinedBehaviorSanitizer: checks with bad pointers, alignments, enums and
// shapes, the workspace queries over the edges of their ranges, and, where no GPU
// is visible, valid calls that plan their launches and fail there.  Nothing here
// dereferences a device pointer.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "bitdelta_int8.h"
#include "bitdelta_sample.h"

static int failures = 0;
#define EXPECT(call, want)                                                                                  \
    do {                                                                                                    \
        const int got__ = (int)(call);                                                                      \
        if (got__ != (int)(want)) {                                                                         \
            fprintf(stderr, "line %d: %s returned %d, expected %d (%s)\n", __LINE__, #call, got__, (int)(want), \
                    bitdelta_last_error());                                                                 \
            ++failures;                                                                                     \
        }                                                                                                   \
    } while (0)

int main()
{
    void *P = reinterpret_cast<void *>(uintptr_t(4096));
    float *F = static_cast<float *>(P);
    int8_t *Q = static_cast<int8_t *>(P);
    uint8_t *B = static_cast<uint8_t *>(P);
    int32_t *I = static_cast<int32_t *>(P);
    int devices = 0;
    const bool gpu = hipGetDeviceCount(&devices) == hipSuccess && devices > 0;
    const int64_t edges[] = {INT64_MIN, -1, 0, 1, 7, 8, 16, 17, 32, 33, 64, 65, 100, 128, 129, 1000, 4096, 16384, 28672, 131064,
                             131072, 1 << 20, 1 << 24, 1 << 26, (1 << 26) + 1, INT_MAX, (int64_t)INT_MAX + 1, INT64_MAX};

    // quantize_int8
    for (int64_t m : edges)
        for (int64_t d : edges) {
            const bool good = m >= 0 && m <= INT_MAX && d >= 1 && d <= BD_INT8_MAX_WIDTH;
            if (good && (gpu || (m > 0 && m * d > (int64_t)1 << 40)))
                continue;
            const int got = bitdelta_quantize_int8(P, d, BD_BF16, m, d, Q, F, nullptr);
            if (!good)
                EXPECT(got, BD_ESHAPE);
            else if (m == 0)
                EXPECT(got, BD_OK);
            else if (got == BD_OK)
                EXPECT(got, -1);
        }

    // linear_int8: the query, and calls of its size
    for (int64_t m : edges)
        for (int64_t n : edges)
            for (int64_t k : edges)
                for (int v : {INT_MIN, -1, 0, 1, 14, 4096, 4097, INT_MAX}) {
                    const size_t need = bitdelta_linear_int8_workspace(m, v, n, k);
                    const bool deltas = v > 0;
                    for (int ids = 0; ids < (deltas ? 2 : 1); ++ids) {
                        if (gpu && m != 0)
                            continue;
                        const int got = bitdelta_linear_int8(Q, F, m, Q, F, deltas ? B + 1 : nullptr, deltas ? F : nullptr,
                                                             BD_ALPHA_ROW, ids ? I : nullptr, v, n, k, P, BD_BF16, P, need,
                                                             nullptr);
                        if (got == BD_OK && m != 0)
                            EXPECT(got, -1);
                        // whole dwords of signs: the tiles' plan too
                        if (deltas && got != BD_EINVAL && got != BD_ESHAPE)
                            EXPECT(bitdelta_linear_int8(Q, F, m, Q, F, B, F, BD_ALPHA_ROW, ids ? I : nullptr, v, n, k, P,
                                                        BD_BF16, P, need, nullptr), got);
                    }
                }

    // sample
    for (int64_t m : edges)
        for (int64_t vocab : edges) {
            const size_t need = bitdelta_sample_workspace(m, vocab);
            const bool good = m >= 0 && m <= BD_SAMPLE_MAX_ROWS && vocab >= 1 && vocab <= BD_SAMPLE_MAX_VOCAB;
            if (!good || m == 0)
                EXPECT(need, 0);
            if (good && m > 0 && gpu)
                continue;
            const int got = bitdelta_sample(P, vocab, BD_F32, m, vocab, F, nullptr, 1.0f, nullptr, 0, F, 1.0f, nullptr, 0.0f, I,
                                            F, P, need, nullptr);
            if (!good)
                EXPECT(got, BD_ESHAPE);
            else if (m == 0)
                EXPECT(got, BD_OK);
            else if (got == BD_OK)
                EXPECT(got, -1);
        }
    printf("int8 driver: %d failures\n", failures);
    return failures != 0;
}
