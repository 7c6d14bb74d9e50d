// The entries of bitdelta_decoder.h under AddressSanitizer and
// UndefinedBehaviorSanitizer: every check with bad pointers, alignments, enums,
// shapes and workspaces, the workspace query over the edges of its ranges, and,
// where no GPU is visible, valid calls that plan their launch and fail there.
// Nothing here dereferences a device pointer.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "bitdelta_decoder.h"

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
    uint16_t *F = reinterpret_cast<uint16_t *>(uintptr_t(4096)), *G = reinterpret_cast<uint16_t *>(uintptr_t(8192));
    uint16_t *ODD = reinterpret_cast<uint16_t *>(uintptr_t(4098));
    int32_t *I = reinterpret_cast<int32_t *>(F);
    double *D = reinterpret_cast<double *>(F);
    int devices = 0;
    const bool gpu = hipGetDeviceCount(&devices) == hipSuccess && devices > 0;
    const int64_t big = (int64_t)1 << 40;

    // block_norm
    const auto norm = [&](int64_t m, int64_t d, int64_t stride, const uint16_t *res, const uint16_t *blk, uint16_t *out,
                          uint16_t *x, float eps, int rt = 0, int wt = 0, int act = 1, int nv = 3) {
        return bitdelta_block_norm(res, stride, rt, blk, stride, blk, stride, act, 1.0f, blk, F, wt, I, nv, m, d, eps, out,
                                   stride, x, nullptr);
    };
    EXPECT(norm(0, 8, 8, nullptr, F, G, G, 1e-6f), BD_OK);
    for (int64_t m : {(int64_t)-1, (int64_t)INT_MAX + 1, big, INT64_MIN, INT64_MAX})
        EXPECT(norm(m, 8, 8, F, F, G, G, 1e-6f), BD_ESHAPE);
    for (int64_t d : {(int64_t)0, (int64_t)-1, (int64_t)BD_NORM_MAX_WIDTH + 1, INT64_MIN, INT64_MAX})
        EXPECT(norm(4, d, big, F, F, G, G, 1e-6f), BD_ESHAPE);
    for (int64_t stride : {(int64_t)7, (int64_t)0, (int64_t)-8, big + 1, INT64_MAX, INT64_MIN})
        EXPECT(norm(4, 8, stride, F, F, G, G, 1e-6f), BD_ESHAPE);
    for (float eps : {-1.0f, (float)NAN, -INFINITY})
        EXPECT(norm(4, 8, 8, F, F, G, G, eps), BD_EINVAL);
    for (int v : {-1, 2, INT_MAX, INT_MIN}) {
        EXPECT(norm(4, 8, 8, F, F, G, G, 1e-6f, v), BD_EINVAL);
        EXPECT(norm(4, 8, 8, F, F, G, G, 1e-6f, 0, v), BD_EINVAL);
        EXPECT(norm(4, 8, 8, F, F, G, G, 1e-6f, 0, 0, v < 0 ? v : v + (v == 2)), BD_EINVAL);
    }
    EXPECT(norm(4, 8, 8, F, F, G, G, 1e-6f, 0, 0, 1, 0), BD_EINVAL);
    EXPECT(norm(4, 8, 8, nullptr, F, G, G, 1e-6f), BD_EINVAL);
    EXPECT(norm(4, 8, 8, F, F, G, nullptr, 1e-6f), BD_EINVAL);
    EXPECT(norm(4, 8, 8, ODD, F, G, G, 1e-6f, 1), BD_EALIGN);
    EXPECT(norm(4, 8, 8, F, ODD, G, G, 1e-6f, 0, 1), BD_EALIGN);
    if (!gpu)
        for (int64_t m : {(int64_t)1, (int64_t)1 << 20, ((int64_t)1 << 20) + 1, (int64_t)INT_MAX})
            for (int64_t d : {1, 2048, 2049, 16384, 16385, BD_NORM_MAX_WIDTH})
                EXPECT(norm(m, d, d, F, F, G, G, 1e-6f), BD_EDEVICE);

    // the cache and the batch of both other entries
    bd_kv_cache c = {F, F, nullptr, nullptr, 0, 9, 2, 16, 128};
    bd_batch b = {I, I, I, I, I, I, 4, 2, 3, 1, 2, 0};
    const auto append = [&](const bd_kv_cache &kc, const bd_batch &kb, int heads = 8, int rotary = 128, int inter = 0) {
        const int64_t q = (int64_t)heads * kc.head_dim, k = (int64_t)kc.n_kv_heads * kc.head_dim;
        return bitdelta_kv_append(F, q, F, k, F, k, heads, D, rotary, inter, &kc, &kb, G, nullptr);
    };
    const auto attend = [&](const bd_kv_cache &kc, const bd_batch &kb, int heads = 8, float scale = 0.1f, size_t ws = SIZE_MAX) {
        return bitdelta_attention(F, (int64_t)heads * kc.head_dim, heads, scale, &kc, &kb, G, F, ws, nullptr);
    };
    EXPECT(bitdelta_kv_append(F, 8, F, 8, F, 8, 8, D, 16, 0, nullptr, &b, G, nullptr), BD_EINVAL);
    EXPECT(bitdelta_attention(F, 8, 8, 0.1f, &c, nullptr, G, F, 0, nullptr), BD_EINVAL);
    EXPECT(bitdelta_attention_workspace(8, nullptr, &b) != 0, 0);
    EXPECT(bitdelta_attention_workspace(8, &c, nullptr) != 0, 0);
    const int32_t ints[] = {INT_MIN, -1, 0, 1, 2, 3, 16, 64, 128, 1024, 1025, 4096, 4097, INT_MAX};
    for (int32_t v : ints) {
        bd_kv_cache k = c;
        for (int32_t *f : {&k.dtype, &k.n_pages, &k.n_kv_heads, &k.page_size, &k.head_dim}) {
            const int32_t kept = *f;
            *f = v;
            (void)bitdelta_attention_workspace(8, &k, &b);
            const int heads = k.n_kv_heads > 0 && k.n_kv_heads <= 1024 ? k.n_kv_heads : 8;
            const bd_status s = gpu ? BD_ESHAPE : append(k, b, heads, 0);
            if (s != BD_EINVAL && s != BD_ESHAPE && s != BD_EDEVICE) {
                fprintf(stderr, "line %d: %d (%s)\n", __LINE__, (int)s, bitdelta_last_error());
                ++failures;
            }
            *f = kept;
        }
        bd_batch w = b;
        for (int32_t *f : {&w.n_seqs, &w.max_pages, &w.n_groups, &w.max_prefix_pages, &w.max_new}) {
            const int32_t kept = *f;
            *f = v;
            for (int64_t T : {(int64_t)1, (int64_t)65, (int64_t)2049, (int64_t)INT_MAX / 8}) {
                w.n_tokens = T;
                const size_t need = bitdelta_attention_workspace(8, &c, &w);
                const bd_status s = gpu ? BD_OK : attend(c, w);
                if (!gpu && s != BD_ESHAPE && s != BD_EDEVICE) {
                    fprintf(stderr, "line %d: %d (%s)\n", __LINE__, (int)s, bitdelta_last_error());
                    ++failures;
                }
                if (s == BD_EDEVICE && need)
                    EXPECT(attend(c, w, 8, 0.1f, need - 1), BD_EWORKSPACE);
            }
            *f = kept;
        }
        (void)bitdelta_attention_workspace(v, &c, &b);
        if (v < 1 || v > 1024 || v % 2)
            EXPECT(attend(c, b, v), BD_ESHAPE);
        if (v < 0 || v > 128 || v % 16) {
            EXPECT(append(c, b, 8, v), BD_ESHAPE);
        }
        if (v != 0 && v != 1)
            EXPECT(append(c, b, 8, 16, v), BD_EINVAL);
    }
    for (int64_t T : {(int64_t)-1, (int64_t)INT_MAX + 1, big, INT64_MIN, INT64_MAX}) {
        bd_batch w = b;
        w.n_tokens = T;
        EXPECT(append(c, w), BD_ESHAPE);
        EXPECT(attend(c, w), BD_ESHAPE);
        EXPECT(bitdelta_attention_workspace(8, &c, &w) != 0, 0);
    }
    for (int heads : {16, 1024}) {       // queries of 2^31 heads and more
        bd_batch w = b;
        w.n_tokens = INT_MAX / heads + 1;
        EXPECT(attend(c, w, heads), BD_ESHAPE);
    }
    for (float s : {0.0f, -1.0f, (float)NAN, INFINITY})
        EXPECT(attend(c, b, 8, s), BD_EINVAL);
    printf("decoder driver: %d failures\n", failures);
    return failures ? 1 : 0;
}
