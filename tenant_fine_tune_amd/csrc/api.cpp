// C ABI of the BitDelta library (declared in include/bitdelta.h).
//
// Every argument is checked on the host before anything is launched; a bad
// argument returns a status and launches nothing, so the checks are testable
// on a machine without a GPU.  No call allocates device memory.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <limits>

#include "../../include/bitdelta.h"
#include "bd_launch.h"
#include "decoder_launch.h"

namespace {

thread_local char g_err[512] = "";

bd_status fail(bd_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
bd_status fail(bd_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

bd_status device(hipError_t e, const char *what)
{
    if (e == hipSuccess)
        return BD_OK;
    return fail(BD_EDEVICE, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxGrid = std::numeric_limits<int32_t>::max();
// Workgroups of `threads` of one launch: from 2^32 threads on it wraps around
// without an error.
constexpr int64_t max_workgroups(int64_t threads) { return std::numeric_limits<uint32_t>::max() / threads; }

bd_status check_matrix(int64_t d_out, int64_t d_in)
{
    if (d_out <= 0)
        return fail(BD_ESHAPE, "d_out must be positive (got %lld)", (long long)d_out);
    if (d_in <= 0 || d_in % 8 != 0)
        return fail(BD_ESHAPE, "d_in must be a positive multiple of 8 (got %lld)", (long long)d_in);
    if (d_out > kMaxGrid || d_in > (int64_t)1 << 40 || d_out > std::numeric_limits<int64_t>::max() / d_in)
        return fail(BD_ESHAPE, "matrix [%lld, %lld] too large", (long long)d_out, (long long)d_in);
    return BD_OK;
}

// The prefill kernels address x, W_base, signs and y through 32-bit buffer
// offsets: each operand (per variant for signs) must stay below 2 GiB.
bool operands_fit(int64_t m, int64_t d_out, int64_t d_in)
{
    // a * b * 2 < 2^31 for positive a, b, without forming the product
    const auto fits = [](int64_t a, int64_t b) { return a <= 0 || b <= 0 || a <= ((int64_t(1) << 30) - 1) / b; };
    return fits(m, d_in) && fits(d_out, d_in) && fits(m, d_out);
}

bd_status check_mode(int mode)
{
    if (mode != BD_ALPHA_ROW && mode != BD_ALPHA_MATRIX)
        return fail(BD_EINVAL, "alpha_mode must be BD_ALPHA_ROW (0) or BD_ALPHA_MATRIX (1), got %d", mode);
    return BD_OK;
}

#define BD_TRY(expr)                  \
    do {                              \
        bd_status s__ = (expr);       \
        if (s__ != BD_OK)             \
            return s__;               \
    } while (0)

#define BD_NONNULL(p)                                             \
    do {                                                          \
        if (!(p))                                                 \
            return fail(BD_EINVAL, "%s must not be NULL", #p);    \
    } while (0)

#define BD_ALIGNED(p, a)                                                        \
    do {                                                                        \
        if (!aligned((p), (a)))                                                 \
            return fail(BD_EALIGN, "%s must be %d-byte aligned", #p, (int)(a)); \
    } while (0)

}  // namespace

extern "C" {

int bitdelta_version(void) { return 100; }

const char *bitdelta_status_string(int s)
{
    switch (s) {
    case BD_OK: return "BD_OK";
    case BD_EINVAL: return "BD_EINVAL: invalid argument";
    case BD_ESHAPE: return "BD_ESHAPE: unsupported or invalid shape";
    case BD_EALIGN: return "BD_EALIGN: misaligned pointer";
    case BD_EWORKSPACE: return "BD_EWORKSPACE: workspace too small";
    case BD_EDEVICE: return "BD_EDEVICE: HIP launch failed";
    case BD_EBUSY: return "BD_EBUSY: no delta-cache slot can be freed";
    default: return "unknown bitdelta status";
    }
}

const char *bitdelta_last_error(void) { return g_err; }

size_t bitdelta_compress_workspace(int64_t d_out, int64_t d_in, int alpha_mode)
{
    (void)d_in;
    if (alpha_mode != BD_ALPHA_MATRIX || d_out <= 0)
        return 0;
    return sizeof(double) * (size_t)d_out;
}

bd_status bitdelta_compress(const bd_bf16 *w_base, const void *w_ft, int ft_dtype, int64_t d_out,
                            int64_t d_in, int alpha_mode, uint8_t *signs, float *alpha,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    BD_TRY(check_mode(alpha_mode));
    if (ft_dtype != BD_BF16 && ft_dtype != BD_F32)
        return fail(BD_EINVAL, "ft_dtype must be BD_BF16 (0) or BD_F32 (1), got %d", ft_dtype);
    BD_TRY(check_matrix(d_out, d_in));
    if (d_out > max_workgroups(256))
        return fail(BD_ESHAPE, "matrix [%lld, %lld] exceeds the compress grid", (long long)d_out, (long long)d_in);
    BD_NONNULL(w_base);
    BD_NONNULL(w_ft);
    BD_NONNULL(signs);
    BD_NONNULL(alpha);
    BD_ALIGNED(w_base, 16);
    BD_ALIGNED(w_ft, 16);
    BD_ALIGNED(alpha, 4);
    const bool per_matrix = alpha_mode == BD_ALPHA_MATRIX;
    const size_t need = bitdelta_compress_workspace(d_out, d_in, alpha_mode);
    if (workspace_bytes < need)
        return fail(BD_EWORKSPACE, "compress needs %zu workspace bytes, got %zu", need, workspace_bytes);
    if (need) {
        BD_NONNULL(workspace);
        BD_ALIGNED(workspace, 8);
    }
    return device(bd::launch_compress(w_base, w_ft, ft_dtype == BD_F32, d_out, d_in, per_matrix, signs,
                                      alpha, static_cast<double *>(workspace), (hipStream_t)stream),
                  "bitdelta_compress");
}

bd_status bitdelta_reconstruct(const bd_bf16 *w_base, const uint8_t *signs, const float *alpha,
                               int alpha_mode, int64_t d_out, int64_t d_in, bd_bf16 *w_eff,
                               void *stream)
{
    BD_TRY(check_mode(alpha_mode));
    BD_TRY(check_matrix(d_out, d_in));
    BD_NONNULL(w_base);
    BD_NONNULL(signs);
    BD_NONNULL(alpha);
    BD_NONNULL(w_eff);
    BD_ALIGNED(w_base, 16);
    BD_ALIGNED(w_eff, 16);
    BD_ALIGNED(alpha, 4);
    const int64_t bpr = (d_in / 8 + 255) / 256;
    if (bpr > max_workgroups(256) || d_out > max_workgroups(256) / bpr)
        return fail(BD_ESHAPE, "matrix [%lld, %lld] exceeds the reconstruct grid", (long long)d_out, (long long)d_in);
    return device(bd::launch_reconstruct(w_base, signs, alpha, alpha_mode == BD_ALPHA_MATRIX, d_out, d_in, w_eff,
                                         (hipStream_t)stream),
                  "bitdelta_reconstruct");
}

size_t bitdelta_linear_workspace(int64_t m, int64_t d_out, int64_t d_in)
{
    if (d_out <= 0 || d_in <= 0 || d_in % 8 != 0 || m < 1)
        return 0;
    // decode: only few rows of long width need one (split row steps); shapes
    // the decode path rejects need none
    if (m <= bd::kGemvMaxM)
        return (int64_t)bd::kGemvMaxM * d_in * 2 >= ((int64_t)1 << 31) ? 0 : bd::gemv_workspace_bytes((int)m, d_out, d_in);
    // shapes the prefill path rejects need no workspace
    if (!operands_fit(m, d_out, d_in))
        return 0;
    return bd::gemm_workspace_bytes(m, d_out, d_in);
}

bd_status bitdelta_linear(const bd_bf16 *x, int64_t m, const bd_bf16 *w_base, const uint8_t *signs,
                          const float *alpha, int alpha_mode, int64_t d_out, int64_t d_in, bd_bf16 *y,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    BD_TRY(check_mode(alpha_mode));
    BD_TRY(check_matrix(d_out, d_in));
    if (m < 0)
        return fail(BD_ESHAPE, "m must be >= 0 (got %lld)", (long long)m);
    const size_t need = bitdelta_linear_workspace(m, d_out, d_in);
    if (workspace_bytes < need)
        return fail(BD_EWORKSPACE, "linear needs %zu workspace bytes, got %zu", need, workspace_bytes);
    if (m == 0)
        return BD_OK;
    BD_NONNULL(x);
    BD_NONNULL(w_base);
    BD_NONNULL(signs);
    BD_NONNULL(alpha);
    BD_NONNULL(y);
    BD_ALIGNED(x, 16);
    BD_ALIGNED(w_base, 16);
    BD_ALIGNED(y, 16);
    BD_ALIGNED(alpha, 4);
    if (need) {
        BD_NONNULL(workspace);
        BD_ALIGNED(workspace, 16);
    }
    const bool per_matrix = alpha_mode == BD_ALPHA_MATRIX;
    hipStream_t s = (hipStream_t)stream;
    if (m <= bd::kGemvMaxM) {
        // The decode kernels address x and each launched chunk of W_base (at
        // least 16 rows) through 32-bit buffer offsets.
        if ((int64_t)bd::kGemvMaxM * d_in * 2 >= ((int64_t)1 << 31))
            return fail(BD_ESHAPE, "decode linear needs 16 rows of W_base below 2 GiB (d_in=%lld)", (long long)d_in);
        // (chunks of wider rows are below 2 GiB / 32 rows, at most 64 threads each)
        if (d_in < 16 && d_out > max_workgroups(64))
            return fail(BD_ESHAPE, "linear d_out=%lld of width %lld exceeds the decode grid", (long long)d_out,
                        (long long)d_in);
        return device(bd::launch_gemv(x, (int)m, w_base, signs, alpha, per_matrix, d_out, d_in, y, workspace, s),
                      "bitdelta_linear (decode)");
    }
    if (!operands_fit(m, d_out, d_in))
        return fail(BD_ESHAPE, "prefill operands must each be below 2 GiB (m=%lld, d_out=%lld, d_in=%lld)",
                    (long long)m, (long long)d_out, (long long)d_in);
    const int64_t tiles = ((m + bd::kGemmBM - 1) / bd::kGemmBM) * ((d_out + bd::kGemmBN - 1) / bd::kGemmBN);
    if (tiles > kMaxGrid)
        return fail(BD_ESHAPE, "linear m=%lld d_out=%lld exceeds the prefill grid", (long long)m, (long long)d_out);
    if (need >= ((size_t)1 << 31))
        return fail(BD_ESHAPE, "linear m=%lld d_out=%lld d_in=%lld needs a split-K workspace above 2 GiB",
                    (long long)m, (long long)d_out, (long long)d_in);
    return device(bd::launch_gemm(x, m, w_base, signs, alpha, per_matrix, d_out, d_in, y, workspace, s),
                  "bitdelta_linear (prefill)");
}

size_t bitdelta_linear_grouped_workspace(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in)
{
    (void)d_out;
    (void)d_in;
    if (m < 0 || m > std::numeric_limits<int32_t>::max() / 2 || n_variants <= 0 || n_variants > 4096)
        return 0;
    return bd::grouped_workspace_bytes(m, n_variants);
}

}  // extern "C"

namespace {

// Checks shared by the two grouped entry points (everything but the table's
// memory); BD_OK with *empty set for m = 0, a no-op.
bd_status check_grouped(const bd_bf16 *x, int64_t m, const int32_t *variant_ids, int32_t n_variants,
                        const bd_bf16 *w_base, const uint8_t *signs, const float *alpha, int alpha_mode,
                        int64_t d_out, int64_t d_in, bd_bf16 *y)
{
    BD_TRY(check_mode(alpha_mode));
    if (n_variants <= 0 || n_variants > 4096)
        return fail(BD_EINVAL, "n_variants must be in [1, 4096] (got %d)", n_variants);
    BD_TRY(check_matrix(d_out, d_in));
    if (m < 0)
        return fail(BD_ESHAPE, "m must be >= 0 (got %lld)", (long long)m);
    if (m > std::numeric_limits<int32_t>::max() / 2)
        return fail(BD_ESHAPE, "grouped m=%lld too large for int32 token indices", (long long)m);
    if (m == 0)
        return BD_OK;
    BD_NONNULL(x);
    BD_NONNULL(variant_ids);
    BD_NONNULL(w_base);
    BD_NONNULL(signs);
    BD_NONNULL(alpha);
    BD_NONNULL(y);
    BD_ALIGNED(x, 16);
    BD_ALIGNED(w_base, 16);
    BD_ALIGNED(y, 16);
    BD_ALIGNED(alpha, 4);
    BD_ALIGNED(variant_ids, 4);
    if (!operands_fit(m, d_out, d_in))
        return fail(BD_ESHAPE, "grouped operands must each be below 2 GiB (m=%lld, d_out=%lld, d_in=%lld)",
                    (long long)m, (long long)d_out, (long long)d_in);
    const int64_t tiles = bd::grouped_max_tiles(m, n_variants) * ((d_out + bd::kGemmBN - 1) / bd::kGemmBN);
    if (tiles > kMaxGrid)
        return fail(BD_ESHAPE, "grouped m=%lld d_out=%lld exceeds the grid", (long long)m, (long long)d_out);
    return BD_OK;
}

}  // namespace

extern "C" {

bd_status bitdelta_linear_grouped(const bd_bf16 *x, int64_t m, const int32_t *variant_ids, int32_t n_variants,
                                  const bd_bf16 *w_base, const uint8_t *signs, const float *alpha,
                                  int alpha_mode, int64_t d_out, int64_t d_in, bd_bf16 *y,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    BD_TRY(check_grouped(x, m, variant_ids, n_variants, w_base, signs, alpha, alpha_mode, d_out, d_in, y));
    const size_t need = bitdelta_linear_grouped_workspace(m, n_variants, d_out, d_in);
    if (workspace_bytes < need)
        return fail(BD_EWORKSPACE, "linear_grouped needs %zu workspace bytes, got %zu", need, workspace_bytes);
    if (m == 0)
        return BD_OK;
    BD_NONNULL(workspace);
    BD_ALIGNED(workspace, 16);
    return device(bd::launch_grouped(x, m, variant_ids, n_variants, w_base, signs, alpha,
                                     alpha_mode == BD_ALPHA_MATRIX, d_out, d_in, y,
                                     static_cast<int32_t *>(workspace), (hipStream_t)stream),
                  "bitdelta_linear_grouped");
}

bd_status bitdelta_linear_grouped_noalloc(const bd_bf16 *x, int64_t m, const int32_t *variant_ids,
                                          int32_t n_variants, const bd_bf16 *w_base, const uint8_t *signs,
                                          const float *alpha, int alpha_mode, int64_t d_out, int64_t d_in,
                                          bd_bf16 *y, void *stream)
{
    static_assert(BD_GROUPED_NOALLOC_MAX_TOKENS == bd::kGroupedNoallocMaxTokens, "token limit");
    BD_TRY(check_grouped(x, m, variant_ids, n_variants, w_base, signs, alpha, alpha_mode, d_out, d_in, y));
    if (m > BD_GROUPED_NOALLOC_MAX_TOKENS)
        return fail(BD_ESHAPE, "linear_grouped_noalloc takes at most %d tokens (got %lld)",
                    BD_GROUPED_NOALLOC_MAX_TOKENS, (long long)m);
    const size_t need = bitdelta_linear_grouped_workspace(m, n_variants, d_out, d_in);
    if (need > bd::grouped_scratch_bytes())
        return fail(BD_ESHAPE, "linear_grouped_noalloc needs %zu table bytes, the library holds %zu", need,
                    bd::grouped_scratch_bytes());
    if (m == 0)
        return BD_OK;
    int32_t *table = nullptr;
    BD_TRY(device(bd::grouped_scratch(&table), "bitdelta_linear_grouped_noalloc (table address)"));
    return device(bd::launch_grouped(x, m, variant_ids, n_variants, w_base, signs, alpha,
                                     alpha_mode == BD_ALPHA_MATRIX, d_out, d_in, y, table, (hipStream_t)stream),
                  "bitdelta_linear_grouped_noalloc");
}

size_t bitdelta_similarity_workspace(int32_t n_variants, int64_t d_out, int64_t d_in)
{
    (void)d_in;
    if (n_variants < 1 || n_variants > bd::kSimilarityMaxVariants)
        return 0;
    return bd::similarity_workspace_bytes(n_variants, d_out);
}

bd_status bitdelta_similarity(const uint8_t *signs, const float *alpha, int alpha_mode, int32_t n_variants,
                              int64_t d_out, int64_t d_in, double *gram, double *cosine, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    BD_TRY(check_mode(alpha_mode));
    if (n_variants < 1 || n_variants > bd::kSimilarityMaxVariants)
        return fail(BD_EINVAL, "n_variants must be in [1, %d] (got %d)", bd::kSimilarityMaxVariants, n_variants);
    BD_TRY(check_matrix(d_out, d_in));
    if (d_in % 32 != 0)
        return fail(BD_ESHAPE, "similarity needs d_in a multiple of 32 (got %lld)", (long long)d_in);
    if ((int64_t)n_variants * d_out * (d_in / 8) >= ((int64_t)1 << 31))
        return fail(BD_ESHAPE, "similarity sign tensor [%d, %lld, %lld] must be below 2 GiB", n_variants,
                    (long long)d_out, (long long)(d_in / 8));
    if ((int64_t)n_variants * (n_variants - 1) / 2 * d_out * 4 >= ((int64_t)1 << 31))
        return fail(BD_ESHAPE, "similarity of %d variants over %lld rows needs pair counts of 2 GiB or more",
                    n_variants, (long long)d_out);
    const size_t need = bitdelta_similarity_workspace(n_variants, d_out, d_in);
    if (workspace_bytes < need)
        return fail(BD_EWORKSPACE, "similarity needs %zu workspace bytes, got %zu", need, workspace_bytes);
    BD_NONNULL(signs);
    BD_NONNULL(alpha);
    BD_NONNULL(gram);
    BD_NONNULL(cosine);
    BD_ALIGNED(signs, 4);
    BD_ALIGNED(alpha, 4);
    BD_ALIGNED(gram, 8);
    BD_ALIGNED(cosine, 8);
    if (need) {
        BD_NONNULL(workspace);
        BD_ALIGNED(workspace, 4);
    }
    return device(bd::launch_similarity(signs, alpha, alpha_mode == BD_ALPHA_MATRIX, n_variants, d_out, d_in, gram,
                                        cosine, static_cast<int32_t *>(workspace), (hipStream_t)stream),
                  "bitdelta_similarity");
}

size_t bitdelta_similarity_delta_workspace(int32_t n_variants, int64_t d_out, int64_t d_in)
{
    (void)d_in;
    if (n_variants < 1 || n_variants > bd::kSimilarityMaxVariants)
        return 0;
    return bd::similarity_delta_workspace_bytes(n_variants, d_out);
}

bd_status bitdelta_similarity_delta(const bd_bf16 *w_base, const void *w_ft, int ft_dtype, int32_t n_variants,
                                    int64_t d_out, int64_t d_in, double *gram, double *cosine, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    if (ft_dtype != BD_BF16 && ft_dtype != BD_F32)
        return fail(BD_EINVAL, "ft_dtype must be BD_BF16 (0) or BD_F32 (1), got %d", ft_dtype);
    if (n_variants < 1 || n_variants > bd::kSimilarityMaxVariants)
        return fail(BD_EINVAL, "n_variants must be in [1, %d] (got %d)", bd::kSimilarityMaxVariants, n_variants);
    BD_TRY(check_matrix(d_out, d_in));
    // a row's workgroup has a wave for each pair of tiles of four variants
    const int tiles = (n_variants + 3) / 4;
    if (d_out > max_workgroups(64 * tiles * (tiles + 1) / 2))
        return fail(BD_ESHAPE, "matrix [%lld, %lld] exceeds the similarity_delta grid", (long long)d_out, (long long)d_in);
    const size_t need = bitdelta_similarity_delta_workspace(n_variants, d_out, d_in);
    if (workspace_bytes < need)
        return fail(BD_EWORKSPACE, "similarity_delta needs %zu workspace bytes, got %zu", need, workspace_bytes);
    BD_NONNULL(w_base);
    BD_NONNULL(w_ft);
    BD_NONNULL(gram);
    BD_NONNULL(cosine);
    BD_NONNULL(workspace);
    BD_ALIGNED(w_base, 16);
    BD_ALIGNED(w_ft, 16);
    BD_ALIGNED(gram, 8);
    BD_ALIGNED(cosine, 8);
    BD_ALIGNED(workspace, 8);
    return device(bd::launch_similarity_delta(w_base, w_ft, ft_dtype == BD_F32, n_variants, d_out, d_in, gram, cosine,
                                              static_cast<double *>(workspace), (hipStream_t)stream),
                  "bitdelta_similarity_delta");
}

size_t bitdelta_monosoup_workspace(int64_t rows, int64_t cols, int32_t k, int32_t rank)
{
    const int64_t lim = (int64_t)1 << 21;
    if (rows < 1 || cols < 4 || rows > lim || cols > lim || k < 1 || k > 64 || rank < 0 || rank > bd::kMsL)
        return 0;
    return bd::monosoup_workspace_bytes(rows, cols, k, rank);
}

bd_status bitdelta_monosoup(const bd_bf16 *w_base, const float *w_ft, const float *omega, int32_t k, int64_t rows,
                            int64_t cols, int32_t rank, int32_t power_iters, float *w_merged, double *sigma,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    const int64_t lim = (int64_t)1 << 21;
    if (rows < 1 || cols < 4 || cols % 4 != 0 || rows > lim || cols > lim)
        return fail(BD_ESHAPE, "monosoup needs rows in [1, 2^21] and cols a multiple of 4 in [4, 2^21] (got %lld, %lld)",
                    (long long)rows, (long long)cols);
    if (k < 1 || k > 64)
        return fail(BD_EINVAL, "monosoup needs k in [1, 64] (got %d)", k);
    const int64_t max_rank = rows < cols ? (rows < bd::kMsL ? rows : bd::kMsL) : (cols < bd::kMsL ? cols : bd::kMsL);
    if (rank < 0 || rank > max_rank)
        return fail(BD_EINVAL, "monosoup rank must be in [0, %lld] (got %d)", (long long)max_rank, rank);
    if (power_iters < 0 || power_iters > 256)
        return fail(BD_EINVAL, "monosoup power_iters must be in [0, 256] (got %d)", power_iters);
    const size_t need = bitdelta_monosoup_workspace(rows, cols, k, rank);
    if (workspace_bytes < need)
        return fail(BD_EWORKSPACE, "monosoup needs %zu workspace bytes, got %zu", need, workspace_bytes);
    BD_NONNULL(w_base);
    BD_NONNULL(w_ft);
    BD_NONNULL(w_merged);
    BD_ALIGNED(w_base, 8);
    BD_ALIGNED(w_ft, 16);
    BD_ALIGNED(w_merged, 16);
    if (rank > 0) {
        BD_NONNULL(omega);
        BD_ALIGNED(omega, 16);
    }
    if (sigma)
        BD_ALIGNED(sigma, 8);
    if (need) {
        BD_NONNULL(workspace);
        BD_ALIGNED(workspace, 256);
    }
    return device(bd::launch_monosoup(reinterpret_cast<const uint16_t *>(w_base), w_ft, omega, k, rows, cols, rank,
                                      power_iters, w_merged, sigma, workspace, (hipStream_t)stream),
                  "bitdelta_monosoup");
}

int64_t bitdelta_probe_read_sink_words(int64_t bytes)
{
    if (bytes < 16 || bytes % 16 != 0 || bytes >= ((int64_t)1 << 31))
        return 0;
    return bd::probe_read_sink_words(bytes);
}

bd_status bitdelta_probe_read(const void *src, int64_t bytes, uint32_t *sink, void *stream)
{
    if (bytes < 16 || bytes % 16 != 0 || bytes >= ((int64_t)1 << 31))
        return fail(BD_ESHAPE, "probe_read needs bytes a multiple of 16 in [16, 2^31 - 1] (got %lld)",
                    (long long)bytes);
    BD_NONNULL(src);
    BD_NONNULL(sink);
    BD_ALIGNED(src, 16);
    BD_ALIGNED(sink, 4);
    return device(bd::launch_probe_read(src, bytes, sink, (hipStream_t)stream), "bitdelta_probe_read");
}

bd_status bitdelta_probe_mfma(int32_t blocks, int32_t iters, float a, float b, uint32_t *sink, void *stream)
{
    if (blocks < 1 || blocks > (1 << 20) || iters < 1 || iters > (1 << 20))
        return fail(BD_ESHAPE, "probe_mfma needs blocks and iters in [1, 2^20] (got %d, %d)", blocks, iters);
    BD_NONNULL(sink);
    BD_ALIGNED(sink, 4);
    return device(bd::launch_probe_mfma(blocks, iters, a, b, sink, (hipStream_t)stream), "bitdelta_probe_mfma");
}

bd_status bitdelta_probe_lds(int32_t blocks, int32_t iters, int32_t mode, int32_t stride, const void *src,
                             int64_t src_bytes, uint32_t *sink, uint64_t *cycles, void *stream)
{
    if (mode < 0 || mode > 3)
        return fail(BD_EINVAL, "probe_lds mode must be 0..3 (got %d)", mode);
    if (blocks < 1 || blocks > (1 << 20) || iters < 1 || iters > (1 << 16) || stride < 1 || stride > (1 << 20))
        return fail(BD_ESHAPE, "probe_lds needs blocks in [1, 2^20], iters in [1, 2^16], stride in [1, 2^20] "
                               "(got %d, %d, %d)", blocks, iters, stride);
    if (mode == 3) {
        if (src_bytes < 1024 || src_bytes > ((int64_t)1 << 30) || (src_bytes & (src_bytes - 1)) != 0)
            return fail(BD_ESHAPE, "probe_lds mode 3 needs src_bytes a power of two in [1 KB, 1 GiB] (got %lld)",
                        (long long)src_bytes);
        BD_NONNULL(src);
        BD_ALIGNED(src, 16);
    }
    BD_NONNULL(sink);
    BD_NONNULL(cycles);
    BD_ALIGNED(sink, 4);
    BD_ALIGNED(cycles, 8);
    return device(bd::launch_probe_lds(blocks, iters, mode, stride, src, src_bytes, sink, cycles, (hipStream_t)stream),
                  "bitdelta_probe_lds");
}

// ---------------------------------------------- between the linears of a layer

namespace {

bd_status check_cache(const bd_kv_cache *cache)
{
    BD_NONNULL(cache);
    const bd_kv_cache &c = *cache;
    if (c.dtype != BD_KV_BF16 && c.dtype != BD_KV_E4M3)
        return fail(BD_EINVAL, "cache dtype must be BD_KV_BF16 (0) or BD_KV_E4M3 (1), got %d", c.dtype);
    if (c.n_pages < 1 || c.n_kv_heads < 1 || c.n_kv_heads > 1024)
        return fail(BD_ESHAPE, "cache needs n_pages >= 1 and n_kv_heads in [1, 1024] (got %d, %d)", c.n_pages,
                    c.n_kv_heads);
    if (c.page_size < 1 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)) != 0)
        return fail(BD_ESHAPE, "page_size must be a power of two in [1, 1024] (got %d)", c.page_size);
    if (c.head_dim != 64 && c.head_dim != 128)
        return fail(BD_ESHAPE, "head_dim must be 64 or 128 (got %d)", c.head_dim);
    // a cell's number is 32 bits wide in the kernels (its address is not)
    if ((int64_t)c.n_pages * c.n_kv_heads > kMaxGrid / c.page_size)
        return fail(BD_ESHAPE, "n_pages * n_kv_heads * page_size must be below 2^31");
    if (c.dtype == BD_KV_BF16 && (c.k_scale || c.v_scale))
        return fail(BD_EINVAL, "a bf16 cache takes no k_scale or v_scale");
    BD_NONNULL(c.k);
    BD_NONNULL(c.v);
    BD_ALIGNED(c.k, 16);
    BD_ALIGNED(c.v, 16);
    BD_ALIGNED(c.k_scale, 4);
    BD_ALIGNED(c.v_scale, 4);
    return BD_OK;
}

bd_status check_batch(const bd_batch *batch)
{
    BD_NONNULL(batch);
    const bd_batch &b = *batch;
    if (b.n_tokens < 0 || b.n_tokens > kMaxGrid)
        return fail(BD_ESHAPE, "n_tokens must be in [0, 2^31) (got %lld)", (long long)b.n_tokens);
    if (b.n_seqs < 0 || b.n_seqs > BD_MAX_SEQS || b.n_groups < 0 || b.n_groups > BD_MAX_GROUPS)
        return fail(BD_ESHAPE, "n_seqs must be in [0, %d] and n_groups in [0, %d] (got %d, %d)", BD_MAX_SEQS,
                    BD_MAX_GROUPS, b.n_seqs, b.n_groups);
    if (b.max_new < 0)
        return fail(BD_ESHAPE, "max_new must not be negative (got %d)", b.max_new);
    if (b.n_seqs > 0) {
        if (b.max_pages < 1)
            return fail(BD_ESHAPE, "max_pages must be positive (got %d)", b.max_pages);
        BD_NONNULL(b.q_start);
        BD_NONNULL(b.kv_len);
        BD_NONNULL(b.page_table);
        BD_ALIGNED(b.q_start, 4);
        BD_ALIGNED(b.kv_len, 4);
        BD_ALIGNED(b.page_table, 4);
    }
    if (b.n_groups > 0) {
        if (b.max_prefix_pages < 1)
            return fail(BD_ESHAPE, "max_prefix_pages must be positive (got %d)", b.max_prefix_pages);
        BD_NONNULL(b.group_start);
        BD_NONNULL(b.prefix_len);
        BD_NONNULL(b.prefix_table);
        BD_ALIGNED(b.group_start, 4);
        BD_ALIGNED(b.prefix_len, 4);
        BD_ALIGNED(b.prefix_table, 4);
    }
    return BD_OK;
}

bd_status check_rows(const char *name, int64_t stride, int64_t width, int64_t multiple)
{
    if (stride < width || stride % multiple != 0 || stride > (int64_t)1 << 40)
        return fail(BD_ESHAPE, "%s row stride must be a multiple of %lld and at least %lld (got %lld)", name,
                    (long long)multiple, (long long)width, (long long)stride);
    return BD_OK;
}

bd_status check_heads(int32_t n_heads, const bd_kv_cache &c, const bd_batch &b)
{
    if (n_heads < 1 || n_heads > 1024 || n_heads % c.n_kv_heads != 0)
        return fail(BD_ESHAPE, "n_heads must be a multiple of n_kv_heads = %d in [1, 1024] (got %d)", c.n_kv_heads,
                    n_heads);
    if (b.n_tokens > kMaxGrid / n_heads)
        return fail(BD_ESHAPE, "n_tokens * n_heads must be below 2^31 (got %lld x %d)", (long long)b.n_tokens, n_heads);
    return BD_OK;
}

}  // namespace

bd_status bitdelta_block_norm(const void *residual, int64_t residual_stride, int residual_dtype, const bd_bf16 *block,
                              int64_t block_stride, const bd_bf16 *gate, int64_t gate_stride, int gate_act,
                              float scale, const void *post_weight, const void *pre_weight, int weight_dtype,
                              const int32_t *variant_ids, int32_t n_variants, int64_t m, int64_t d, float eps,
                              void *residual_out, int64_t residual_out_stride, bd_bf16 *x, void *stream)
{
    if (residual_dtype != BD_BF16 && residual_dtype != BD_F32)
        return fail(BD_EINVAL, "residual_dtype must be BD_BF16 (0) or BD_F32 (1), got %d", residual_dtype);
    if (weight_dtype != BD_BF16 && weight_dtype != BD_F32)
        return fail(BD_EINVAL, "weight_dtype must be BD_BF16 (0) or BD_F32 (1), got %d", weight_dtype);
    if (gate_act != BD_GATE_NONE && gate_act != BD_GATE_SIGMOID && gate_act != BD_GATE_SILU)
        return fail(BD_EINVAL, "gate_act must be BD_GATE_NONE, _SIGMOID or _SILU (0..2), got %d", gate_act);
    if (n_variants < 1)
        return fail(BD_EINVAL, "n_variants must be positive (got %d)", n_variants);
    if (!(eps >= 0.0f))
        return fail(BD_EINVAL, "eps must not be negative or NaN");
    if (m < 0 || m > kMaxGrid)
        return fail(BD_ESHAPE, "m must be in [0, 2^31) (got %lld)", (long long)m);
    if (d < 1 || d > BD_NORM_MAX_WIDTH)
        return fail(BD_ESHAPE, "d must be in [1, %d] (got %lld)", BD_NORM_MAX_WIDTH, (long long)d);
    if (m == 0)   // an empty tensor has no address
        return BD_OK;
    if (!block && (post_weight || gate))
        return fail(BD_EINVAL, "post_weight and gate need a block");
    if (!pre_weight && !residual_out)
        return fail(BD_EINVAL, "block_norm has no output: give pre_weight or residual_out");
    BD_NONNULL(residual);
    BD_TRY(check_rows("residual", residual_stride, d, 1));
    const size_t re = residual_dtype == BD_F32 ? 4 : 2, we = weight_dtype == BD_F32 ? 4 : 2;
    BD_ALIGNED(residual, re);
    if (block) {
        BD_TRY(check_rows("block", block_stride, d, 1));
        BD_ALIGNED(block, 2);
    }
    if (gate) {
        BD_TRY(check_rows("gate", gate_stride, d, 1));
        BD_ALIGNED(gate, 2);
    }
    if (residual_out) {
        BD_TRY(check_rows("residual_out", residual_out_stride, d, 1));
        BD_ALIGNED(residual_out, re);
        if (residual_out == residual && residual_out_stride != residual_stride)
            return fail(BD_EINVAL, "residual_out over residual needs the same row stride");
    }
    if (pre_weight) {
        BD_NONNULL(x);
        BD_ALIGNED(x, 2);
    }
    BD_ALIGNED(post_weight, we);
    BD_ALIGNED(pre_weight, we);
    BD_ALIGNED(variant_ids, 4);
    bd::NormArgs a;
    a.residual = residual, a.block = block, a.gate = gate, a.post_weight = post_weight, a.pre_weight = pre_weight;
    // without weights there is nothing for an id to be outside of
    a.ids = post_weight || pre_weight ? variant_ids : nullptr;
    a.residual_out = residual_out, a.x = x;
    a.residual_stride = residual_stride, a.block_stride = block_stride, a.gate_stride = gate_stride;
    a.out_stride = residual_out_stride, a.m = m;
    a.n_variants = n_variants, a.d = (int32_t)d, a.gate_act = gate_act, a.scale = scale, a.eps = eps;
    a.residual_f32 = residual_dtype == BD_F32, a.weight_f32 = weight_dtype == BD_F32;
    return device(bd::launch_block_norm(a, (hipStream_t)stream), "bitdelta_block_norm");
}

bd_status bitdelta_kv_append(const bd_bf16 *q, int64_t q_stride, const bd_bf16 *k, int64_t k_stride, const bd_bf16 *v,
                             int64_t v_stride, int32_t n_heads, const double *inv_freq, int32_t rotary,
                             int interleaved, const bd_kv_cache *cache, const bd_batch *batch, bd_bf16 *q_out,
                             void *stream)
{
    BD_TRY(check_cache(cache));
    BD_TRY(check_batch(batch));
    if (interleaved != 0 && interleaved != 1)
        return fail(BD_EINVAL, "interleaved must be 0 or 1 (got %d)", interleaved);
    if (rotary < 0 || rotary > cache->head_dim || rotary % 16 != 0)
        return fail(BD_ESHAPE, "rotary must be a multiple of 16 in [0, head_dim] (got %d)", rotary);
    if (n_heads != 0)
        BD_TRY(check_heads(n_heads, *cache, *batch));
    else if (q || q_out)
        return fail(BD_EINVAL, "q and q_out must be NULL where n_heads is 0");
    if (batch->n_tokens == 0)
        return BD_OK;
    BD_NONNULL(k);
    BD_NONNULL(v);
    BD_ALIGNED(k, 16);
    BD_ALIGNED(v, 16);
    BD_TRY(check_rows("k", k_stride, (int64_t)cache->n_kv_heads * cache->head_dim, 8));
    BD_TRY(check_rows("v", v_stride, (int64_t)cache->n_kv_heads * cache->head_dim, 8));
    if (n_heads) {
        BD_NONNULL(q);
        BD_NONNULL(q_out);
        BD_ALIGNED(q, 16);
        BD_ALIGNED(q_out, 16);
        BD_TRY(check_rows("q", q_stride, (int64_t)n_heads * cache->head_dim, 8));
        if (q_out == q && q_stride != (int64_t)n_heads * cache->head_dim)
            return fail(BD_EINVAL, "q_out over q needs a dense q");
    }
    if (rotary) {
        BD_NONNULL(inv_freq);
        BD_ALIGNED(inv_freq, 8);
    }
    return device(bd::launch_kv_append(q, q_stride, k, k_stride, v, v_stride, n_heads, inv_freq, rotary,
                                       interleaved != 0, *cache, *batch, q_out, (hipStream_t)stream),
                  "bitdelta_kv_append");
}

size_t bitdelta_attention_workspace(int32_t n_heads, const bd_kv_cache *cache, const bd_batch *batch)
{
    if (check_cache(cache) != BD_OK || check_batch(batch) != BD_OK || check_heads(n_heads, *cache, *batch) != BD_OK)
        return 0;
    return bd::attention_workspace_bytes(n_heads, *cache, *batch);
}

bd_status bitdelta_attention(const bd_bf16 *q, int64_t q_stride, int32_t n_heads, float scale,
                             const bd_kv_cache *cache, const bd_batch *batch, bd_bf16 *out, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    BD_TRY(check_cache(cache));
    BD_TRY(check_batch(batch));
    BD_TRY(check_heads(n_heads, *cache, *batch));
    if (!(scale > 0.0f) || scale > std::numeric_limits<float>::max())
        return fail(BD_EINVAL, "scale must be positive and finite");
    if (batch->n_tokens == 0)
        return BD_OK;
    BD_NONNULL(q);
    BD_NONNULL(out);
    BD_ALIGNED(q, 16);
    BD_ALIGNED(out, 16);
    BD_TRY(check_rows("q", q_stride, (int64_t)n_heads * cache->head_dim, 8));
    const size_t need = bd::attention_workspace_bytes(n_heads, *cache, *batch);
    if (workspace_bytes < need)
        return fail(BD_EWORKSPACE, "attention needs %zu workspace bytes, got %zu", need, workspace_bytes);
    if (need) {
        BD_NONNULL(workspace);
        BD_ALIGNED(workspace, 16);
    }
    return device(bd::launch_attention(q, q_stride, n_heads, scale, *cache, *batch, out, workspace,
                                       (hipStream_t)stream),
                  "bitdelta_attention");
}

}  // extern "C"
