// Launchers of the linears over an 8-bit base (include/bitdelta_int8.h).
// Arguments are checked by api.cpp before any of them is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/bitdelta_int8.h"

namespace bd {

// quantize.hip
hipError_t launch_quantize_int8(const void *x, int64_t x_stride, bool f32, int64_t m, int64_t d, int8_t *q,
                                float *scale, hipStream_t s);

// linear_int8.hip
struct Int8Args {
    const int8_t *q, *w;
    const float *q_scale, *w_scale;
    const uint8_t *signs;      // NULL: no delta
    const float *alpha;
    const int32_t *ids;        // NULL: one delta for all
    void *y;
    int64_t m, d_out, d_in;
    int32_t n_variants;
    bool per_matrix, f32;
};
size_t linear_int8_workspace_bytes(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in);
hipError_t launch_linear_int8(const Int8Args &a, void *workspace, hipStream_t s);

}  // namespace bd
