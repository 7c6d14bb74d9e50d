// Launcher of the draw of tokens (include/bitdelta_sample.h).  Arguments are
// checked by api.cpp before it is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/bitdelta_sample.h"

namespace bd {

struct SampleArgs {
    const void *logits;
    int64_t stride, m;
    int32_t vocab;
    bool f32;
    const float *u, *temperature, *top_p, *min_p;   // NULL: the value beside it
    const int32_t *top_k;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
    int32_t *tokens;
    float *logprobs;
};
size_t sample_workspace_bytes(int64_t m, int64_t vocab);
hipError_t launch_sample(const SampleArgs &a, void *workspace, hipStream_t s);

}  // namespace bd
