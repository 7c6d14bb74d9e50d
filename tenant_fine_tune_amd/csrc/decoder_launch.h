// Launchers of the operators between the linears (include/bitdelta_decoder.h).
// Arguments are checked by api.cpp before any of them is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/bitdelta_decoder.h"

namespace bd {

// Workgroups of one dimension of a launch by token: a dimension of 2^32 threads
// or more wraps around without an error, so tokens past these go into another.
constexpr int64_t kTokensAcross = 1 << 20;

struct NormArgs {
    const void *residual;
    const uint16_t *block, *gate;
    const void *post_weight, *pre_weight;
    const int32_t *ids;
    void *residual_out;
    uint16_t *x;
    int64_t residual_stride, block_stride, gate_stride, out_stride, m;
    int32_t n_variants, d, gate_act;
    float scale, eps;
    bool residual_f32, weight_f32;
};
hipError_t launch_block_norm(const NormArgs &a, hipStream_t s);

hipError_t launch_kv_append(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                            const uint16_t *v, int64_t v_stride, int32_t n_heads, const double *inv_freq,
                            int32_t rotary, bool interleaved, const bd_kv_cache &c, const bd_batch &b,
                            uint16_t *q_out, hipStream_t s);

size_t attention_workspace_bytes(int32_t n_heads, const bd_kv_cache &c, const bd_batch &b);
hipError_t launch_attention(const uint16_t *q, int64_t q_stride, int32_t n_heads, float scale, const bd_kv_cache &c,
                            const bd_batch &b, uint16_t *out, void *workspace, hipStream_t s);

}  // namespace bd
