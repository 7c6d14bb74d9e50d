// Device-side reading of a batch over a paged cache (bd_batch, bd_kv_cache).
// Every index that comes from device memory is bounded here before it is used
// as an address.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bitdelta_decoder.h"

namespace bd {

struct Paged {
    bd_batch b;
    int32_t n_pages, n_kv, page_shift;
};

__device__ __forceinline__ int clampi(int64_t x, int64_t lo, int64_t hi)
{
    return (int)(x < lo ? lo : x > hi ? hi : x);
}

// First token of sequence s, or of the padding behind the last one (s = n_seqs).
__device__ __forceinline__ int seq_begin(const Paged &p, int s) { return clampi(p.b.q_start[s], 0, p.b.n_tokens); }

__device__ __forceinline__ int own_keys(const Paged &p, int s)
{
    return clampi(p.b.kv_len[s], 0, ((int64_t)p.b.max_pages << p.page_shift));
}

__device__ __forceinline__ int prefix_keys(const Paged &p, int g)
{
    return clampi(p.b.prefix_len[g], 0, ((int64_t)p.b.max_prefix_pages << p.page_shift));
}

__device__ __forceinline__ int group_begin(const Paged &p, int g) { return clampi(p.b.group_start[g], 0, p.b.n_seqs); }

// The number of i in [0, n) with clamp(a[i + 1]) <= x, counted by the whole
// workgroup: the sequence of token x, or the group of sequence x, where the
// starts do not decrease; n where x lies behind the last one.
__device__ __forceinline__ int count_upto(const int32_t *a, int n, int64_t x, int64_t hi)
{
    int c = 0;
    for (int i = 0; i < n; i += blockDim.x) {
        const int j = i + threadIdx.x;
        c += __syncthreads_count(j < n && clampi(a[j + 1], 0, hi) <= x);
    }
    return c;
}

// Token t's sequence, or -1 for padding: after it, begin <= t < end holds
// whatever the starts are, so t's place is below own_keys().
__device__ __forceinline__ int seq_of(const Paged &p, int64_t t)
{
    const int s = count_upto(p.b.q_start, p.b.n_seqs, t, p.b.n_tokens);
    return s < p.b.n_seqs && seq_begin(p, s) <= t && t < seq_begin(p, s + 1) ? s : -1;
}

// The group of sequence s, or -1.
__device__ __forceinline__ int group_of(const Paged &p, int s)
{
    if (p.b.n_groups == 0)
        return -1;
    const int g = count_upto(p.b.group_start, p.b.n_groups, s, p.b.n_seqs);
    return g < p.b.n_groups && group_begin(p, g) <= s && s < group_begin(p, g + 1) ? g : -1;
}

}  // namespace bd
