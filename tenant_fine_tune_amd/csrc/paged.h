// Reading of a batch over a paged cache (bd_batch, bd_kv_cache), on the device
// and, for the tests, on the host.  Every index that comes from device memory
// is bounded here before it is used as an address.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bitdelta_decoder.h"

namespace bd {

#define BD_HD __host__ __device__ __forceinline__

struct Paged {
    bd_batch b;
    int32_t n_pages, n_kv, page_shift;
};

BD_HD int clampi(int64_t x, int64_t lo, int64_t hi) { return (int)(x < lo ? lo : x > hi ? hi : x); }

// First token of sequence s, or of the padding behind the last one (s = n_seqs).
BD_HD int seq_begin(const Paged &p, int s) { return clampi(p.b.q_start[s], 0, p.b.n_tokens); }

// Keys that a page table of `pages` columns can hold, at most 2^30 (so that
// places and the ends of tiles past them fit 32 bits).
BD_HD int64_t table_keys(const Paged &p, int32_t pages)
{
    const int64_t n = (int64_t)pages << p.page_shift;
    return n < (1 << 30) ? n : 1 << 30;
}

BD_HD int own_keys(const Paged &p, int s) { return clampi(p.b.kv_len[s], 0, table_keys(p, p.b.max_pages)); }
BD_HD int prefix_keys(const Paged &p, int g) { return clampi(p.b.prefix_len[g], 0, table_keys(p, p.b.max_prefix_pages)); }

BD_HD int group_begin(const Paged &p, int g) { return clampi(p.b.group_start[g], 0, p.b.n_seqs); }

// The groups of a batch, held in LDS: what a sequence has to know of its own.
struct Groups {
    int begin[BD_MAX_GROUPS + 1];     // first sequence
    int prefix[BD_MAX_GROUPS];        // keys
    uint8_t shared[BD_MAX_GROUPS];    // see attention_schedule.h
};

// The group of sequence s, or -1: the number of groups that end at or before
// s, where the starts do not decrease.
BD_HD int group_of(const Paged &p, const Groups &gr, int s)
{
    int lo = 0, hi = p.b.n_groups;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (gr.begin[mid + 1] <= s)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < p.b.n_groups && gr.begin[lo] <= s && s < gr.begin[lo + 1] ? lo : -1;
}

// The cell (in units of head_dim numbers) of one head's key j of a page list,
// or -1 where the list names no page of the cache.
BD_HD int cell_of(const Paged &p, const int32_t *table, int head, int j)
{
    const int page = table[j >> p.page_shift];
    if ((unsigned)page >= (unsigned)p.n_pages)
        return -1;
    return ((page * p.n_kv + head) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
}

// Token t's sequence, or -1 for padding, found by the whole workgroup; with
// it begin <= t < end holds whatever the starts are, so t's place is below
// own_keys().
__device__ __forceinline__ int seq_of(const Paged &p, int64_t t)
{
    int s = 0;
    for (int i = 0; i < p.b.n_seqs; i += blockDim.x) {
        const int j = i + threadIdx.x;
        s += __syncthreads_count(j < p.b.n_seqs && seq_begin(p, j + 1) <= t);
    }
    return s < p.b.n_seqs && seq_begin(p, s) <= t && t < seq_begin(p, s + 1) ? s : -1;
}

// The group of sequence s, or -1, found by the whole workgroup without a table.
__device__ __forceinline__ int group_around(const Paged &p, int s)
{
    if (!p.b.n_groups)
        return -1;
    int g = 0;
    for (int i = 0; i < p.b.n_groups; i += blockDim.x) {
        const int j = i + threadIdx.x;
        g += __syncthreads_count(j < p.b.n_groups && group_begin(p, j + 1) <= s);
    }
    return g < p.b.n_groups && group_begin(p, g) <= s && s < group_begin(p, g + 1) ? g : -1;
}

}  // namespace bd
