// How the work of one attention call is cut, from the batch's device-side
// lengths: every workgroup of the three kernels derives the same cut for
// itself, so a call needs no plan from the host and can be captured.
//
// A row is a (token, query head of one key head) pair; row r of a sequence is
// token r / G, head r % G.  A sequence of few rows (at most `few`) belongs to
// the streaming kernel, one of more rows to the tiled kernel.  The prefix of
// a group is either taken with each sequence's own keys, or, where the group
// is `shared`, once for the rows of all its sequences by the tiled kernel.
//
//   streaming kernel: runs of (sequence, key head, row tile), each kRunCost
//     units for its beginning and one unit per kStreamKeys keys, laid end to
//     end; workgroup w takes units [w * c, (w + 1) * c).  A run whose keys a
//     workgroup boundary cuts leaves partial states in the slots 2w (keys
//     began before w) and 2w + 1 (they go on after w).
//   tiled kernel: items (segment, row tile, split, key head); a segment is a
//     sequence or a shared prefix.  A split segment, and every segment of a
//     shared group, leaves partial states in planes [split][token][head]:
//     planes [0, splits) for own keys, [splits, 2 splits) for prefixes.
#pragma once

#include "paged.h"

namespace bd {

constexpr int kStreamKeys = 32;      // keys of a streaming unit
constexpr int kTileKeys = 64;        // keys of a tiled step
// Rows of a tiled item: 32 a wave at 128 columns, 64 at 64, where their sums
// fit beside a second wave's on the SIMD and every fragment read from LDS
// serves twice the matrix work.
constexpr int tile_rows(int head_dim) { return head_dim == 64 ? 256 : 128; }
constexpr int kRunCost = 4;          // units that a run's beginning and end cost (0: 75 us for 128 short
                                     // contexts of 64 query heads, a workgroup then got up to 17 runs; 4: 33 us)
constexpr int kMinUnits = 4;         // units that are worth a workgroup: one a wave
constexpr int kMinTiles = 4;         // key tiles that are worth a split
constexpr int kItemCost = 5;         // key tiles that a tiled item's beginning and end cost
constexpr float kSplitCost = 0.06f;  // key tiles that the states of one split of an item cost to write and join
                                     // (0: 78 us for 128 users behind three prefixes, 77 for a chunk of 256 tokens
                                     // beside 15 decodes of 200 to 4000 keys; 0.06: 67 and 70)
constexpr int kSharedNew = 16;       // new tokens a sequence up to which a group is shared
constexpr int kTiledSlots = 512;     // workgroups of the tiled kernel that run at once

struct Sched {
    Paged p;
    int32_t n_heads, group;          // query heads, and those of one key head
    int32_t few;                     // rows up to which a sequence is streamed (INT32_MAX: all)
    int32_t stream_rows;             // rows of a streaming tile
    int32_t stream_wgs;              // workgroups of the streaming kernel
    int32_t tile_rows;               // rows of a tiled item
    int32_t splits;                  // bound of a segment's splits
    bool tiled;                      // the tiled kernel runs
};

struct Segment {
    int tok0, ntok;                  // tokens
    int pre, own;                    // keys of the prefix taken with it, and of its own pages
    int group;                       // its group or -1
    bool shared;                     // the group's prefix is taken once for all
};

BD_HD int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Group g's entry of `gr` (and with the last group the end of the list).
BD_HD void fill_group(const Sched &s, Groups &gr, int g)
{
    const int a = group_begin(s.p, g), b = group_begin(s.p, g + 1);
    gr.begin[g] = a;
    if (g == s.p.b.n_groups - 1)
        gr.begin[g + 1] = b;
    gr.prefix[g] = prefix_keys(s.p, g);
    // a batch without sequences has no starts to read
    const int64_t toks = b - a >= 2 ? (int64_t)seq_begin(s.p, b) - seq_begin(s.p, a) : 0;
    gr.shared[g] = s.tiled && gr.prefix[g] > 0 && toks > 0 && toks <= (int64_t)kSharedNew * (b - a);
}

BD_HD Segment sequence(const Sched &s, const Groups &gr, int i)
{
    Segment g;
    g.tok0 = seq_begin(s.p, i);
    const int n = seq_begin(s.p, i + 1) - g.tok0;
    g.ntok = n < 0 ? 0 : n;
    g.own = own_keys(s.p, i);
    g.group = s.p.b.n_groups ? group_of(s.p, gr, i) : -1;
    g.shared = g.group >= 0 && gr.shared[g.group];
    g.pre = g.group >= 0 && !g.shared ? gr.prefix[g.group] : 0;
    return g;
}

// The shared prefix of group g as a segment of its own (no tokens: not shared).
BD_HD Segment prefix(const Sched &s, const Groups &gr, int g)
{
    Segment q;
    q.shared = gr.shared[g];
    q.group = g;
    q.tok0 = q.shared ? seq_begin(s.p, gr.begin[g]) : 0;
    q.ntok = q.shared ? seq_begin(s.p, gr.begin[g + 1]) - q.tok0 : 0;
    q.pre = q.shared ? gr.prefix[g] : 0;
    q.own = 0;
    return q;
}

BD_HD int64_t rows_of(const Sched &s, const Segment &g) { return (int64_t)g.ntok * s.group; }
BD_HD bool streamed(const Sched &s, const Segment &g) { return rows_of(s, g) <= s.few; }
BD_HD int key_tiles(const Segment &g, int keys) { return (int)(cdiv(g.pre, keys) + cdiv(g.own, keys)); }

// Own keys that token i of n sees.
BD_HD int own_seen(const Segment &g, int i)
{
    const int n = g.own - g.ntok + i + 1;
    return n < 0 ? 0 : n;
}

// ------------------------------------------------------------ streaming kernel
BD_HD int64_t stream_row_tiles(const Sched &s, const Segment &g) { return cdiv(rows_of(s, g), s.stream_rows); }
BD_HD int stream_run(const Segment &g) { return kRunCost + key_tiles(g, kStreamKeys); }
BD_HD int64_t stream_units(const Sched &s, const Segment &g)
{
    return g.ntok && streamed(s, g) && g.pre + g.own > 0 ? s.p.n_kv * stream_row_tiles(s, g) * stream_run(g) : 0;
}
// Units of a workgroup, of `total` in all.
BD_HD int64_t stream_chunk(const Sched &s, int64_t total)
{
    const int64_t c = cdiv(total, s.stream_wgs);
    return c < kMinUnits ? kMinUnits : c;
}

// ---------------------------------------------------------------- tiled kernel
// Segments [0, n_seqs) are sequences, the next n_groups shared prefixes.
BD_HD Segment tiled_segment(const Sched &s, const Groups &gr, int i)
{
    if (i >= s.p.b.n_seqs)
        return prefix(s, gr, i - s.p.b.n_seqs);
    Segment g = sequence(s, gr, i);
    if (streamed(s, g))
        g.ntok = 0;
    return g;
}
BD_HD int64_t tiled_row_tiles(const Sched &s, const Segment &g) { return cdiv(rows_of(s, g), s.tile_rows); }
// Work of a segment in key tiles (a causal one's as if it were not).
BD_HD int64_t tiled_work(const Sched &s, const Segment &g)
{
    return s.p.n_kv * tiled_row_tiles(s, g) * key_tiles(g, kTileKeys);
}
// Time of the whole work, in key tiles, if each of `items` unsplit items with
// `work` key tiles in all were cut into k.
BD_HD float tiled_time(int64_t items, int64_t work, int k)
{
    const float join = k > 1 ? kSplitCost * items * k : 0.0f;
    return ceilf((float)items * k / kTiledSlots) * (ceilf((float)work / ((float)items * k)) + kItemCost) + join;
}
// Key tiles of a split where items are cut into k on the average.
BD_HD int64_t tiled_depth(int64_t items, int64_t work, int k)
{
    const int64_t d = items > 0 ? cdiv(work, items * k) : 0;
    return d < kMinTiles ? kMinTiles : d;
}
BD_HD int tiled_splits(const Sched &s, const Segment &g, int64_t depth)
{
    const int64_t n = (key_tiles(g, kTileKeys) + depth / 2) / depth;
    return (int)(n < 1 ? 1 : n > s.splits ? s.splits : n);
}
BD_HD int64_t tiled_items(const Sched &s, const Segment &g, int64_t depth)
{
    return g.ntok ? s.p.n_kv * tiled_row_tiles(s, g) * tiled_splits(s, g, depth) : 0;
}

}  // namespace bd
