// Walks the cut of attention_schedule.h on the host as the kernels do, over
// random batches, some with starts, lengths, groups and page numbers that make
// no sense.  For every batch: no index leaves the arrays that it is bound to;
// for batches that make sense also: every (row, key that it sees) is weighed
// exactly once, every partial state that a join reads was written once, and
// every row is finished exactly once.
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <random>
#include <set>
#include <vector>

#include "../tenant_fine_tune_amd/csrc/attention_schedule.h"

using namespace bd;

static int failures = 0;
#define EXPECT(c)                                                      \
    do {                                                               \
        if (!(c) && failures++ < 20)                                   \
            fprintf(stderr, "line %d: %s (case %d)\n", __LINE__, #c, current); \
    } while (0)
static int current = 0;

struct Case {
    std::vector<int32_t> q_start, kv_len, table, group_start, prefix_len, ptable;
    Sched s;
    bool sane;
};

static Case make(std::mt19937 &r, bool sane)
{
    const auto u = [&](int a, int b) { return (int)(a + r() % (unsigned)(b - a + 1)); };
    Case c;
    c.sane = sane;
    Paged &p = c.s.p;
    const int n = u(0, 12), page = 1 << u(0, 5), groups = n ? u(0, 3) : 0;
    p.page_shift = __builtin_ctz(page);
    p.n_kv = u(1, 3);
    c.s.group = u(1, 9);
    c.s.n_heads = p.n_kv * c.s.group;
    int t = 0, most = 0, keys = 0, pkeys = 0;
    c.q_start.push_back(0);
    for (int i = 0; i < n; ++i) {
        const int m = u(0, 3) ? u(0, 3) : u(0, 90), ctx = u(0, 2) ? u(0, 40) : u(0, 700);
        t += m;
        c.q_start.push_back(t);
        c.kv_len.push_back(u(0, 9) ? ctx + m : u(0, m));
        keys = std::max(keys, c.kv_len.back());
        most = std::max(most, m);
    }
    for (int g = 0; g < groups; ++g) {
        c.prefix_len.push_back(u(0, 3) ? u(1, 300) : u(0, 2500));
        pkeys = std::max(pkeys, c.prefix_len.back());
    }
    if (groups) {
        c.group_start.push_back(u(0, n));
        for (int g = 0; g < groups; ++g)
            c.group_start.push_back(u(c.group_start.back(), n));
    }
    p.b.n_tokens = t + u(0, 3);
    p.b.n_seqs = n, p.b.n_groups = groups;
    p.b.max_pages = std::max(1, (keys + page - 1) / page);
    p.b.max_prefix_pages = std::max(1, (pkeys + page - 1) / page);
    p.n_pages = 50;
    c.table.resize((size_t)n * p.b.max_pages);
    c.ptable.resize((size_t)groups * p.b.max_prefix_pages);
    for (auto *v : {&c.table, &c.ptable})
        for (auto &x : *v)
            x = u(0, 9) ? u(0, p.n_pages - 1) : (int32_t)r();
    if (!sane)
        for (auto *v : {&c.q_start, &c.kv_len, &c.group_start, &c.prefix_len})
            for (auto &x : *v)
                if (u(0, 2) == 0)
                    x = u(0, 1) ? (int32_t)r() : u(-3, 30);
    p.b.q_start = c.q_start.data(), p.b.kv_len = c.kv_len.data(), p.b.page_table = c.table.data();
    p.b.group_start = c.group_start.data(), p.b.prefix_len = c.prefix_len.data();
    p.b.prefix_table = c.ptable.data();
    c.s.tiled = groups > 0 || u(0, 1);
    c.s.few = c.s.tiled ? 32 : INT_MAX;
    c.s.stream_rows = u(0, 1) ? 16 : 32;
    c.s.stream_wgs = u(0, 2) ? u(1, 40) : 512;
    c.s.tile_rows = tile_rows(u(0, 1) ? 64 : 128);
    c.s.splits = c.s.tiled ? u(1, 9) : 1;
    return c;
}

int main()
{
    std::mt19937 r(7);
    for (current = 0; current < 500; ++current) {
        Case c = make(r, current % 2 == 0);
        const Sched &s = c.s;
        const Paged &p = s.p;
        Groups gr;
        for (int g = 0; g < p.b.n_groups; ++g)
            fill_group(s, gr, g);
        const int64_t T = p.b.n_tokens, H = s.n_heads;
        typedef std::pair<int64_t, int64_t> Row;                       // token, head
        std::map<Row, std::map<int64_t, int>> weighed;                  // key: place, or -1 - place of a prefix
        std::map<Row, int> finished;
        std::map<int64_t, int> part;                                    // partial rows written
        const int64_t slots = 2 * (int64_t)s.stream_wgs * s.stream_rows, plane = T * H;
        const int64_t planes = p.b.n_groups ? 2 * s.splits : s.splits > 1 ? s.splits : 0;

        const auto weigh = [&](const Segment &g, int64_t row, int head, int seq, int t, int keys) {
            const int tok = (int)(row / s.group);
            const int64_t at = g.tok0 + tok;
            EXPECT(at >= 0 && at < T);
            const int pre_tiles = (int)cdiv(g.pre, keys);
            const bool own = t >= pre_tiles;
            const int j0 = (own ? t - pre_tiles : t) * keys;
            for (int j = j0; j < j0 + keys; ++j) {
                if (j >= (own ? g.own : g.pre))
                    break;
                // the place is in the table's columns
                EXPECT((j >> p.page_shift) < (own ? p.b.max_pages : p.b.max_prefix_pages));
                EXPECT(own ? seq >= 0 && seq < p.b.n_seqs : g.group >= 0 && g.group < p.b.n_groups);
                const int cell = cell_of(p, own ? &c.table[(size_t)seq * p.b.max_pages]
                                                : &c.ptable[(size_t)g.group * p.b.max_prefix_pages], head, j);
                EXPECT(cell >= -1 && cell < (int64_t)p.n_pages * p.n_kv << p.page_shift);
                if (own && j >= own_seen(g, tok))
                    continue;
                ++weighed[{at, head * s.group + row % s.group}][own ? j : -1 - (int64_t)j];
            }
        };
        // streaming kernel
        int64_t total = 0;
        std::vector<int64_t> begin;
        for (int i = 0; i < p.b.n_seqs; ++i)
            begin.push_back(total), total += stream_units(s, sequence(s, gr, i));
        const int64_t chunk = stream_chunk(s, total);
        for (int64_t w = 0; w < s.stream_wgs; ++w) {
            int64_t at = w * chunk, end = std::min(total, at + chunk);
            int seq = 0;
            while (at < end) {
                while (begin[seq] + stream_units(s, sequence(s, gr, seq)) <= at)
                    ++seq;
                EXPECT(seq < p.b.n_seqs);
                const Segment g = sequence(s, gr, seq);
                const int tiles = key_tiles(g, kStreamKeys);
                const int len = stream_run(g);
                const int64_t run = (at - begin[seq]) / len, rt = stream_row_tiles(s, g);
                const int from = (int)((at - begin[seq]) % len), to = (int)std::min<int64_t>(len, from + end - at);
                const int t0 = std::max(from - kRunCost, 0), t1 = to - kRunCost;
                at += to - from;
                if (t0 >= t1)
                    continue;
                const int head = (int)(run / rt);
                EXPECT(head < p.n_kv);
                const int64_t row0 = run % rt * s.stream_rows;
                const bool whole = t0 == 0 && t1 == tiles;
                for (int64_t row = row0; row < std::min(rows_of(s, g), row0 + s.stream_rows); ++row) {
                    for (int t = t0; t < t1; ++t)
                        weigh(g, row, head, seq, t, kStreamKeys);
                    const int64_t out = (g.tok0 + row / s.group) * H + head * s.group + row % s.group;
                    if (whole && !g.shared) {
                        ++finished[{out / H, out % H}];
                    } else {
                        const int64_t pr = whole ? slots + out : (2 * w + (t0 == 0)) * s.stream_rows + row - row0;
                        EXPECT(pr >= 0 && pr < slots + planes * plane);
                        ++part[pr];
                    }
                }
            }
        }
        EXPECT(total <= chunk * s.stream_wgs);
        // tiled kernel
        int64_t work = 0, items_all = 0, depth = INT_MAX;
        const int n_seg = p.b.n_seqs + p.b.n_groups;
        for (int i = 0; i < n_seg; ++i) {
            const Segment g = tiled_segment(s, gr, i);
            work += g.ntok ? tiled_work(s, g) : 0;
            items_all += g.ntok ? p.n_kv * tiled_row_tiles(s, g) : 0;
        }
        if (s.splits > 1) {
            int best = 1;
            for (int k = 2; k <= s.splits; ++k)
                if (tiled_time(items_all, work, k) < tiled_time(items_all, work, best))
                    best = k;
            depth = tiled_depth(items_all, work, best);
        }
        EXPECT(s.tiled || work == 0);
        for (int seg = 0; seg < n_seg; ++seg) {
            const Segment g = tiled_segment(s, gr, seg);
            const int64_t items = tiled_items(s, g, depth);
            for (int64_t idx = 0; idx < items; ++idx) {
                const int splits = tiled_splits(s, g, depth), head = (int)(idx % p.n_kv);
                const int split = (int)(idx / p.n_kv % splits);
                const int64_t row0 = (tiled_row_tiles(s, g) - 1 - idx / p.n_kv / splits) * s.tile_rows;
                const int64_t rows = std::min<int64_t>(s.tile_rows, rows_of(s, g) - row0);
                EXPECT(row0 >= 0 && rows > 0);
                const bool is_prefix = seg >= p.b.n_seqs;
                const int last = is_prefix ? 0 : own_seen(g, (int)((row0 + rows - 1) / s.group));
                const int per = (int)cdiv(key_tiles(g, kTileKeys), splits);
                const int t0 = split * per, t1 = (int)std::min<int64_t>(t0 + per, cdiv(g.pre, kTileKeys) + cdiv(last, kTileKeys));
                for (int64_t row = row0; row < row0 + rows; ++row) {
                    for (int t = t0; t < t1; ++t)
                        weigh(g, row, head, is_prefix ? -1 : seg, t, kTileKeys);
                    const int64_t out = (g.tok0 + row / s.group) * H + head * s.group + row % s.group;
                    if (splits == 1 && !g.shared) {
                        ++finished[{out / H, out % H}];
                    } else {
                        const int64_t pr = slots + (is_prefix ? s.splits + split : split) * plane + out;
                        EXPECT(pr >= 0 && pr < slots + planes * plane);
                        ++part[pr];
                    }
                }
            }
        }
        // join
        for (int64_t tok = 0; tok < T; ++tok) {
            int seq = 0;
            for (int i = 0; i < p.b.n_seqs; ++i)
                seq += seq_begin(p, i + 1) <= tok;
            if (!(seq < p.b.n_seqs && seq_begin(p, seq) <= tok && tok < seq_begin(p, seq + 1)))
                seq = -1;
            for (int h = 0; h < H; ++h) {
                std::vector<int64_t> reads;
                bool done = false;
                const int64_t out = tok * H + h;
                if (seq >= 0) {
                    const Segment g = sequence(s, gr, seq);
                    if (streamed(s, g)) {
                        const int tiles = key_tiles(g, kStreamKeys), head = h / s.group;
                        const int64_t row = (tok - g.tok0) * s.group + h % s.group;
                        if (tiles) {
                            const int64_t u0 = begin[seq] + kRunCost + (head * stream_row_tiles(s, g) + row / s.stream_rows) * stream_run(g);
                            const int64_t w0 = u0 / chunk, n = (u0 + tiles - 1) / chunk - w0 + 1;
                            if (n == 1 && !g.shared)
                                done = true;
                            else if (n == 1)
                                reads.push_back(slots + out);
                            else
                                for (int64_t i = 0; i < n; ++i)
                                    reads.push_back((2 * (w0 + i) + (i == 0)) * s.stream_rows + row % s.stream_rows);
                        }
                    } else {
                        const int n = tiled_splits(s, g, depth);
                        if (n == 1 && !g.shared)
                            done = true;
                        else
                            for (int i = 0; i < n; ++i)
                                reads.push_back(slots + i * plane + out);
                    }
                    if (g.shared)
                        for (int i = 0; i < tiled_splits(s, prefix(s, gr, g.group), depth); ++i)
                            reads.push_back(slots + (s.splits + i) * plane + out);
                }
                for (int64_t pr : reads)
                    EXPECT(pr >= 0 && pr < slots + planes * plane);
                if (!c.sane)
                    continue;
                for (int64_t pr : reads)
                    EXPECT(part[pr] == 1);
                EXPECT(finished[Row(tok, h)] == (done ? 1 : 0));
                std::map<int64_t, int> want;
                if (seq >= 0) {
                    const int own = own_keys(p, seq), at = own - (seq_begin(p, seq + 1) - (int)tok);
                    for (int j = 0; j <= at; ++j)
                        want[j] = 1;
                    const int g = group_of(p, gr, seq);
                    for (int j = 0; g >= 0 && j < prefix_keys(p, g); ++j)
                        want[-1 - (int64_t)j] = 1;
                }
                EXPECT(weighed[Row(tok, h)] == want);
            }
        }
    }
    printf("schedule: %d failures\n", failures);
    return failures ? 1 : 0;
}
