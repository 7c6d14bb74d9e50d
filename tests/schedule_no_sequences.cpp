// A batch of padding alone that keeps its groups: no sequences, and so none of
// the arrays that describe them.  The cut of attention_schedule.h must read
// nothing of them, whatever the group starts are, and share no prefix.
#include <limits.h>
#include <stdio.h>

#include "../tenant_fine_tune_amd/csrc/attention_schedule.h"

using namespace bd;

int main()
{
    const int32_t starts[][4] = {{0, 0, 0, 0}, {0, 5, 9, 4096}, {3, -1, INT_MAX, INT_MIN}};
    const int32_t lens[3] = {0, 70, INT_MAX}, table[3 * 4] = {0};
    int failures = 0;
    for (const auto &start : starts) {
        Sched s;
        s.p.b = {nullptr, nullptr, nullptr, start, lens, table, 5, 0, 0, 3, 4, 0};
        s.p.n_pages = 9, s.p.n_kv = 2, s.p.page_shift = 4;
        s.group = 4, s.n_heads = 8, s.tiled = true, s.few = 32, s.stream_rows = 16, s.stream_wgs = 256;
        s.tile_rows = tile_rows(64), s.splits = 64;
        Groups gr;
        for (int g = 0; g < 3; ++g) {
            fill_group(s, gr, g);
            failures += gr.shared[g] != 0 || gr.begin[g] != 0;
        }
        for (int i = 0; i < 3; ++i) {
            const Segment g = tiled_segment(s, gr, i);
            failures += g.ntok != 0 || tiled_items(s, g, 4) != 0;
        }
        failures += group_of(s.p, gr, 0) != -1;
    }
    printf("no sequences: %d failures\n", failures);
    return failures ? 1 : 0;
}
