// Walks how the tiled product reads rows of w that end inside 32 columns, on the
// host: no read passes the tensor, and each number of w meets the token's and the
// sign of its own column.
#include <stdio.h>

#include "../tenant_fine_tune_amd/csrc/int8_tiles.h"

using namespace bd;

static int failures = 0;
#define EXPECT(c, ...)                                      \
    do {                                                    \
        if (!(c) && failures++ < 20) {                      \
            fprintf(stderr, "line %d: %s: ", __LINE__, #c); \
            fprintf(stderr, __VA_ARGS__);                   \
            fprintf(stderr, "\n");                          \
        }                                                   \
    } while (0)

int main()
{
    // rows of 8 columns are not read so
    for (int width = 16; width <= 2100; width += 8)
        for (int rows : {1, 2, 5}) {
            const int copied = (width + 31) / 32 * 32, groups = width / 8;
            for (int row = 0; row < rows; ++row) {
                int met = 0;
                for (int k = 0; k < copied; k += 16) {
                    const int from = chunk_column(k, width);
                    EXPECT(from < 0 || row * width + from + 16 <= rows * width, "%d columns, row %d of %d, chunk %d", width,
                           row, rows, k);
                    // all chunks before a row's last step go with the step's column, as one displacement
                    EXPECT(k >= (copied - 1) / 128 * 128 || from == k, "%d columns, chunk %d", width, k);
                    for (int half = 0; half < 2; ++half) {
                        const int group = copied_group(k / 8 + half, groups);
                        EXPECT(group < groups, "%d columns, place %d", width, (k / 8 + half));
                        if (group < 0)
                            continue;
                        ++met;
                        EXPECT(from >= 0 && from / 8 + half == group, "%d columns, place %d", width, (k / 8 + half));
                    }
                }
                EXPECT(met == groups, "%d columns: %d of %d groups", width, met, groups);
            }
        }
    printf("int8 tiles: %d failures\n", failures);
    return failures != 0;
}
