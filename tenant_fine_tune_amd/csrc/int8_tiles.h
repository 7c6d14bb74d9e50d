// The tiled product over an 8-bit base (linear_int8_tiles.hip), for calls of
// many tokens.
#pragma once

#include "int8_launch.h"

namespace bd {

// Whether the tiles take the call's rows: whole dwords of signs, from a whole one on.
bool int8_tiles_take(const Int8Args &a);
size_t int8_tiles_workspace_bytes(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in);
hipError_t launch_int8_tiles(const Int8Args &a, void *workspace, hipStream_t s);

// The tiles read w in chunks of 16 columns from every 16th on, where it stands.  Rows of
// `width` columns, a multiple of 8, may end inside a chunk, and what follows the last row is not
// w's: that chunk is read from 8 columns earlier on.  Column from which the chunk of column k
// is read, -1 if the row has none there.
__host__ __device__ inline int32_t chunk_column(int32_t k, int32_t width)
{
    return k >= width ? -1 : k + 16 > width ? k - 8 : k;
}

// The tokens' numbers and the signs are copied to rows of whole 32 columns then, in groups
// of 8, and stand as w does: group of a row of `groups` at place `at` of the copy, -1
// for zeros.
__host__ __device__ inline int32_t copied_group(int32_t at, int32_t groups)
{
    if (groups % 2 == 0 || at < groups - 1)
        return at < groups ? at : -1;
    return at == groups ? groups - 1 : -1;
}

}  // namespace bd
