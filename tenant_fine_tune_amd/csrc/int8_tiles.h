// The tiled product over an 8-bit base (linear_int8_tiles.hip), for calls of
// many tokens.
#pragma once

#include "int8_launch.h"

namespace bd {

// Whether the tiles take the call's rows: whole dwords of signs, from a whole one on.
bool int8_tiles_take(const Int8Args &a);
size_t int8_tiles_workspace_bytes(int64_t m, int32_t n_variants, int64_t d_out, int64_t d_in);
hipError_t launch_int8_tiles(const Int8Args &a, void *workspace, hipStream_t s);

}  // namespace bd
