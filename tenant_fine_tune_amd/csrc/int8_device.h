// Device-side helpers of the products over an 8-bit base (linear_int8.hip,
// linear_int8_tiles.hip): signs to bytes, the epilogue.
#pragma once

#include "bd_device.h"
#include "int8_launch.h"

namespace bd {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// The signs enter the matrix unit as bytes of 0 and 2 (one shift and one mask for
// four of them): sum q sign = sum q (2 b) - sum q.  Dword i (0..7) of the 32 signs
// in `w` holds twice the bits i, i + 8, i + 16, i + 24.
__device__ __forceinline__ uint32_t twice_sign_bytes(uint32_t w, int i)
{
    return (i == 0 ? w << 1 : w >> (i - 1)) & 0x02020202u;
}

// The 32 bytes X0..X7 put into the order of twice_sign_bytes: dword i becomes the
// bytes i, i + 8, i + 16, i + 24 (two transposes of 4 x 4 bytes).
__device__ __forceinline__ void to_sign_order(u32x4 &lo, u32x4 &hi)
{
    const uint32_t x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    u32x4 out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = x[h], b = x[2 + h], c = x[4 + h], d = x[6 + h];
        const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab2 = __builtin_amdgcn_perm(b, a, 0x07030602u);
        const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd2 = __builtin_amdgcn_perm(d, c, 0x07030602u);
        out[h][0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
        out[h][1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
        out[h][2] = __builtin_amdgcn_perm(cd2, ab2, 0x05040100u);
        out[h][3] = __builtin_amdgcn_perm(cd2, ab2, 0x07060302u);
    }
    lo = out[0];
    hi = out[1];
}

__device__ __forceinline__ i32x4 mfma16(u32x4 a, u32x4 b, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Bytes that 64 lanes load (16 or 4 each) straight into LDS, one lane after another.
template <int CACHE = 0>
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, uint8_t *to, uint32_t lane_offset, uint32_t offset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 16, lane_offset, offset, 0, CACHE);
}
__device__ __forceinline__ void copy4(__amdgpu_buffer_rsrc_t r, uint8_t *to, uint32_t lane_offset, uint32_t offset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 4, lane_offset, offset, 0, 0);
}

// lgkmcnt(0) alone.
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

// y = s (c A + alpha B): the sums are exact, and 64 bits here cost nothing
// beside them, so what is left is the rounding to the output's type.
__device__ __forceinline__ float combine(float s, float c, int A, float alpha, int B)
{
    return (float)((double)s * ((double)c * (double)A + (double)alpha * (double)B));
}

}  // namespace bd
