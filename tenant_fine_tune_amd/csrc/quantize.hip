// Rows as int8 numbers and a scale (bitdelta_quantize_int8).
//
//   s = fl32(max |x| / 127),  q = round(x / s), ties to even
//
// One workgroup per row keeps the row in registers between the maximum and the
// quotients: every input is read once, memory bound.  2049 x 28672 bf16 44 us,
// 4.0 TB/s; 4 x 8192 3.9 us, a launch and one trip to memory.  Rows too wide for that
// (above 32768) are read twice: 1024 x 131064 bf16 112 us (held whole, with spills, 146).
#include "bd_device.h"
#include "decoder_launch.h"
#include "int8_launch.h"

namespace bd {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight consecutive elements as loaded, of which n (0..8) exist, the others zero.
template <typename T>
struct Eight;

template <>
struct Eight<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t *p, int n)
    {
        w = (u32x4){0, 0, 0, 0};
        if (n == 8) {
            w = __builtin_nontemporal_load(reinterpret_cast<const u32x4a2 *>(p));
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? hi_f32(w[i >> 1]) : lo_f32(w[i >> 1]); }
};

template <>
struct Eight<float> {
    u32x4 a, b;
    __device__ __forceinline__ void load(const float *p, int n)
    {
        a = b = (u32x4){0, 0, 0, 0};
        if (n == 8) {
            a = __builtin_nontemporal_load(reinterpret_cast<const u32x4a4 *>(p));
            b = __builtin_nontemporal_load(reinterpret_cast<const u32x4a4 *>(p + 4));
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                (i < 4 ? a : b)[i & 3] = __float_as_uint(p[i]);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i < 4 ? a[i] : b[i - 4]); }
};

// Largest value over the workgroup; every thread gets it.
__device__ __forceinline__ uint32_t max_all(uint32_t v, uint32_t *part)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o));
    const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
    if (waves == 1)
        return v;
    if (lane == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lane < waves ? part[lane] : 0;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return __shfl((int)v, 0);
}

constexpr float kTinyScale = 0x1p-100f;

// x / s to the nearest whole number, the quotient taken exactly.  t = rint(x *
// fl(1/s)) is at most one off; what is left of x, x - t s, is exact in fp32 (at
// most s in size, a multiple of half a step of s), and says whether it is.
__device__ __forceinline__ float nearest(float x, float s, float inv)
{
    float t = rintf(x * inv);
    const float left = fmaf(-t, s, x), half = 0.5f * s;
    if (fabsf(left) >= half) {
        const bool odd = (int)t & 1;
        if (left > half || (left == half && odd))
            t += 1.0f;
        else if (left < -half || (left == -half && odd))
            t -= 1.0f;
    }
    return t;
}

// The row's scale from the bits of its largest magnitude (an infinity is above every
// number, a NaN above that), and its quotients.
struct Quotients {
    float s, inv;
    __device__ __forceinline__ explicit Quotients(uint32_t top)
    {
        s = top < 0x7F800000u ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7FC00000u);
        inv = 1.0f / s;
    }
    // Eight numbers, n of which exist.
    template <typename T>
    __device__ __forceinline__ void store(const Eight<T> &v, int8_t *p, int n) const
    {
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float t;
            if (s < kTinyScale)   // 1/s may not exist in fp32; of 24-bit numbers the fp64 quotient rounds to a half only where it is one
                t = (float)rint((double)v.get(j) / (double)s);
            else
                t = nearest(v.get(j), s, inv);
            b[j] = s > 0.0f ? (uint32_t)(int)fminf(fmaxf(t, -127.0f), 127.0f) & 0xFFu : 0u;
        }
        if (n == 8) {
            typedef uint32_t u32x2a1 __attribute__((ext_vector_type(2), aligned(1)));
            *reinterpret_cast<u32x2a1 *>(p) = (u32x2a1){b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24,
                                                        b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n)
                    p[j] = (int8_t)b[j];
        }
    }
};

// C groups of eight columns a thread and turn, the row in one turn unless WIDE: then
// it is read a second time for the quotients.
template <int C, bool WIDE, typename T>
__global__ __launch_bounds__(1024) void quantize_rows(const T *__restrict__ x, int64_t stride, int64_t m, int d,
                                                      int8_t *__restrict__ q, float *__restrict__ scale)
{
    __shared__ uint32_t part[16];
    const int64_t i = blockIdx.y * kTokensAcross + blockIdx.x;
    if (i >= m)
        return;
    const int step = blockDim.x * 8, at0 = threadIdx.x * 8;
    const T *row = x + i * stride;
    int8_t *out = q + i * d;
    Eight<T> v[C];
    uint32_t top = 0;
    auto load = [&](int from) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            v[c].load(row + from + at0 + c * step, min(max(d - from - at0 - c * step, 0), 8));
    };
    int from = 0;
    do {
        load(from);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, __float_as_uint(v[c].get(j)) & 0x7FFFFFFFu);
        from += C * step;
    } while (WIDE && from < d);
    const Quotients quotients(max_all(top, part));
    if (threadIdx.x == 0)
        scale[i] = quotients.s;
    // the last turn's columns are still here
    do {
        from -= C * step;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = from + at0 + c * step;
            quotients.store(v[c], out + at, min(max(d - at, 0), 8));
        }
        if (WIDE && from > 0)
            load(from - C * step);
    } while (WIDE && from > 0);
}

template <int C, bool WIDE, typename T>
void start(const void *x, int64_t stride, int64_t m, int64_t d, int8_t *q, float *scale, hipStream_t s)
{
    const int threads = WIDE ? 1024 : (int)((d + 512 * C - 1) / (512 * C)) * 64;
    const dim3 grid((unsigned)(m < kTokensAcross ? m : kTokensAcross), (unsigned)((m + kTokensAcross - 1) / kTokensAcross));
    quantize_rows<C, WIDE, T><<<grid, threads, 0, s>>>(static_cast<const T *>(x), stride, m, (int)d, q, scale);
}

template <typename T>
void start(const void *x, int64_t stride, int64_t m, int64_t d, int8_t *q, float *scale, hipStream_t s)
{
    // as many waves as the row has groups of 512 C columns, at most 16
    if (d <= 2048)
        start<1, false, T>(x, stride, m, d, q, scale, s);
    else if (d <= 16384)
        start<2, false, T>(x, stride, m, d, q, scale, s);
    else if (d <= 32768)
        start<4, false, T>(x, stride, m, d, q, scale, s);
    else
        start<4, true, T>(x, stride, m, d, q, scale, s);
}

}  // namespace

hipError_t launch_quantize_int8(const void *x, int64_t x_stride, bool f32, int64_t m, int64_t d, int8_t *q,
                                float *scale, hipStream_t s)
{
    if (f32)
        start<float>(x, x_stride, m, d, q, scale, s);
    else
        start<uint16_t>(x, x_stride, m, d, q, scale, s);
    return hipGetLastError();
}

}  // namespace bd
