// Product of int8 rows with an int8 base and 1-bit deltas, few tokens
// (bitdelta_linear_int8):
//
//   y[i,r] = s_i (c_r sum_k q[i,k] w[r,k] + alpha_v[r] sum_k q[i,k] sign_v[r,k])
//
// Both sums are of whole numbers and exact in int32 (|sum| <= 131064 * 2^14 <
// 2^31), so they may be cut in any way.  Bound by reading w and the signs.
#include <type_traits>

#include "int8_device.h"
#include "int8_tiles.h"

namespace bd {
namespace {

constexpr int kWaves = 8;         // of a workgroup, each with every eighth range of columns
constexpr int kRange = 512;       // columns a wave takes at a time: 4 blocks of 128

// One workgroup: 16 channels, T blocks of 16 tokens.  A wave loads a range of
// the 16 rows (each instruction 64 contiguous bytes of every row, two of them a
// whole line), of the tokens, and of each variant's signs (64 bytes of every
// row in one load).  Lane group p (lanes 16 p ..) of the four holds, for block b
// of 128 columns, the columns 128 b + 32 p .. + 31: two 16-byte operands of w and
// q, and one dword of signs, which a 4 x 4 transpose over the lane groups brings there.
//
// The tokens are ordered by variant, so a variant meets few token blocks; its
// product is formed for whole blocks and kept for the rows that are its own.
template <int T, bool DELTA, bool ODD>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(T == 4 ? 2 : T == 2 ? 3 : 4)))
void int8_stream(Int8Args a)
{
    __shared__ i32x4 part[kWaves][T][DELTA ? 2 : 1][64];
    __shared__ int32_t token_s[16 * T], variant_s[16 * T];

    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // blocks of tokens next to one another: they read the same rows of w
    const unsigned across = (unsigned)((a.m + 16 * T - 1) / (16 * T));
    const int64_t n0 = (int64_t)(blockIdx.x / across) * 16, K = a.d_in, N = a.d_out, G = K >> 3;
    const int64_t t0 = (int64_t)(blockIdx.x % across) * (16 * T);
    const int count = (int)(a.m - t0 < 16 * T ? a.m - t0 : 16 * T);

    // lane p: the token at place p of the order by variant, and its variant
    int token = lane, variant = 0;
    if (DELTA && a.ids) {
        const int id = lane < count ? a.ids[t0 + lane] : 0x7FFFFFFF;
        const bool known = (unsigned)id < (unsigned)a.n_variants;
        const int key = lane < count ? (known ? id : a.n_variants) : 0x7FFFFFFF;
        int place = 0;
#pragma unroll
        for (int i = 0; i < 16 * T; ++i) {
            const int other = __builtin_amdgcn_readlane(key, i);
            place += other < key || (other == key && i < lane) ? 1 : 0;
        }
        place = lane < 16 * T ? place : lane;
        token = __builtin_amdgcn_ds_permute(place * 4, lane);
        variant = __builtin_amdgcn_ds_permute(place * 4, key);
    }
    if (wave == 0 && lane < 16 * T) {
        token_s[lane] = token;
        variant_s[lane] = variant;
    }
    uint32_t qoff[T];
#pragma unroll
    for (int b = 0; b < T; ++b) {
        const int place = 16 * b + col;
        const int t = __shfl(token, place);
        qoff[b] = place < count ? (uint32_t)((t0 + t) * K) : kInvalidOffset;
    }
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.q, a.m * K), rw = make_rsrc(a.w, N * K);
    // rows past the last one read past the buffer, which gives zeros
    const uint32_t woff = (uint32_t)((n0 + col) * K);
    // Columns k .. k + 15 of a row at byte `off` of a buffer.  No access is
    // partly past a buffer's end: with rows of whole 16 columns none can be,
    // other rows are read by eights.
    const bool eights = ODD && K % 16 != 0;
    auto sixteen = [&](__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t k, auto cache) -> u32x4 {
        if (!eights)
            return __builtin_amdgcn_raw_buffer_load_b128(r, k < K ? off + k : kInvalidOffset, 0, decltype(cache)::value);
        const auto lo = __builtin_amdgcn_raw_buffer_load_b64(r, k < K ? off + k : kInvalidOffset, 0, decltype(cache)::value);
        const auto hi = __builtin_amdgcn_raw_buffer_load_b64(r, k + 8 < K ? off + k + 8 : kInvalidOffset, 0, decltype(cache)::value);
        return (u32x4){lo[0], lo[1], hi[0], hi[1]};
    };

    i32x4 acc[T], accd[T], accx[T];
#pragma unroll
    for (int b = 0; b < T; ++b)
        acc[b] = accd[b] = accx[b] = (i32x4){0, 0, 0, 0};

    for (int64_t k0 = (int64_t)wave * kRange; k0 < K; k0 += kWaves * kRange) {
        u32x4 x[T][8], w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t k = (uint32_t)k0 + (j >> 1) * 128 + quad * 32 + (j & 1) * 16;
            w[j] = sixteen(rw, woff, k, std::integral_constant<int, kStream>{});
            // past the row's end the tokens are zero, whatever the signs' bytes hold there
#pragma unroll
            for (int b = 0; b < T; ++b)
                x[b][j] = sixteen(rq, qoff[b], k, std::integral_constant<int, 0>{});
        }
        // the variants' signs, the next ones loaded ahead
        constexpr int kAhead = 3;
        uint64_t heads = 1;
        if (DELTA && a.ids) {
            const int before = __shfl(variant, lane ? lane - 1 : 0);
            heads = __ballot(lane < count && (lane == 0 || variant != before));
        }
        struct Signs {
            u32x4 s;
            int v, begin, end;
        } ring[kAhead + 1];
        auto fetch = [&](Signs &r) {
            if (!heads) {
                r.begin = r.end = 0;
                return;
            }
            r.begin = __builtin_ctzll(heads);
            heads &= heads - 1;
            r.end = heads ? __builtin_ctzll(heads) : count;
            r.v = __builtin_amdgcn_readlane(variant, r.begin);
            const bool known = (unsigned)r.v < (unsigned)a.n_variants;
            const uint8_t *base = a.signs + (known ? r.v : 0) * N * G;
            // signs may start on any byte: a buffer of whole dwords from the one that holds the first
            const uint32_t slip = ODD ? (uint32_t)((uintptr_t)base & 3) : 0;
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(base - slip, (N * G + slip + 3) & ~(int64_t)3);
            const uint32_t in_row = (uint32_t)(k0 >> 3) + quad * 16;
            const uint32_t at = (uint32_t)((n0 + col) * G) + in_row + slip;
            if (!ODD && k0 + kRange <= K) {
                r.s = __builtin_amdgcn_raw_buffer_load_b128(rs, known ? at : kInvalidOffset, 0, kStream);
                return;
            }
            // the row's end, or rows of any alignment: dword by dword
            uint32_t d[5] = {0, 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < (ODD ? 5 : 4); ++i)
                d[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, known && in_row < G ? (at & ~3u) + 4 * i : kInvalidOffset, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.s[i] = ODD ? __builtin_amdgcn_alignbyte(d[i + 1], d[i], at & 3) : d[i];
        };
        if constexpr (DELTA) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                fetch(ring[i]);
        }
        const u32x4 ones = {0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int b = 0; b < T; ++b) {
                acc[b] = mfma16(x[b][j], w[j], acc[b]);
                if constexpr (DELTA)
                    accx[b] = mfma16(x[b][j], ones, accx[b]);
            }
        if constexpr (DELTA) {
#pragma unroll
            for (int b = 0; b < T; ++b)
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    to_sign_order(x[b][j], x[b][j + 1]);
            bool more = true;
            while (more) {
#pragma unroll
                for (int i = 0; i <= kAhead; ++i) {
                    fetch(ring[(i + kAhead) % (kAhead + 1)]);
                    Signs &r = ring[i];
                    if (r.begin == r.end) {
                        more = false;
                        break;
                    }
                    // dword p of lane group g's sixteen bytes goes to group p's dword g
                    uint32_t e[4] = {r.s[0], r.s[1], r.s[2], r.s[3]};
                    auto swap32 = [](uint32_t &p, uint32_t &q) {
                        const auto o = __builtin_amdgcn_permlane32_swap(p, q, false, false);
                        p = o[0], q = o[1];
                    };
                    auto swap16 = [](uint32_t &p, uint32_t &q) {
                        const auto o = __builtin_amdgcn_permlane16_swap(p, q, false, false);
                        p = o[0], q = o[1];
                    };
                    swap32(e[0], e[2]);
                    swap32(e[1], e[3]);
                    swap16(e[0], e[1]);
                    swap16(e[2], e[3]);
                    i32x4 d[T];
#pragma unroll
                    for (int b = 0; b < T; ++b)
                        d[b] = (i32x4){0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        u32x4 s;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            s[c] = sign_bytes(e[j >> 1], (j & 1) * 4 + c);
#pragma unroll
                        for (int b = 0; b < T; ++b)
                            if (T == 1 || (r.begin < 16 * b + 16 && r.end > 16 * b))
                                d[b] = mfma16(x[b][j], s, d[b]);
                    }
#pragma unroll
                    for (int b = 0; b < T; ++b)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int place = 16 * b + quad * 4 + c;
                            accd[b][c] += place >= r.begin && place < r.end ? d[b][c] : 0;
                        }
                }
            }
        }
    }
#pragma unroll
    for (int b = 0; b < T; ++b) {
        part[wave][b][0][lane] = acc[b];
        if constexpr (DELTA)
            part[wave][b][1][lane] = accd[b] * 2 - accx[b];
    }
    __syncthreads();
    // element e of a token block: lane e / 4's number e % 4, row (lane / 16) * 4 + e % 4, channel lane % 16
    for (int at = threadIdx.x; at < T * 256; at += kWaves * 64) {
        const int b = at >> 8, row = (at >> 4) & 15, ch = at & 15;
        const int from = (row >> 2) * 16 + ch, place = b * 16 + row;
        int A = 0, B = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            A += part[w][b][0][from][row & 3];
            if constexpr (DELTA)
                B += part[w][b][1][from][row & 3];
        }
        const int64_t n = n0 + ch;
        if (place >= count || n >= N)
            continue;
        const int64_t t = t0 + token_s[place];
        const int v = DELTA ? variant_s[place] : 0;
        float y = 0.0f;
        if (!DELTA || (unsigned)v < (unsigned)a.n_variants)
            y = combine(a.q_scale[t], a.w_scale[n], A, DELTA ? a.alpha[a.per_matrix ? v : v * N + n] : 0.0f, B);
        if (a.f32)
            static_cast<float *>(a.y)[t * N + n] = y;
        else
            static_cast<uint16_t *>(a.y)[t * N + n] = to_bf16(y);
    }
}

template <int T>
hipError_t stream(const Int8Args &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.d_out + 15) / 16 * ((a.m + 16 * T - 1) / (16 * T))));
    const bool odd = a.d_in % 32 != 0 || ((uintptr_t)a.signs & 3) != 0;
    if (!a.signs) {
        if (a.d_in % 16)
            int8_stream<T, false, true><<<grid, kWaves * 64, 0, s>>>(a);
        else
            int8_stream<T, false, false><<<grid, kWaves * 64, 0, s>>>(a);
    } else if (odd)
        int8_stream<T, true, true><<<grid, kWaves * 64, 0, s>>>(a);
    else
        int8_stream<T, true, false><<<grid, kWaves * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// From this many tokens on the tiles are used.
constexpr int64_t kTilesFrom = 65;

size_t linear_int8_workspace_bytes(int64_t m, int32_t n_variants, int64_t, int64_t)
{
    return m < kTilesFrom ? 0 : int8_tiles_workspace_bytes(m, n_variants);
}

hipError_t launch_linear_int8(const Int8Args &a, void *workspace, hipStream_t s)
{
    if (a.m >= kTilesFrom && int8_tiles_take(a))
        return launch_int8_tiles(a, workspace, s);
    return a.m <= 16 ? stream<1>(a, s) : a.m <= 32 ? stream<2>(a, s) : stream<4>(a, s);
}

}  // namespace bd
