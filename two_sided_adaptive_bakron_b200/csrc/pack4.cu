// pack4.cu -- bakron_pack4 / bakron_unpack4: the 4-bit layout of a rounded layer.
//
// Bound by bytes: a code read (written) once, half a byte written (read). One warp per pair of column
// tiles, 16 rows x 128 columns: on the side of the codes whole 128-byte lines, 16 bytes a lane and
// four lines at once; on the packed side 512 bytes a tile, 16 a lane. The two orders meet in shared
// memory (rows 160 bytes apart, so that neither side's accesses conflict). The grid steps are moved
// by the blocks behind the tiles' blocks.
//
// Measured, 28672 x 8192: 59.8 us there (6.1 TB/s), 61.3 back (6.0); 4096 x 4096 6.8 and 6.5.
#include "lowp.cuh"
#include "pack4.cuh"

namespace bakron {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPitch = 160;          // bytes between a pair's rows in shared memory

// 8 codes, the first in the lowest byte of lo -> one word of the layout.
__device__ __forceinline__ uint32_t to_word(uint2 c) {
    const uint32_t m = (c.x & 0x0F0F0F0Fu) | ((c.y & 0x0F0F0F0Fu) << 4);
    return __byte_perm(m, 0, 0x3120);
}

// Sign extension of the low nibble of every byte.
__device__ __forceinline__ uint32_t extend(uint32_t x) { return x | ((x & 0x08080808u) * 0x1Eu); }

// Whether a byte of x is outside 0..15 (kUnsigned) or -8..7.
template <bool kUnsigned>
__device__ __forceinline__ bool out_of_range(uint32_t x) {
    if (kUnsigned) return (x & 0xF0F0F0F0u) != 0;
    return extend(x & 0x0F0F0F0Fu) != x;
}

// What a warp works on: a row tile and a pair of column tiles.
struct Pair {
    int rt, kt;
    bool two;            // the second tile exists
    __device__ __forceinline__ Pair(const Pack4Shape& P, size_t pair) {
        const int per_row = (P.kt + 1) / 2;
        rt = (int)(pair / per_row), kt = (int)(pair % per_row) * 2, two = kt + 1 < P.kt;
    }
};
// Bytes of one access to the rows of the codes: 16, 4 or 1.
int access_bytes(const int8_t* codes, int64_t ldc) {
    return ldc % 16 == 0 && aligned_to(codes, 16) ? 16 : ldc % 4 == 0 && aligned_to(codes, 4) ? 4 : 1;
}
__host__ __device__ inline size_t pairs(const Pack4Shape& P) { return (size_t)P.mt * ((P.kt + 1) / 2); }

template <bool kUnsigned>
__global__ void __launch_bounds__(kThreads)
pack4_kernel(const int8_t* __restrict__ codes, int64_t ldc, const float* __restrict__ scales,
             int m, int n, int G, int wide, unsigned tile_blocks, uint8_t* __restrict__ packed,
             int* __restrict__ status) {
    __shared__ __align__(16) char smem[kWarps][16 * kPitch];
    const Pack4Shape P(m, n, G);
    if (blockIdx.x >= tile_blocks) {
        const size_t e = (size_t)(blockIdx.x - tile_blocks) * kThreads + threadIdx.x;
        if (e >= P.step_count()) return;
        const int r = (int)(e % 16), row = r / 2 + 8 * (r % 2);
        const size_t tg = e / 16, i = tg / G * 16 + row;
        reinterpret_cast<float*>(packed + P.code_bytes())[e] =
            i < (size_t)m ? scales[i * G + tg % G] : 0.f;
        return;
    }
    const size_t pair = (size_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (pair >= pairs(P)) return;
    const Pair W(P, pair);
    const int lane = threadIdx.x & 31;
    char* s = smem[threadIdx.x / 32];
    uint4 v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int i = W.rt * 16 + 4 * p + lane / 8, j = W.kt * 64 + 16 * (lane % 8);
        v[p] = make_uint4(0, 0, 0, 0);
        if (i < m && j < n) {
            const int8_t* src = codes + (int64_t)i * ldc + j;
            if (wide == 16 && j + 16 <= n) {
                v[p] = *reinterpret_cast<const uint4*>(src);
            } else if (wide >= 4 && j + 16 <= n) {
                const uint32_t* u = reinterpret_cast<const uint32_t*>(src);
                v[p] = make_uint4(u[0], u[1], u[2], u[3]);
            } else {
                __align__(16) int8_t e[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) e[c] = j + c < n ? src[c] : (int8_t)0;
                v[p] = *reinterpret_cast<const uint4*>(e);
            }
        }
    }
    bool bad = false;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        bad |= out_of_range<kUnsigned>(v[p].x) || out_of_range<kUnsigned>(v[p].y) ||
               out_of_range<kUnsigned>(v[p].z) || out_of_range<kUnsigned>(v[p].w);
        *reinterpret_cast<uint4*>(s + (4 * p + lane / 8) * kPitch + 16 * (lane % 8)) = v[p];
    }
    __syncwarp();
    uint4* out = reinterpret_cast<uint4*>(packed) + ((size_t)W.rt * P.kt + W.kt) * 32 + lane;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t w[4];
#pragma unroll
        for (int p = 0; p < 4; ++p)
            w[p] = to_word(*reinterpret_cast<const uint2*>(
                s + (lane / 4 + 8 * (p & 1)) * kPitch + 64 * u + 32 * (p >> 1) + 8 * (lane % 4)));
        if (u == 0 || W.two) out[32 * u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (bad) set_status(status, BAKRON_ERR_INVALID_ARG);
}

template <bool kUnsigned>
__global__ void __launch_bounds__(kThreads)
unpack4_kernel(const uint8_t* __restrict__ packed, int m, int n, int G, int wide,
               unsigned tile_blocks, int8_t* __restrict__ codes, int64_t ldc,
               float* __restrict__ scales) {
    __shared__ __align__(16) char smem[kWarps][16 * kPitch];
    const Pack4Shape P(m, n, G);
    if (blockIdx.x >= tile_blocks) {
        const size_t e = (size_t)(blockIdx.x - tile_blocks) * kThreads + threadIdx.x;
        if (e >= P.step_count()) return;
        const int r = (int)(e % 16), row = r / 2 + 8 * (r % 2);
        const size_t tg = e / 16, i = tg / G * 16 + row;
        if (i < (size_t)m)
            scales[i * G + tg % G] = reinterpret_cast<const float*>(packed + P.code_bytes())[e];
        return;
    }
    const size_t pair = (size_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (pair >= pairs(P)) return;
    const Pair W(P, pair);
    const int lane = threadIdx.x & 31;
    char* s = smem[threadIdx.x / 32];
    const uint4* in = reinterpret_cast<const uint4*>(packed) + ((size_t)W.rt * P.kt + W.kt) * 32 + lane;
    uint4 v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) v[u] = u == 0 || W.two ? in[32 * u] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t x = __byte_perm(w[p], 0, 0x3120);   // its own inverse
            uint2 c = make_uint2(x & 0x0F0F0F0Fu, (x >> 4) & 0x0F0F0F0Fu);
            if (!kUnsigned) c = make_uint2(extend(c.x), extend(c.y));
            *reinterpret_cast<uint2*>(s + (lane / 4 + 8 * (p & 1)) * kPitch + 64 * u +
                                      32 * (p >> 1) + 8 * (lane % 4)) = c;
        }
    }
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int r = 4 * p + lane / 8;
        const int i = W.rt * 16 + r, j = W.kt * 64 + 16 * (lane % 8);
        if (i >= m || j >= n) continue;
        const uint4 c = *reinterpret_cast<const uint4*>(s + r * kPitch + 16 * (lane % 8));
        int8_t* dst = codes + (int64_t)i * ldc + j;
        if (wide == 16 && j + 16 <= n) {
            *reinterpret_cast<uint4*>(dst) = c;
        } else if (wide >= 4 && j + 16 <= n) {
            uint32_t* u = reinterpret_cast<uint32_t*>(dst);
            u[0] = c.x, u[1] = c.y, u[2] = c.z, u[3] = c.w;
        } else {
            __align__(16) int8_t e[16];
            *reinterpret_cast<uint4*>(e) = c;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (j + k < n) dst[k] = e[k];
        }
    }
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" size_t bakron_pack4_bytes(int m, int n, int group_size) {
    if (!pack4_ok(m, n, group_size)) return 0;
    return Pack4Shape(m, n, group_count(group_size, n)).bytes();
}

extern "C" int bakron_pack4(const int8_t* codes, int64_t ldc, const float* scales, int m, int n,
                            int group_size, int unsigned_codes, void* packed, int* dev_status,
                            void* stream) {
    if (!pack4_ok(m, n, group_size) || ldc < n || unsigned_codes < 0 || unsigned_codes > 1 ||
        !codes || !scales || !packed || !aligned_to(packed, 16) || !dev_status)
        return BAKRON_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Pack4Shape P(m, n, group_count(group_size, n));
    const unsigned tb = (unsigned)((pairs(P) + kWarps - 1) / kWarps);
    const unsigned sb = (unsigned)((P.step_count() + kThreads - 1) / kThreads);
    const int wide = access_bytes(codes, ldc);
    auto kern = unsigned_codes ? pack4_kernel<true> : pack4_kernel<false>;
    kern<<<tb + sb, kThreads, 0, st>>>(codes, ldc, scales, m, n, P.groups, wide, tb,
                                       static_cast<uint8_t*>(packed), dev_status);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}

extern "C" int bakron_unpack4(const void* packed, int m, int n, int group_size,
                              int unsigned_codes, int8_t* codes, int64_t ldc, float* scales,
                              void* stream) {
    if (!pack4_ok(m, n, group_size) || ldc < n || unsigned_codes < 0 || unsigned_codes > 1 ||
        !codes || !scales || !packed || !aligned_to(packed, 16))
        return BAKRON_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Pack4Shape P(m, n, group_count(group_size, n));
    const unsigned tb = (unsigned)((pairs(P) + kWarps - 1) / kWarps);
    const unsigned sb = (unsigned)((P.step_count() + kThreads - 1) / kThreads);
    const int wide = access_bytes(codes, ldc);
    auto kern = unsigned_codes ? unpack4_kernel<true> : unpack4_kernel<false>;
    kern<<<tb + sb, kThreads, 0, st>>>(static_cast<const uint8_t*>(packed), m, n, P.groups, wide,
                                       tb, codes, ldc, scales);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}
