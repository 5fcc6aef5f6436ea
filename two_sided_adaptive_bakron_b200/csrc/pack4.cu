// pack4.cu -- bakron_pack4 / bakron_unpack4: the 4-bit layout of a rounded layer.
//
// One warp per tile of 16 rows x 64 columns (512 bytes of the layout). Lane 4 g + t holds the
// four words of rows g and g + 8, columns 8 t and 32 + 8 t, which are its 16 bytes of the tile, so
// the packed side is one coalesced 16-byte access a lane; the code side is four 8-byte accesses,
// each a run of 32 bytes a row. Bound by bytes: a code is read (written) once, half a byte
// written (read). The grid steps are moved by the blocks behind the tiles' blocks.
#include "lowp.cuh"
#include "pack4.cuh"

namespace bakron {
namespace {

constexpr int kThreads = 256;

// 8 codes, the first in the lowest byte of lo -> one word of the layout.
__device__ __forceinline__ uint32_t to_word(uint32_t lo, uint32_t hi) {
    const uint32_t m = (lo & 0x0F0F0F0Fu) | ((hi & 0x0F0F0F0Fu) << 4);
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

template <bool kUnsigned>
__global__ void __launch_bounds__(kThreads)
pack4_kernel(const int8_t* __restrict__ codes, int64_t ldc, const float* __restrict__ scales,
             int m, int n, int G, int wide, unsigned tile_blocks, uint8_t* __restrict__ packed,
             int* __restrict__ status) {
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
    const size_t tile = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (tile >= P.tiles()) return;
    const int lane = threadIdx.x & 31;
    const int i0 = (int)(tile / P.kt) * 16 + lane / 4;
    const int j0 = (int)(tile % P.kt) * 64 + 8 * (lane % 4);
    uint32_t w[4];
    bool bad = false;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int i = i0 + 8 * (p & 1), j = j0 + 32 * (p >> 1);
        uint32_t lo = 0, hi = 0;
        if (i < m) {
            const int8_t* src = codes + (int64_t)i * ldc + j;
            if (wide && j + 8 <= n) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                lo = v.x;
                hi = v.y;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (j + c < n) lo |= (uint32_t)(uint8_t)src[c] << (8 * c);
                    if (j + 4 + c < n) hi |= (uint32_t)(uint8_t)src[4 + c] << (8 * c);
                }
            }
        }
        bad |= out_of_range<kUnsigned>(lo) || out_of_range<kUnsigned>(hi);
        w[p] = to_word(lo, hi);
    }
    reinterpret_cast<uint4*>(packed)[tile * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
    if (bad) set_status(status, BAKRON_ERR_INVALID_ARG);
}

template <bool kUnsigned>
__global__ void __launch_bounds__(kThreads)
unpack4_kernel(const uint8_t* __restrict__ packed, int m, int n, int G, int wide,
               unsigned tile_blocks, int8_t* __restrict__ codes, int64_t ldc,
               float* __restrict__ scales) {
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
    const size_t tile = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (tile >= P.tiles()) return;
    const int lane = threadIdx.x & 31;
    const int i0 = (int)(tile / P.kt) * 16 + lane / 4;
    const int j0 = (int)(tile % P.kt) * 64 + 8 * (lane % 4);
    const uint4 v = reinterpret_cast<const uint4*>(packed)[tile * 32 + lane];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int i = i0 + 8 * (p & 1), j = j0 + 32 * (p >> 1);
        if (i >= m) continue;
        const uint32_t u = __byte_perm(w[p], 0, 0x3120);   // its own inverse
        uint32_t lo = u & 0x0F0F0F0Fu, hi = (u >> 4) & 0x0F0F0F0Fu;
        if (!kUnsigned) lo = extend(lo), hi = extend(hi);
        int8_t* dst = codes + (int64_t)i * ldc + j;
        if (wide && j + 8 <= n) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (j + c < n) dst[c] = (int8_t)(lo >> (8 * c));
                if (j + 4 + c < n) dst[4 + c] = (int8_t)(hi >> (8 * c));
            }
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
    const unsigned tb = (unsigned)((P.tiles() + kThreads / 32 - 1) / (kThreads / 32));
    const unsigned sb = (unsigned)((P.step_count() + kThreads - 1) / kThreads);
    const int wide = ldc % 8 == 0 && aligned_to(codes, 8);
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
    const unsigned tb = (unsigned)((P.tiles() + kThreads / 32 - 1) / (kThreads / 32));
    const unsigned sb = (unsigned)((P.step_count() + kThreads - 1) / kThreads);
    const int wide = ldc % 8 == 0 && aligned_to(codes, 8);
    auto kern = unsigned_codes ? unpack4_kernel<true> : unpack4_kernel<false>;
    kern<<<tb + sb, kThreads, 0, st>>>(static_cast<const uint8_t*>(packed), m, n, P.groups, wide,
                                       tb, codes, ldc, scales);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}
