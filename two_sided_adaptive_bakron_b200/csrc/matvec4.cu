// matvec4.cu -- bakron_matvec4: a layer in the 4-bit layout times the activations of a few tokens.
//
//   y[t][i] = sum_j s[i][g(j)] v(code_ij) x[t][j]
//
// One block per row tile (16 rows) and 4 tokens; its warps take the tile's column tiles in turn.
// Lane 4 g + t of a warp holds rows g and g + 8 of 16 columns a tile; the lanes of one g and the
// warps are summed at the end, in a fixed order.
#include <cmath>

#include "pack4.cuh"

namespace bakron {
namespace {

constexpr int kThreads = 128;
constexpr int kTok = 4;

struct Book { float v[16]; };

template <class X, class Y>
__global__ void __launch_bounds__(kThreads)
matvec4_kernel(const uint8_t* __restrict__ packed, int m, int n, int G, int gs, Book book,
               const X* __restrict__ x, int64_t ldx, const float* __restrict__ xs, int Gx, int gx,
               int tokens, Y* __restrict__ y, int64_t ldy) {
    __shared__ float red[kThreads / 32][16][kTok];
    __shared__ float lut[16];
    const Pack4Shape P(m, n, G);
    const int rt = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int g = lane / 4, t = lane % 4;
    const int t0 = blockIdx.y * kTok;
    if (threadIdx.x < 16) lut[threadIdx.x] = book.v[threadIdx.x];
    __syncthreads();
    float acc[2][kTok] = {};
    const uint4* tiles = reinterpret_cast<const uint4*>(packed) + (size_t)rt * P.kt * 32;
    const float* steps = reinterpret_cast<const float*>(packed + P.code_bytes());
    for (int kt = warp; kt < P.kt; kt += kThreads / 32) {
        const uint4 v = tiles[(size_t)kt * 32 + lane];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j0 = kt * 64 + 32 * h + 8 * t;
            if (j0 >= n) continue;
            const float* s = steps + (((size_t)rt * G + j0 / gs) * 8 + g) * 2;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (j0 + c >= n) break;
                const int nib = ((c & 1) << 2) | (c & 2) | (c >> 2);
                const float a = s[0] * lut[(w[2 * h] >> (4 * nib)) & 15];
                const float b = s[1] * lut[(w[2 * h + 1] >> (4 * nib)) & 15];
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
                    if (t0 + k >= tokens) break;
                    float xv = to_f32(x[(int64_t)(t0 + k) * ldx + j0 + c]);
                    if (xs) xv *= xs[(size_t)(t0 + k) * Gx + (j0 + c) / gx];
                    acc[0][k] = fmaf(a, xv, acc[0][k]);
                    acc[1][k] = fmaf(b, xv, acc[1][k]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            float a = acc[r][k];
            a += __shfl_xor_sync(0xffffffffu, a, 1);
            a += __shfl_xor_sync(0xffffffffu, a, 2);
            if (t == 0) red[warp][g + 8 * r][k] = a;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * kTok; e += kThreads) {
        const int r = e % 16, k = e / 16;
        const int64_t i = (int64_t)rt * 16 + r;
        if (i >= m || t0 + k >= tokens) continue;
        float a = 0.f;
        for (int q = 0; q < kThreads / 32; ++q) a += red[q][r][k];
        from_f32(a, y[(int64_t)(t0 + k) * ldy + i]);
    }
}

struct Args {
    const uint8_t* packed; int m, n, G, gs; Book book;
    const void* x; int64_t ldx; const float* xs; int Gx, gx, tokens; void* y; int64_t ldy;
    cudaStream_t st;
};

template <int XD, int YD>
int launch(const Args& a) {
    using X = typename Elem<XD>::T;
    using Y = typename Elem<YD>::T;
    matvec4_kernel<X, Y><<<dim3((a.m + 15) / 16, (a.tokens + kTok - 1) / kTok), kThreads, 0,
                           a.st>>>(
        a.packed, a.m, a.n, a.G, a.gs, a.book, static_cast<const X*>(a.x), a.ldx, a.xs, a.Gx,
        a.gx, a.tokens, static_cast<Y*>(a.y), a.ldy);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}

template <int XD>
int launch_y(const Args& a, int y_dtype) {
    switch (y_dtype) {
        case BAKRON_F32: return launch<XD, BAKRON_F32>(a);
        case BAKRON_F16: return launch<XD, BAKRON_F16>(a);
        default: return launch<XD, BAKRON_BF16>(a);
    }
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" int bakron_matvec4(const void* packed, int m, int n, int group_size,
                              const float* codebook, int bits, const void* x, int x_dtype,
                              int64_t ldx, const float* x_scales, int x_group_size, int tokens,
                              void* y, int y_dtype, int64_t ldy, void* stream) {
    const bool i8 = x_dtype == BAKRON_I8;
    if (!pack4_ok(m, n, group_size) || tokens < 0 || tokens > 65535 ||
        (!i8 && !float_dtype(x_dtype)) || !float_dtype(y_dtype) || ldx < n || ldy < m ||
        (i8 && !group_ok(x_group_size, n)) || (codebook && (bits < 1 || bits > 4)))
        return BAKRON_ERR_INVALID_ARG;
    if (codebook)
        for (int k = 0; k < (1 << bits); ++k)
            if (!std::isfinite(codebook[k])) return BAKRON_ERR_INVALID_ARG;
    if (tokens == 0) return BAKRON_OK;
    if (!packed || !x || !y || i8 != (x_scales != nullptr) || !aligned_to(packed, 16) ||
        !aligned_to(x, dtype_bytes(x_dtype)) || !aligned_to(y, dtype_bytes(y_dtype)))
        return BAKRON_ERR_INVALID_ARG;
    Args a{static_cast<const uint8_t*>(packed), m, n, group_count(group_size, n),
           group_size < n ? group_size : n, {}, x, ldx, x_scales,
           i8 ? group_count(x_group_size, n) : 1, i8 && x_group_size < n ? x_group_size : n, tokens,
           y, ldy, static_cast<cudaStream_t>(stream)};
    for (int k = 0; k < 16; ++k) {
        if (!codebook) {
            a.book.v[k] = (float)(k < 8 ? k : k - 16);
        } else {
            a.book.v[k] = k < (1 << bits) ? codebook[k] : 0.f;
        }
    }
    switch (x_dtype) {
        case BAKRON_F32: return launch_y<BAKRON_F32>(a, y_dtype);
        case BAKRON_F16: return launch_y<BAKRON_F16>(a, y_dtype);
        case BAKRON_BF16: return launch_y<BAKRON_BF16>(a, y_dtype);
        default: return launch_y<BAKRON_I8>(a, y_dtype);
    }
}
