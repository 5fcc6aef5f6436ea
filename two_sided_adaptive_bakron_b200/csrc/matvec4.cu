// matvec4.cu -- bakron_matvec4: a layer in the 4-bit layout times the activations of a few tokens.
//
//   y[t][i] = sum_j s[i][g(j)] v(code_ij) x[t][j]
//
// Bound by the bytes of the layer (half a byte a weight: 4 operations a byte for one token, 128 for
// 32, where HBM pays for 250 tensor-core operations a byte), so everything else has to cost less
// than the loads. Unpacking dominates: a weight may take about 2.7 instruction slots of a lane at
// the full rate of HBM (148 SMs x 128 lanes x 1.9 GHz / (2 x 6465e9 weights/s)), and a
// multiply-add on the CUDA cores would need an unpacked fp32 factor and one instruction a weight
// and token. The legacy tensor path (mma.sync m16n8k16 / k32) takes both factors in 16 or 8 bits
// from registers and multiplies 8 columns at once: one token leaves most of it idle, eight cost the
// same. (tcgen05.mma takes them from shared or tensor memory, where they would have to be put first, one
// more write and read of every weight for products that are not what bounds a few tokens.)
//
//   * A warp owns a row tile (16 rows) and a slice of the columns. Each lane's 16 bytes of a 512-byte
//     tile are its own fragments of four m16n8k16 (two m16n8k32) products. A warp copies its tiles
//     and their steps into a ring of its own in shared memory with cp.async, a stage of eight tiles
//     ahead of the one in use: nothing waits for another warp, and no
//     registers hold what is on its way.
//   * The codes become f16 or bf16 by setting the exponent bits around them (1024 + code and
//     128 + code are exact) and one subtraction a pair; int8 by masking: a code in the upper half of
//     its byte is 16 times the code. fp32 activations are split in three bf16 parts of 8 bits, which
//     stand in three columns of the tensor tile, so their products are exact too.
//   * Codebook entries come in pairs from a table in shared memory that is indexed by a byte of two
//     codes and has one copy a lane (bank), so the reads never conflict; an entry is held as two
//     16-bit parts (three for fp32 activations, and for bf16 ones with an fp32 result), each multiplied
//     on its own.
//   * Products are summed over 64 (32) columns in the tensor core's fp32 (int8: exactly, in int32),
//     then scaled and added in fp32 round-to-nearest.
//   * A cluster's blocks take slices of the columns for the same rows and add their sums through
//     distributed shared memory in rank order: no atomics, the same bits every time.
//
// Measured, 28672 x 8192, group 128 (19.3 us at the measured copy rate): one token of bf16 29.1, fp16
// 26.5, int8 25.1 (5.0 TB/s), fp32 32.2 us; 8 bf16 tokens 32.5, 16 tokens 45.5, 32 tokens 97.2; with a
// codebook 50 to 52 (fp32 70, fp32 results of bf16 64), where the table's reads fill shared memory's
// data path. With four product tiles most instantiations spill 12 to 72 bytes a thread (128 registers).
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "bakron_internal.h"
#include "pack4.cuh"
#include "tcgemm_host.cuh"

namespace bakron {
namespace {

namespace cg = cooperative_groups;

constexpr int kStages = 2;
// Shared memory of a block: static arrays (128 bytes at most) and the dynamic part together.
constexpr size_t kSmemLimit = 227 * 1024, kStaticSmem = 128;

// kBf16Wide: bf16 activations with a codebook and an fp32 result, which would show entries of 16 bits.
enum Kind { kF16, kBf16, kF32, kI8, kF16Book, kBf16Book, kBf16Wide, kF32Book };
constexpr bool is_book(int k) { return k >= kF16Book; }
constexpr int planes(int k) { return k >= kBf16Wide ? 3 : 2; }
constexpr bool is_split(int k) { return k == kF32 || k == kF32Book; }   // fp32 activations
constexpr bool is_half(int k) { return k == kF16 || k == kF16Book; }
// tokens in one 8-column tile of the product, staged rows a token
constexpr int tile_tokens(int k) { return is_split(k) ? 2 : 8; }
constexpr int token_rows(int k) { return is_split(k) ? 3 : 1; }

// Stages, warps of a block and blocks of an SM: 16 warps an SM, which share one table of codebook
// pairs (64 to 96 KB) where there is one. Without one, blocks of 8 warps leave room for activations:
// 16 tokens of bf16, 28672 x 8192: 45.4 us, with 16 warps a block 54.4.
constexpr int batch_of(int k) { return is_book(k) ? 4 : 8; }   // column tiles of a stage
constexpr int warps_of(int k) { return is_book(k) ? 16 : 8; }
constexpr int blocks_of(int k) { return 16 / warps_of(k); }

struct Book { uint32_t part[3][16]; };   // 16-bit parts of the entries (host-made)

struct Args {
    const uint8_t* packed; int m, n, G, gs;
    const void* x; int x_dtype; int64_t ldx; const float* xs; int Gx, gx;
    int tokens; void* y; int y_dtype; int64_t ldy;
    int slice;               // column tiles of a block
    int batch_groups;        // groups that kBatch tiles may touch
    int step_shift;          // kPerTile: column tile u of a batch takes step u >> step_shift
    int batch_gq, batch_gr;  // columns of kBatch tiles in whole groups and the rest
    int clusters;            // the row tiles are dealt out over so many clusters of blocks
    int tiles_each, tiles_rest;   // so many row tiles each, and one more for the first few
    int max_tiles;           // the most that one of them gets
    int chunk;               // tokens of a block
    int pitch;               // bytes between staged rows of x
    float out1, out2;        // powers of two for the result
    Book book;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Copies 16 bytes, or fills them with zeros.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d = a b + c
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1, const int (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]),
          "r"(c[2]), "r"(c[3]));
}

// (w & mask) ^ bits
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}

// The 8 codes of a word as four f16 pairs: columns (0, 1), (2, 3), (4, 5), (6, 7). Integers become
// floating point by setting exponent bits around them, as published by Kim et al., 2022 ("Who Says
// Elephants Can't Run"): the xor turns the two's complement nibble into code + 8 under the exponent
// of 1024 (or 64 for the upper nibble, with the product by 1/16).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&p)[4]) {
    const __half2 c0 = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));
    const __half2 c1 = __floats2half2_rn(-72.f, -72.f), r16 = __floats2half2_rn(0.0625f, 0.0625f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t u = q & 1 ? w >> 8 : w;
        const uint32_t v = q & 2 ? and_xor(u, 0x00F000F0u, 0x64806480u)
                                 : and_xor(u, 0x000F000Fu, 0x64086408u);
        __half2 h = *reinterpret_cast<const __half2*>(&v);
        h = q & 2 ? __hfma2(h, r16, c1) : __hsub2(h, c0);
        p[q] = *reinterpret_cast<uint32_t*>(&h);
    }
}
// The same in bf16, which holds 128 + (code + 8) exactly.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t (&p)[4]) {
    const __nv_bfloat162 c = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int nib = (q & 1) * 2 + (q >> 1);
        const uint32_t v = and_xor(w >> (4 * nib), 0x000F000Fu, 0x43084308u);
        const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), c);
        p[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
}

// 8 activations of a token (zeros from `have` on) as raw values of type X.
template <class X>
__device__ __forceinline__ void load8(const X* src, int have, bool wide, X (&v)[8]) {
    if (wide && have >= 8) {
        using V = typename std::conditional<sizeof(X) == 1, uint2, uint4>::type;
        constexpr int per = sizeof(V) / sizeof(X);
#pragma unroll
        for (int q = 0; q < 8 / per; ++q)
            reinterpret_cast<V*>(v)[q] = reinterpret_cast<const V*>(src)[q];
    } else {
        memset(v, 0, sizeof v);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < have) v[c] = src[c];
    }
}

// An fp32 value as three bf16 parts of 8 bits each, cut off, which add up to it exactly (the last
// part of values below 2^-110 may underflow). What is not finite stands in the first part.
__device__ __forceinline__ void split3(float v, uint32_t (&h)[3]) {
    if (fabsf(v) < INFINITY) {
        const float a = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), r = v - a;
        const float b = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
        h[0] = __float_as_uint(a) >> 16;
        h[1] = __float_as_uint(b) >> 16;
        h[2] = __float_as_uint(r - b) >> 16;
    } else {
        h[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        h[1] = h[2] = 0;
    }
}

// Copies columns [j0, j0 + 64 tiles) of tokens [t0, t0 + count) to shared memory as the products
// take them: 16-bit and 8-bit activations as they are (asynchronously where their rows are aligned),
// int8 as f16 for a codebook, fp32 in its three parts. Columns from n on are zeros.
template <int K, int kThreads, class X>
__device__ __forceinline__ void stage_x(char* sx, const Args& a, int t0, int count, int j0,
                                        int tiles) {
    const X* x = static_cast<const X*>(a.x) + (int64_t)t0 * a.ldx;
    const bool wide = a.ldx * sizeof(X) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
    if constexpr (!is_split(K) && !(K == kF16Book && std::is_same<X, int8_t>::value)) {
        constexpr int per = 16 / sizeof(X);
        const int chunks = tiles * 64 / per;
        for (int t = 0; t < count; ++t) {
            const X* row = x + (int64_t)t * a.ldx;
            char* dst = sx + t * a.pitch;
            for (int q = threadIdx.x; q < chunks; q += kThreads) {
                const int j = j0 + per * q;
                if (wide && j + per <= a.n) {
                    copy16((uint32_t)__cvta_generic_to_shared(dst + 16 * q), row + j);
                } else {
                    __align__(16) X v[per];
                    memset(v, 0, sizeof v);
#pragma unroll
                    for (int c = 0; c < per; ++c)
                        if (j + c < a.n) v[c] = row[j + c];
                    *reinterpret_cast<uint4*>(dst + 16 * q) = *reinterpret_cast<const uint4*>(v);
                }
            }
        }
    } else {
        const int chunks = tiles * 8;
        for (int t = 0; t < count; ++t) {
            const X* row = x + (int64_t)t * a.ldx;
#pragma unroll 2
            for (int q = threadIdx.x; q < chunks; q += kThreads) {
                const int j = j0 + 8 * q;
                __align__(16) X v[8];
                load8<X>(row + j, a.n - j, wide, v);
                uint32_t h[3][8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if constexpr (is_split(K)) {
                        uint32_t s[3];
                        split3(v[c], s);
                        h[0][c] = s[0], h[1][c] = s[1], h[2][c] = s[2];
                    } else {
                        h[0][c] = __half_as_ushort(__int2half_rn(v[c]));
                    }
                }
#pragma unroll
                for (int s = 0; s < token_rows(K); ++s)
                    *reinterpret_cast<uint4*>(sx + (t * token_rows(K) + s) * a.pitch + q * 16) =
                        make_uint4(h[s][0] | h[s][1] << 16, h[s][2] | h[s][3] << 16,
                                   h[s][4] | h[s][5] << 16, h[s][6] | h[s][7] << 16);
            }
        }
    }
}

// Where the steps change: never within a batch, every 1, 2 or 4 column tiles of it, or anywhere
// (at multiples of 32 columns).
enum Steps { kPerBatch, kPerTile, kAnywhere };

// K: kind, NT: 8-column tiles of the product.
template <int K, int NT, int STEPS>
__global__ void __launch_bounds__(warps_of(K) * 32, blocks_of(K))
matvec4_kernel(const __grid_constant__ Args a) {
    constexpr int kTok = NT * tile_tokens(K), kBatch = batch_of(K);
    constexpr bool HALF = STEPS == kAnywhere;
    constexpr int kWarps = warps_of(K), kThreads = kWarps * 32;
    extern __shared__ __align__(128) char smem[];
    __shared__ int head_tile[kWarps];      // the tile that a warp ends but did not begin, or -1
    cg::cluster_group cluster = cg::this_cluster();
    const int ck = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, g = lane / 4, t = lane % 4;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0);   // uniform
    const Pack4Shape P(a.m, a.n, a.G);
    const int kt0 = min(P.kt, rank * a.slice), kt1 = min(P.kt, kt0 + a.slice);
    const int cl = blockIdx.x / ck;
    const int rt0 = cl * a.tiles_each + min(cl, a.tiles_rest);
    const int rt1 = rt0 + a.tiles_each + (cl < a.tiles_rest);
    const int batches = (kt1 - kt0 + kBatch - 1) / kBatch;
    const int t0 = blockIdx.y * a.chunk, count = min(a.chunk, a.tokens - t0);

    // stages of this warp: kBatch tiles, then the steps of their groups
    const int stage_bytes = kBatch * 512 + a.batch_groups * 64;
    char* ring = smem + warp * kStages * stage_bytes;
    char* sx = smem + kWarps * kStages * stage_bytes;
    char* at = sx + a.chunk * token_rows(K) * a.pitch;
    const uint32_t* table = reinterpret_cast<const uint32_t*>(at);
    if constexpr (is_book(K)) at += planes(K) * 32768;
    const int rows = a.max_tiles * 16;
    float* part = reinterpret_cast<float*>(at);           // [kTok][rows]
    // [warp][kTok][16], without a place for the first warp, which begins all of its tiles
    float* head = part + kTok * (rows - 16);
    float* sxs = head + kWarps * kTok * 16;               // [kTok][steps of x in the slice]
    const int xg0 = a.Gx > 1 ? kt0 * 64 / a.gx : 0;

    if constexpr (is_split(K)) {
        stage_x<K, kThreads, float>(sx, a, t0, count, kt0 * 64, batches * kBatch);
    } else if constexpr (K == kF16) {
        stage_x<K, kThreads, __half>(sx, a, t0, count, kt0 * 64, batches * kBatch);
    } else if constexpr (K == kI8) {
        stage_x<K, kThreads, int8_t>(sx, a, t0, count, kt0 * 64, batches * kBatch);
    } else if constexpr (K == kF16Book) {
        if (a.x_dtype == BAKRON_I8) stage_x<K, kThreads, int8_t>(sx, a, t0, count, kt0 * 64, batches * kBatch);
        else stage_x<K, kThreads, __half>(sx, a, t0, count, kt0 * 64, batches * kBatch);
    } else {
        stage_x<K, kThreads, __nv_bfloat16>(sx, a, t0, count, kt0 * 64, batches * kBatch);
    }
    copy_commit();

    // The block's batches, row tile after row tile, are dealt out evenly over its warps. All of
    // a warp's steps commit a group, those without work an empty one, so that the waits count alike.
    const int units = (rt1 - rt0) * batches;
    const int u0 = units * warp / kWarps;
    const int u1 = units * (warp + 1) / kWarps;
    const int first_tile = batches > 0 ? rt0 + u0 / batches : 0;
    const int first_batch = batches > 0 ? u0 % batches : 0;
    const uint32_t ring32 = (uint32_t)__cvta_generic_to_shared(ring) + lane * 16;

    // where the next batch to be copied stands: tiles, first group, columns of it that are past
    int f_left = u1 - u0, f_batch = first_batch, f_tile = first_tile, f_stage = 0;
    int f_kt = kt0 + f_batch * kBatch;
    int f_grp = f_kt * 64 / a.gs, f_past = f_kt * 64 - f_grp * a.gs;
    const int grp0 = kt0 * 64 / a.gs, past0 = kt0 * 64 - grp0 * a.gs;
    const uint8_t* f_src = a.packed + ((size_t)f_tile * P.kt + f_kt) * 512 + lane * 16;
    const uint8_t* f_steps = a.packed + P.code_bytes() + (size_t)f_tile * a.G * 64 + lane * 16;
    auto fetch = [&]() {
        if (f_left > 0) {
            --f_left;
            const uint32_t dst = ring32 + f_stage * stage_bytes;
            if (f_kt + kBatch <= kt1) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) copy16(dst + u * 512, f_src + u * 512);
            } else {
                // tiles behind the slice are zeros, which meet zeros of x
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    copy16_or_zero(dst + u * 512, f_src + u * 512, f_kt + u < kt1);
            }
            if (lane < 4 * a.batch_groups)
                copy16_or_zero(dst + kBatch * 512, f_steps + (size_t)f_grp * 64,
                               f_grp + lane / 4 < a.G);
            if (STEPS == kAnywhere && lane + 32 < 4 * a.batch_groups)
                copy16_or_zero(dst + kBatch * 512 + 512, f_steps + (size_t)f_grp * 64 + 512,
                               f_grp + 8 + lane / 4 < a.G);
            f_src += kBatch * 512, f_kt += kBatch;
            f_grp += a.batch_gq, f_past += a.batch_gr;
            if (f_past >= a.gs) f_past -= a.gs, ++f_grp;
            if (++f_batch == batches) {
                f_batch = 0, ++f_tile, f_kt = kt0, f_grp = grp0, f_past = past0;
                f_src += ((int64_t)P.kt - (int64_t)batches * kBatch) * 512;
                f_steps += (size_t)a.G * 64;
            }
        }
        copy_commit();
        f_stage = f_stage + 1 == kStages ? 0 : f_stage + 1;
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch();

    if constexpr (is_book(K)) {
        // entry b, codes b % 16 and b / 16, once for every lane: planes 0 and 1 of a lane side by
        // side, plane 2 behind them
        uint4* dst = reinterpret_cast<uint4*>(const_cast<uint32_t*>(table));
        const auto pair = [&](int pl, int b) {
            return a.book.part[pl][b % 16] | a.book.part[pl][b / 16] << 16;
        };
        for (int e = threadIdx.x; e < 4096; e += kThreads) {
            const uint32_t u = pair(0, e / 16), v = pair(1, e / 16);
            dst[e] = make_uint4(u, v, u, v);
        }
        if constexpr (planes(K) == 3)
            for (int e = threadIdx.x; e < 2048; e += kThreads) {
                const uint32_t v = pair(2, e / 8);
                dst[4096 + e] = make_uint4(v, v, v, v);
            }
    }
    const int xgn = a.Gx > 1 ? (kt1 * 64 + a.gx - 1) / a.gx - xg0 : 0;   // steps of x in the slice
    if constexpr (K == kI8 || K == kF16Book) {
        for (int e = threadIdx.x; e < kTok * xgn; e += kThreads) {
            const int tk = e / xgn, q = e - tk * xgn;
            sxs[e] = tk < count && xg0 + q < a.Gx ? a.xs[(size_t)(t0 + tk) * a.Gx + xg0 + q] : 0.f;
        }
    }
    if (units == 0)                 // a slice behind the last column
        for (int e = threadIdx.x; e < kTok * rows; e += kThreads) part[e] = 0.f;
    if (lane == 0) head_tile[warp] = u0 < u1 && first_batch > 0 ? first_tile - rt0 : -1;
    copy_wait<kStages - 1>();       // x is there; the ring's stages may still be on their way
    __syncthreads();
    if constexpr (K == kI8) {
        // bytes in the order of the masked nibbles: columns 0, 2, 1, 3
        const int words = batches * kBatch * 4;
        for (int tk = 0; tk < count; ++tk)
            for (int e = threadIdx.x; e < words; e += kThreads) {
                uint4* p = reinterpret_cast<uint4*>(sx + tk * a.pitch) + e;
                const uint4 v = *p;
                *p = make_uint4(__byte_perm(v.x, 0, 0x3120), __byte_perm(v.y, 0, 0x3120),
                                __byte_perm(v.z, 0, 0x3120), __byte_perm(v.w, 0, 0x3120));
            }
        __syncthreads();
    }

    // staged row of this lane's column in each product tile. A column without a token takes the
    // first one: columns do not meet in a product, and nobody reads its sums.
    const char* brow[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int tok = is_split(K) ? 2 * q + (g & 1) : 8 * q + g;
        const int row = is_split(K) ? tok * 3 + g / 2 : tok;
        const bool on = tok < count && !(is_split(K) && g >= 6);
        brow[q] = sx + (on ? row * a.pitch : 0) + (K == kI8 ? 8 : 16) * t;
    }

    float tot[NT][4];
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) tot[q][c] = 0.f;

    int c_stage = 0, c_tile = first_tile, c_batch = first_batch;
    int past = (kt0 + first_batch * kBatch) * 64 % a.gs;     // columns into the group
    bool whole = first_batch == 0;      // whether this warp began the tile
    for (int unit = u0; unit < u1; ++unit) {
        copy_wait<kStages - 2>();
        __syncwarp();            // the steps were copied by other lanes; all are done with the
        fetch();                 // stage before this one, which is filled now
        const char* stage = ring + c_stage * stage_bytes;
        c_stage = c_stage + 1 == kStages ? 0 : c_stage + 1;
        const float2* steps = reinterpret_cast<const float2*>(stage + kBatch * 512) + g;
        const int xbatch = c_batch * kBatch * 64;
        const char* xb[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) xb[q] = brow[q] + xbatch * (K == kI8 ? 1 : 2);
        float2 s;
        if (STEPS == kPerBatch) s = *steps;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint4 wv = *reinterpret_cast<const uint4*>(stage + u * 512 + lane * 16);
            const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
            float d[NT][4];
            int di[NT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool fresh = h == 0 || HALF;       // the first products of a sum
                float z[4] = {0.f, 0.f, 0.f, 0.f};
                int zi[4] = {0, 0, 0, 0};
                const uint32_t w0 = w[2 * h], w1 = w[2 * h + 1];
                if constexpr (K == kI8) {
                    const uint32_t A[4] = {(w0 << 4) & 0xF0F0F0F0u, (w1 << 4) & 0xF0F0F0F0u,
                                           w0 & 0xF0F0F0F0u, w1 & 0xF0F0F0F0u};
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        const uint2 B = *reinterpret_cast<const uint2*>(xb[q] + 64 * u + 32 * h);
                        mma_s8(di[q], A, B.x, B.y, fresh ? zi : di[q]);
                    }
                } else {
                    uint4 B[NT];      // B0, B1 of the first product, then of the second
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        const uint4 v =
                            *reinterpret_cast<const uint4*>(xb[q] + 128 * u + 64 * h);
                        if constexpr (is_book(K))     // pairs as the table gives them
                            B[q] = make_uint4(__byte_perm(v.x, v.z, 0x5410),
                                              __byte_perm(v.y, v.w, 0x5410),
                                              __byte_perm(v.x, v.z, 0x7632),
                                              __byte_perm(v.y, v.w, 0x7632));
                        else
                            B[q] = v;
                    }
                    uint2 e0[4], e1[4];      // codebook: planes 0 and 1
                    if constexpr (is_book(K)) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            // byte * 256 + lane * 8
                            const char* tb = reinterpret_cast<const char*>(table);
                            e0[q] = *reinterpret_cast<const uint2*>(
                                tb + __byte_perm(w0, 8 * lane, 0x5504 | q << 4));
                            e1[q] = *reinterpret_cast<const uint2*>(
                                tb + __byte_perm(w1, 8 * lane, 0x5504 | q << 4));
                        }
                    }
#pragma unroll
                    for (int pl = 0; pl < (is_book(K) ? planes(K) : 1); ++pl) {
                        uint32_t p0[4], p1[4];
                        if constexpr (is_book(K)) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if (pl < 2) {
                                    p0[q] = pl ? e0[q].y : e0[q].x;
                                    p1[q] = pl ? e1[q].y : e1[q].x;
                                } else {      // byte * 128 + lane * 4 of a table of its own
                                    const char* tb =
                                        reinterpret_cast<const char*>(table) + 65536 + 4 * lane;
                                    p0[q] = *reinterpret_cast<const uint32_t*>(
                                        tb + (w0 >> (8 * q) & 0xFF) * 128);
                                    p1[q] = *reinterpret_cast<const uint32_t*>(
                                        tb + (w1 >> (8 * q) & 0xFF) * 128);
                                }
                            }
                        } else if constexpr (is_half(K)) {
                            codes_f16(w0, p0);
                            codes_f16(w1, p1);
                        } else {
                            codes_bf16(w0, p0);
                            codes_bf16(w1, p1);
                        }
                        const uint32_t A0[4] = {p0[0], p1[0], p0[1], p1[1]};
                        const uint32_t A1[4] = {p0[2], p1[2], p0[3], p1[3]};
#pragma unroll
                        for (int q = 0; q < NT; ++q) {
                            if constexpr (is_half(K)) {
                                mma_f16(d[q], A0, B[q].x, B[q].y, fresh && pl == 0 ? z : d[q]);
                                mma_f16(d[q], A1, B[q].z, B[q].w, d[q]);
                            } else {
                                mma_bf16(d[q], A0, B[q].x, B[q].y, fresh && pl == 0 ? z : d[q]);
                                mma_bf16(d[q], A1, B[q].z, B[q].w, d[q]);
                            }
                        }
                    }
                }
                if (h == 1 || HALF) {
                    if constexpr (STEPS == kPerTile) s = steps[(u >> a.step_shift) * 8];
                    if constexpr (STEPS == kAnywhere) {
                        s = *steps;
                        past += 32;
                        if (past >= a.gs) past -= a.gs, steps += 8;
                    }
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        float s4[4] = {s.x, s.x, s.y, s.y};
                        if constexpr (K == kI8 || K == kF16Book) {
                            if (a.Gx > 1) {
                                const int xg = (kt0 * 64 + xbatch + 64 * u + (HALF ? 32 * h : 0)) / a.gx - xg0;
                                const float* xr = sxs + (8 * q + 2 * t) * xgn + min(xg, xgn - 1);
                                const float x0 = xr[0], x1 = xr[xgn];
                                s4[0] *= x0, s4[1] *= x1, s4[2] *= x0, s4[3] *= x1;
                            }
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tot[q][c] = fmaf(s4[c], K == kI8 ? (float)di[q][c] : d[q][c],
                                             tot[q][c]);
                    }
                }
            }
        }
        if (++c_batch == batches || unit + 1 == u1) {
            // the tile's sums: whole tiles and a tile's first part to its rows, the end of a tile
            // that another warp began to this warp's place
            float* out = whole ? part + (c_tile - rt0) * 16 : head + warp * kTok * 16;
            const int ld = whole ? rows : 16;
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                if constexpr (is_split(K)) {  // columns 0..5: part (lane t) of tokens 2 q, 2 q + 1
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float v = t == 3 ? 0.f : tot[q][c];
                        v += __shfl_xor_sync(0xffffffffu, v, 2);
                        v += __shfl_xor_sync(0xffffffffu, v, 1);
                        if (t == 0) out[(2 * q + (c & 1)) * ld + g + 8 * (c >> 1)] = v;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        out[(8 * q + 2 * t + (c & 1)) * ld + g + 8 * (c >> 1)] = tot[q][c];
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) tot[q][c] = 0.f;
            }
            c_batch = 0, ++c_tile, past = past0;
            whole = true;
        }
    }
    __syncthreads();
    // ends of tiles that another warp began, warp after warp (one thread an element)
    for (int w = 1; w < kWarps; ++w) {
        const int tile = head_tile[w];
        if (tile < 0) continue;
        for (int e = threadIdx.x; e < kTok * 16; e += kThreads)
            part[(e / 16) * rows + tile * 16 + e % 16] += head[w * kTok * 16 + e];
    }

    // the blocks of the cluster add up a share of the rows each, four rows a thread
    if (ck > 1) cluster.sync();
    else __syncthreads();
    const int quads = (rt1 - rt0) * 4, share = (quads + ck - 1) / ck;
    for (int e = threadIdx.x; e < share * count; e += kThreads) {
        const int tk = e / share, quad = rank * share + e - tk * share;
        const int64_t i = (int64_t)rt0 * 16 + 4 * quad;
        if (quad >= quads || i >= a.m) continue;
        float4 got[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < ck)
                got[c] = *reinterpret_cast<const float4*>(
                    (ck > 1 ? cluster.map_shared_rank(part, c) : part) + tk * rows + 4 * quad);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < ck) v[0] += got[c].x, v[1] += got[c].y, v[2] += got[c].z, v[3] += got[c].w;
        float f = 1.f;
        if (K == kI8 || K == kF16Book)
            if (a.Gx == 1 && a.xs) f = a.xs[t0 + tk];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = v[r] * a.out1 * a.out2 * f;
        const int64_t o = (int64_t)(t0 + tk) * a.ldy + i;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (i + r >= a.m) break;
            if (a.y_dtype == BAKRON_F32) static_cast<float*>(a.y)[o + r] = v[r];
            else if (a.y_dtype == BAKRON_F16) from_f32(v[r], static_cast<__half*>(a.y)[o + r]);
            else from_f32(v[r], static_cast<__nv_bfloat16*>(a.y)[o + r]);
        }
    }
    if (ck > 1) cluster.sync();
}

// ------------------------------------------------------------------------------------- host
template <int K, int NT, int STEPS>
int launch(const Args& a, int ck, size_t smem, cudaStream_t st) {
    auto kern = matvec4_kernel<K, NT, STEPS>;
    if (smem > 48 * 1024 && !allow_smem<kSmemLimit - kStaticSmem>(kern)) return BAKRON_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.clusters * ck), (unsigned)((a.tokens + a.chunk - 1) / a.chunk));
    cfg.blockDim = dim3(warps_of(K) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ck;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    count_launches(1);
    return cuda_err(e);
}

// One way to cut the work: ck slices of the columns, the row tiles dealt out over clusters of ck
// blocks, as many as fit the GPU at once (times the chunks of tokens). 28672 x 8192 of bf16 in 1, 2,
// 4 and 8 slices: one token 28.9 / 29.3 / 31.7 / 33.8 us, 8 tokens 31.3 / 31.8 / 34.6 / 43.4, and 16
// tokens, whose activations do not fit in one slice, 53.3 / 54.4 / 45.1 / 56.3.
struct Cut { int ck = 0, slice, pitch, chunk, clusters, max_tiles; size_t smem; double cost; };

template <int K>
Cut cut(const Args& a, int ck, int nt, int sms, bool few_tiles) {
    const Pack4Shape P(a.m, a.n, a.G);
    constexpr int kBatch = batch_of(K);
    Cut c;
    c.slice = (P.kt + ck - 1) / ck;
    c.slice = (c.slice + kBatch - 1) / kBatch * kBatch;
    // rows of staged activations, apart by what keeps their reads free of bank conflicts
    const int row = c.slice * 64 * (K == kI8 ? 1 : 2);
    c.pitch = K == kI8 ? row + 32 : row % 128 ? row : row + 64;
    const int tok = nt * tile_tokens(K);
    const size_t limit = kSmemLimit;
    // What a block takes, the static array at most: its bytes stand for the place of the first warp.
    const size_t first = (size_t)tok * 16 * 4;
    static_assert(tile_tokens(K) * 16 * 4 >= kStaticSmem, "a place is no less than the static array");
    const auto bytes = [&] {
        size_t b = (size_t)warps_of(K) * kStages * (kBatch * 512 + a.batch_groups * 64) +
                   (size_t)c.chunk * token_rows(K) * c.pitch +
                   (size_t)tok * 16 * 4 * (c.max_tiles + warps_of(K));
        if (is_book(K)) b += planes(K) * 32768;
        if (a.Gx > 1) b += (size_t)tok * 4 * ((size_t)c.slice * 64 / a.gx + 2);
        return b;
    };
    // tiles an SM goes through, and its share of staged activations (from L2)
    const auto taken = [&] {
        const long long chunks = (a.tokens + c.chunk - 1) / c.chunk;
        const long long per_sm = ((long long)c.clusters * ck * chunks + sms - 1) / sms;
        c.ck = ck;
        c.cost = (double)per_sm * (c.max_tiles * (double)c.slice +
                                   0.08 * c.slice * c.chunk * token_rows(K) + 4.0);
    };
    c.chunk = std::min(a.tokens, tok);
    // SMs that clusters of ck blocks can fill (they do not cross a GPC): on a B200 132 of 148 in fours,
    // 120 in eights, as its occupancy query says; one more would wait for a second wave
    const int fit = ck <= 2 ? sms : ck == 4 ? sms * 33 / 37 : sms * 30 / 37;
    // blocks an SM and row tiles a cluster depend on each other through shared memory: from the
    // most blocks down to what fits
    for (int occ = few_tiles ? 0 : blocks_of(K); occ >= 1; --occ) {
        for (;; c.chunk /= 2) {
            const int chunks = (a.tokens + c.chunk - 1) / c.chunk;
            c.clusters = std::max(1, std::min(P.mt, occ * fit / ck / std::min(chunks, 1 << 20)));
            c.max_tiles = (P.mt + c.clusters - 1) / c.clusters;
            // sums of at most 64 row tiles stay in shared memory: more clusters than fit at once
            if (c.max_tiles > 64) c.max_tiles = 64, c.clusters = (P.mt + 63) / 64;
            if (occ * (bytes() + 1024) <= 228 * 1024 && bytes() <= limit) {
                c.smem = bytes() - first;
                taken();
                return c;
            }
            if (occ > 1 || c.chunk == 1) break;
        }
    }
    for (c.chunk = std::min(a.tokens, tok); few_tiles && c.chunk >= 1; c.chunk /= 2) {
        c.max_tiles = 0;
        const size_t fixed = bytes();
        if (fixed >= limit) continue;
        c.max_tiles = (int)std::min<size_t>((limit - fixed) / ((size_t)tok * 64), 64);
        if (c.max_tiles < 1) continue;
        c.clusters = (P.mt + c.max_tiles - 1) / c.max_tiles;
        c.max_tiles = (P.mt + c.clusters - 1) / c.clusters;
        c.smem = bytes() - first;
        taken();
        return c;
    }
    return c;
}

// The cheapest cut for a call on `sms` SMs, also entered in its arguments, and its product tiles nt.
template <int K>
Cut choose(Args& a, int sms, int& best_nt) {
    const Pack4Shape P(a.m, a.n, a.G);
    constexpr int kBatch = batch_of(K), cols = kBatch * 64;
    a.batch_groups = a.G == 1 || a.gs % cols == 0 ? 1
                     : cols % a.gs == 0           ? cols / a.gs
                                                  : (cols - 1) / a.gs + 2;
    a.batch_gq = cols / a.gs, a.batch_gr = cols % a.gs;
    Cut best;
    best_nt = 1;
    // Where the sums of a cluster's row tiles never fit beside one token (long rows of fp32 with a
    // codebook): fewer tiles a cluster, more clusters than fit the GPU at once.
    for (int few = 0; few < 2 && !best.ck; ++few)
        for (int nt = 1; nt <= 4; nt *= 2) {
            if (nt > 1 && a.tokens <= nt / 2 * tile_tokens(K)) break;
            for (int ck = 1; ck <= 8 && (ck == 1 || P.kt >= kBatch * ck); ck *= 2) {
                const Cut c = cut<K>(a, ck, nt, sms, few != 0);
                if (c.ck && (!best.ck || c.cost < best.cost)) best = c, best_nt = nt;
            }
        }
    if (!best.ck) return best;
    a.slice = best.slice, a.pitch = best.pitch, a.chunk = best.chunk;
    a.clusters = best.clusters, a.max_tiles = best.max_tiles;
    a.tiles_each = P.mt / a.clusters, a.tiles_rest = P.mt % a.clusters;
    return best;
}

template <int K>
int plan(Args& a, cudaStream_t st) {
    const int sms = tc::sm_count();
    if (sms <= 0) return BAKRON_ERR_CUDA;
    constexpr int cols = batch_of(K) * 64;
    int best_nt;
    const Cut best = choose<K>(a, sms, best_nt);
    if (!best.ck) return BAKRON_ERR_INVALID_ARG;
    const int ck = best.ck;
    const size_t smem = best.smem;
    // batches begin at multiples of `cols` columns
    a.step_shift = a.gs == 64 ? 0 : a.gs == 128 ? 1 : 2;
    int steps = a.G == 1 || a.gs % cols == 0                    ? kPerBatch
                : a.gs >= 64 && cols % a.gs == 0 ? kPerTile
                                                 : kAnywhere;
    if (a.Gx > 1 && a.gx % 64) steps = kAnywhere;
    switch (best_nt * 4 + steps) {
        case 4: return launch<K, 1, kPerBatch>(a, ck, smem, st);
        case 5: return launch<K, 1, kPerTile>(a, ck, smem, st);
        case 6: return launch<K, 1, kAnywhere>(a, ck, smem, st);
        case 8: return launch<K, 2, kPerBatch>(a, ck, smem, st);
        case 9: return launch<K, 2, kPerTile>(a, ck, smem, st);
        case 10: return launch<K, 2, kAnywhere>(a, ck, smem, st);
        case 16: return launch<K, 4, kPerBatch>(a, ck, smem, st);
        case 17: return launch<K, 4, kPerTile>(a, ck, smem, st);
        default: return launch<K, 4, kAnywhere>(a, ck, smem, st);
    }
}

uint32_t bits_of(float f) {
    uint32_t u;
    std::memcpy(&u, &f, 4);
    return u;
}
float cut16(float f) {       // its upper 16 bits: a bf16, rounded toward zero
    const uint32_t u = bits_of(f) & 0xFFFF0000u;
    float r;
    std::memcpy(&r, &u, 4);
    return r;
}

// The 16-bit parts of the entries. f16: the entries are first brought to [2^13, 2^14) by a power
// of two (out1, out2 undo it), then a part is the rounding of what is left: 22 bits and more of
// the largest. bf16: upper bits, then the rounding of what is left: 16 bits, or 24 in three parts.
template <int K>
void split_book(const float* c, int entries, Args& a) {
    std::memset(&a.book, 0, sizeof a.book);
    if (K == kF16Book) {
        float top = 0.f;
        for (int k = 0; k < entries; ++k) top = std::fmax(top, std::fabs(c[k]));
        int e = 0;
        if (top > 0.f) {
            std::frexp(top, &e);
            e = 14 - e;
        }
        a.out1 = std::ldexp(1.f, -(e / 2));
        a.out2 = std::ldexp(1.f, -(e - e / 2));
        for (int k = 0; k < entries; ++k) {
            const double v = std::ldexp((double)c[k], e);
            const __half hi = __float2half_rn((float)v);
            const __half lo = __float2half_rn((float)(v - (double)__half2float(hi)));
            a.book.part[0][k] = __half_as_ushort(hi);
            a.book.part[1][k] = __half_as_ushort(lo);
        }
    } else {
        for (int k = 0; k < entries; ++k) {
            const float hi = cut16(c[k]), r = c[k] - hi, mid = cut16(r);
            a.book.part[0][k] = bits_of(hi) >> 16;
            if (K == kBf16Book) {
                a.book.part[1][k] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
            } else {
                a.book.part[1][k] = bits_of(mid) >> 16;
                a.book.part[2][k] = bits_of(r - mid) >> 16;
            }
        }
    }
}

Args arguments(const void* packed, int m, int n, int group_size, const void* x, int x_dtype,
               int64_t ldx, const float* x_scales, int x_group_size, int tokens, void* y,
               int y_dtype, int64_t ldy) {
    Args a{};
    a.packed = static_cast<const uint8_t*>(packed);
    a.m = m, a.n = n;
    a.G = group_count(group_size, n);
    a.gs = a.G > 1 ? group_size : 1 << 30;     // one step: no column is past it
    a.x = x, a.x_dtype = x_dtype, a.ldx = ldx, a.xs = x_scales;
    a.Gx = x_dtype == BAKRON_I8 ? group_count(x_group_size, n) : 1;
    a.gx = a.Gx > 1 ? x_group_size : 64 * ((n + 63) / 64);
    a.tokens = tokens, a.y = y, a.y_dtype = y_dtype, a.ldy = ldy;
    a.out1 = a.out2 = 1.f;
    return a;
}

// f(the kind that a call takes)
template <class F>
int with_kind(const Args& a, bool book, F f) {
    if (book) {
        if (a.x_dtype == BAKRON_F32) return f(std::integral_constant<int, kF32Book>());
        if (a.x_dtype == BAKRON_BF16 && a.y_dtype == BAKRON_F32)
            return f(std::integral_constant<int, kBf16Wide>());
        if (a.x_dtype == BAKRON_BF16) return f(std::integral_constant<int, kBf16Book>());
        return f(std::integral_constant<int, kF16Book>());
    }
    switch (a.x_dtype) {
        case BAKRON_F32: return f(std::integral_constant<int, kF32>());
        case BAKRON_F16: return f(std::integral_constant<int, kF16>());
        case BAKRON_BF16: return f(std::integral_constant<int, kBf16>());
        default: return f(std::integral_constant<int, kI8>());
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
    Args a = arguments(packed, m, n, group_size, x, x_dtype, ldx, x_scales, x_group_size, tokens, y,
                       y_dtype, ldy);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_kind(a, codebook != nullptr, [&](auto kind) {
        constexpr int K = decltype(kind)::value;
        if constexpr (is_book(K)) split_book<K>(codebook, 1 << bits, a);
        if constexpr (K == kI8) a.out1 = 1.f / 16.f;    // the codes stand in the upper halves of bytes
        return plan<K>(a, st);
    });
}

extern "C" int bakron_internal_matvec4_plan(int m, int n, int group_size, int x_dtype,
                                            int x_group_size, int y_dtype, int book, int tokens,
                                            int sms, int64_t* out) {
    Args a = arguments(nullptr, m, n, group_size, nullptr, x_dtype, n, nullptr, x_group_size, tokens,
                       nullptr, y_dtype, m);
    return with_kind(a, book != 0, [&](auto kind) {
        constexpr int K = decltype(kind)::value;
        int nt;
        const Cut c = choose<K>(a, sms, nt);
        if (!c.ck) return (int)BAKRON_ERR_INVALID_ARG;
        const int64_t r[8] = {(int64_t)c.smem, c.ck, c.slice, c.chunk, c.clusters, c.max_tiles, nt,
                              warps_of(K)};
        std::copy(r, r + 8, out);
        return (int)BAKRON_OK;
    });
}
