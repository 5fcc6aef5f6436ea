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
// same. (tcgen05.mma would want the unpacked weights in shared memory first: two more passes over
// them there, for products that are not what bounds this kernel.)
//
//   * A warp owns a row tile (16 rows) and a slice of the columns. Its loads are the layout's 512-byte
//     tiles, 16 bytes a lane, four tiles ahead of their use, in registers: each lane's 16 bytes are its
//     own fragments of four m16n8k16 (two m16n8k32) products.
//   * The codes become f16 or bf16 by setting the exponent bits around them (1024 + code and
//     128 + code are exact) and one subtraction a pair; int8 by masking: a code in the upper half of
//     its byte is 16 times the code. fp32 activations are split in three bf16 parts of 8 bits, which
//     stand in three columns of the tensor tile, so their products are exact too.
//   * Codebook entries come in pairs from a table in shared memory that is indexed by a byte of two
//     codes and has one copy a lane (bank), so the reads never conflict; an entry is held as two
//     16-bit parts (fp32 activations: three), each multiplied on its own.
//   * Products are summed over 64 (32) columns in the tensor core's fp32 (int8: exactly, in int32),
//     then scaled and added in fp32 round-to-nearest.
//   * A cluster's blocks take slices of the columns for the same rows and add their sums through
//     distributed shared memory in rank order: no atomics, the same bits every time.
#include <cooperative_groups.h>

#include <cmath>
#include <cstring>

#include "pack4.cuh"

namespace bakron {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kAhead = 4;          // column tiles a warp loads ahead

enum Kind { kF16, kBf16, kF32, kI8, kF16Book, kBf16Book, kF32Book };
constexpr bool is_book(int k) { return k >= kF16Book; }
constexpr int planes(int k) { return k == kF32Book ? 3 : 2; }
constexpr bool is_split(int k) { return k == kF32 || k == kF32Book; }   // fp32 activations
constexpr bool is_half(int k) { return k == kF16 || k == kF16Book; }
// tokens in one 8-column tile of the product, staged rows a token
constexpr int tile_tokens(int k) { return is_split(k) ? 2 : 8; }
constexpr int token_rows(int k) { return is_split(k) ? 3 : 1; }

struct Book { uint32_t part[3][16]; };   // 16-bit parts of the entries (host-made)

struct Args {
    const uint8_t* packed; int m, n, G, gs;
    const void* x; int x_dtype; int64_t ldx; const float* xs; int Gx, gx;
    int tokens; void* y; int y_dtype; int64_t ldy;
    int slice;               // column tiles of a block
    int tpw;                 // row tiles of a warp
    int pitch;               // bytes between staged rows of x
    float out1, out2;        // powers of two for the result
    Book book;
};

__device__ __forceinline__ uint4 load_tile(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (w & mask) ^ bits
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}

// The 8 codes of a word as four f16 pairs: columns (0, 1), (4, 5), (2, 3), (6, 7). The xor turns
// the two's complement nibble into code + 8 under the exponent of 1024 (or 64 for the upper
// nibble, with the product by 1/16).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&p)[4]) {
    const __half2 c0 = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));
    const __half2 c1 = __floats2half2_rn(-72.f, -72.f), r16 = __floats2half2_rn(0.0625f, 0.0625f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t u = q < 2 ? w : w >> 8;
        const uint32_t v = (q & 1) ? and_xor(u, 0x00F000F0u, 0x64806480u)
                                   : and_xor(u, 0x000F000Fu, 0x64086408u);
        __half2 h = *reinterpret_cast<const __half2*>(&v);
        h = (q & 1) ? __hfma2(h, r16, c1) : __hsub2(h, c0);
        p[q] = *reinterpret_cast<uint32_t*>(&h);
    }
}
// The same in bf16, which holds 128 + (code + 8) exactly.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t (&p)[4]) {
    const __nv_bfloat162 c = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t v = and_xor(w >> (4 * q), 0x000F000Fu, 0x43084308u);
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

// Copies columns [j0, j0 + 8 chunks) of tokens [t0, t0 + count) to shared memory, in the type and the
// order within 8 columns that the products take.
template <int K, class X>
__device__ __forceinline__ void stage_x(char* sx, const Args& a, int t0, int count, int j0,
                                        int chunks) {
    const X* x = static_cast<const X*>(a.x);
    const bool wide = a.ldx * sizeof(X) % 16 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
    for (int e = threadIdx.x; e < count * chunks; e += kThreads) {
        const int t = e / chunks, q = e - t * chunks, j = j0 + 8 * q;
        __align__(16) X v[8];
        load8<X>(x + (int64_t)(t0 + t) * a.ldx + j, a.n - j, wide, v);
        if constexpr (K == kI8) {
            // bytes in the order of the masked nibbles; a tile's two halves of a lane side by side
            const uint2 u = *reinterpret_cast<const uint2*>(v);
            char* dst = sx + t * a.pitch + (q / 8) * 64 + (q % 4) * 16 + (q / 4 % 2) * 8;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(__byte_perm(u.x, 0, 0x3120), __byte_perm(u.y, 0, 0x3120));
        } else {
            uint32_t h[3][8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if constexpr (is_split(K)) {
                    uint32_t s[3];
                    split3(v[c], s);
                    h[0][c] = s[0], h[1][c] = s[1], h[2][c] = s[2];
                } else if constexpr (std::is_same<X, int8_t>::value) {
                    h[0][c] = __half_as_ushort(__int2half_rn(v[c]));
                } else {
                    h[0][c] = *reinterpret_cast<const uint16_t*>(&v[c]);
                }
            }
#pragma unroll
            for (int s = 0; s < token_rows(K); ++s) {
                uint4 o;
                if constexpr (is_book(K))     // pairs as the table gives them
                    o = make_uint4(h[s][0] | h[s][4] << 16, h[s][2] | h[s][6] << 16,
                                   h[s][1] | h[s][5] << 16, h[s][3] | h[s][7] << 16);
                else                          // first and second product's pairs
                    o = make_uint4(h[s][0] | h[s][1] << 16, h[s][4] | h[s][5] << 16,
                                   h[s][2] | h[s][3] << 16, h[s][6] | h[s][7] << 16);
                *reinterpret_cast<uint4*>(sx + (t * token_rows(K) + s) * a.pitch + q * 16) = o;
            }
        }
    }
}

// K: kind, NT: 8-column tiles of the product, HALF: steps change every 32 columns.
template <int K, int NT, bool HALF>
__global__ void __launch_bounds__(kThreads, 2) matvec4_kernel(const __grid_constant__ Args a) {
    constexpr int kTok = NT * tile_tokens(K);
    constexpr int kFlush = HALF ? 2 : 1;
    extern __shared__ __align__(128) char smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int ck = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
    const Pack4Shape P(a.m, a.n, a.G);
    const int kt0 = rank * a.slice, kt1 = min(P.kt, kt0 + a.slice);
    const int block = blockIdx.x / ck;
    const int rt_first = block * kWarps * a.tpw + warp;
    const int t0 = blockIdx.y * kTok, count = min(kTok, a.tokens - t0);

    char* sx = smem;
    char* at = smem + kTok * token_rows(K) * a.pitch;
    const uint32_t* table = reinterpret_cast<const uint32_t*>(at);
    if constexpr (is_book(K)) at += planes(K) * 32768;
    float* part = reinterpret_cast<float*>(at);           // [kTok][rows of the block]
    const int rows = kWarps * a.tpw * 16;
    float* sxs = part + kTok * rows;                      // [kTok][steps of x in the slice]
    const int xg0 = a.Gx > 1 ? kt0 * 64 / a.gx : 0;

    const uint4* tiles = reinterpret_cast<const uint4*>(a.packed) + lane;
    const float2* steps = reinterpret_cast<const float2*>(a.packed + P.code_bytes()) + g;

    // the first tiles are on their way before x is staged
    uint4 cur[kAhead], nxt[kAhead];
    float2 scur[kAhead][kFlush], snxt[kAhead][kFlush];
    auto fetch = [&](int rt, int kt, uint4 (&w)[kAhead], float2 (&s)[kAhead][kFlush]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (rt < P.mt && kt + u < kt1) {
                w[u] = load_tile(tiles + ((size_t)rt * P.kt + kt + u) * 32);
#pragma unroll
                for (int f = 0; f < kFlush; ++f) {
                    // a tile's second half may lie behind the last step
                    const int grp = min((int)((unsigned)((kt + u) * 64 + 32 * f) / (unsigned)a.gs),
                                        a.G - 1);
                    s[u][f] = __ldg(steps + ((size_t)rt * a.G + grp) * 8);
                }
            } else {
                w[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int f = 0; f < kFlush; ++f) s[u][f] = make_float2(0.f, 0.f);
            }
        }
    };
    fetch(rt_first, kt0, cur, scur);

    const int chunks = max(0, kt1 - kt0) * 8;
    if constexpr (K == kF32 || K == kF32Book) {
        stage_x<K, float>(sx, a, t0, count, kt0 * 64, chunks);
    } else if constexpr (K == kF16) {
        stage_x<K, __half>(sx, a, t0, count, kt0 * 64, chunks);
    } else if constexpr (K == kI8) {
        stage_x<K, int8_t>(sx, a, t0, count, kt0 * 64, chunks);
    } else if constexpr (K == kF16Book) {
        if (a.x_dtype == BAKRON_I8) stage_x<K, int8_t>(sx, a, t0, count, kt0 * 64, chunks);
        else stage_x<K, __half>(sx, a, t0, count, kt0 * 64, chunks);
    } else {
        stage_x<K, __nv_bfloat16>(sx, a, t0, count, kt0 * 64, chunks);
    }
    if constexpr (is_book(K)) {
        // entry e of a plane: codes e % 16 and e / 16, once for every lane
        uint4* dst = reinterpret_cast<uint4*>(const_cast<uint32_t*>(table));
        for (int e = threadIdx.x; e < planes(K) * 256 * 8; e += kThreads) {
            const int pl = e / 2048, b = e / 8 % 256;
            const uint32_t v = a.book.part[pl][b % 16] | a.book.part[pl][b / 16] << 16;
            dst[e] = make_uint4(v, v, v, v);
        }
    }
    if constexpr (K == kI8 || K == kF16Book) {
        if (a.Gx > 1) {
            const int xgn = (kt1 * 64 + a.gx - 1) / a.gx - xg0;     // groups of the slice
            for (int e = threadIdx.x; e < kTok * xgn; e += kThreads) {
                const int tk = e / xgn, q = e - tk * xgn;
                sxs[e] = tk < count && xg0 + q < a.Gx
                             ? a.xs[(size_t)(t0 + tk) * a.Gx + xg0 + q] : 0.f;
            }
        }
    }
    __syncthreads();
    const int xgn = a.Gx > 1 ? (kt1 * 64 + a.gx - 1) / a.gx - xg0 : 0;

    // staged row of this lane's column in each product tile; columns without one multiply zeros
    const char* brow[NT];
    bool bon[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int tok = is_split(K) ? 2 * q + (g & 1) : 8 * q + g;
        const int row = is_split(K) ? tok * 3 + g / 2 : tok;
        bon[q] = tok < count && !(is_split(K) && g >= 6);
        brow[q] = sx + row * a.pitch + (K == kI8 ? 16 * t : 16 * t);
    }

    float tot[NT][4];
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) tot[q][c] = 0.f;

    const int batches = (max(0, kt1 - kt0) + kAhead - 1) / kAhead;
    for (int i = 0; i < a.tpw; ++i) {
        const int rt = rt_first + i * kWarps;
        for (int b = 0; b < batches; ++b) {
            const int kt = kt0 + b * kAhead;
            if (b + 1 < batches) fetch(rt, kt + kAhead, nxt, snxt);
            else if (i + 1 < a.tpw) fetch(rt + kWarps, kt0, nxt, snxt);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (kt + u >= kt1) break;
                const uint32_t w[4] = {cur[u].x, cur[u].y, cur[u].z, cur[u].w};
                float d[NT][4];
                int di[NT][4];
                uint4 bi[NT];      // int8: both halves at once
                if constexpr (K == kI8) {
#pragma unroll
                    for (int q = 0; q < NT; ++q)
                        bi[q] = bon[q] ? *reinterpret_cast<const uint4*>(brow[q] + (kt + u - kt0) * 64)
                                       : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 0 || HALF) {
#pragma unroll
                        for (int q = 0; q < NT; ++q)
#pragma unroll
                            for (int c = 0; c < 4; ++c) d[q][c] = 0.f, di[q][c] = 0;
                    }
                    if constexpr (K == kI8) {
                        const uint32_t A[4] = {(w[2 * h] << 4) & 0xF0F0F0F0u,
                                               (w[2 * h + 1] << 4) & 0xF0F0F0F0u,
                                               w[2 * h] & 0xF0F0F0F0u, w[2 * h + 1] & 0xF0F0F0F0u};
#pragma unroll
                        for (int q = 0; q < NT; ++q)
                            mma_s8(di[q], A, h ? bi[q].z : bi[q].x, h ? bi[q].w : bi[q].y);
                    } else {
                        uint4 B[NT];
#pragma unroll
                        for (int q = 0; q < NT; ++q)
                            B[q] = bon[q] ? *reinterpret_cast<const uint4*>(
                                                brow[q] + (kt + u - kt0) * 128 + 64 * h)
                                          : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int pl = 0; pl < (is_book(K) ? planes(K) : 1); ++pl) {
                            uint32_t p0[4], p1[4];
                            if constexpr (is_book(K)) {
                                const char* tb = reinterpret_cast<const char*>(table) + pl * 32768;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const uint32_t u0 = w[2 * h], u1 = w[2 * h + 1];
                                    const uint32_t s0 = q == 0 ? u0 << 7 : u0 >> (8 * q - 7);
                                    const uint32_t s1 = q == 0 ? u1 << 7 : u1 >> (8 * q - 7);
                                    p0[q] = *reinterpret_cast<const uint32_t*>(
                                        tb + ((s0 & 0x7F80u) | (4 * lane)));
                                    p1[q] = *reinterpret_cast<const uint32_t*>(
                                        tb + ((s1 & 0x7F80u) | (4 * lane)));
                                }
                            } else if constexpr (is_half(K)) {
                                codes_f16(w[2 * h], p0);
                                codes_f16(w[2 * h + 1], p1);
                            } else {
                                codes_bf16(w[2 * h], p0);
                                codes_bf16(w[2 * h + 1], p1);
                            }
                            const uint32_t A0[4] = {p0[0], p1[0], p0[1], p1[1]};
                            const uint32_t A1[4] = {p0[2], p1[2], p0[3], p1[3]};
#pragma unroll
                            for (int q = 0; q < NT; ++q) {
                                if constexpr (is_half(K)) {
                                    mma_f16(d[q], A0, B[q].x, B[q].y);
                                    mma_f16(d[q], A1, B[q].z, B[q].w);
                                } else {
                                    mma_bf16(d[q], A0, B[q].x, B[q].y);
                                    mma_bf16(d[q], A1, B[q].z, B[q].w);
                                }
                            }
                        }
                    }
                    if (h == 1 || HALF) {
                        const float2 s = scur[u][HALF ? h : 0];
#pragma unroll
                        for (int q = 0; q < NT; ++q) {
                            float s4[4] = {s.x, s.x, s.y, s.y};
                            if constexpr (K == kI8 || K == kF16Book) {
                                if (a.Gx > 1) {
                                    const int xg = ((kt + u) * 64 + (HALF ? 32 * h : 0)) / a.gx - xg0;
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
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                cur[u] = nxt[u];
#pragma unroll
                for (int f = 0; f < kFlush; ++f) scur[u][f] = snxt[u][f];
            }
        }
        // this row tile's sums to shared memory
        const int r0 = (warp + i * kWarps) * 16 + g;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            if constexpr (is_split(K)) {      // columns 0..5: part (lane t) of tokens 2 q, 2 q + 1
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float v = tot[q][c];
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    if (t == 0) part[(2 * q + (c & 1)) * rows + r0 + 8 * (c >> 1)] = v;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    part[(8 * q + 2 * t + (c & 1)) * rows + r0 + 8 * (c >> 1)] = tot[q][c];
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) tot[q][c] = 0.f;
        }
    }

    // the blocks of the cluster add up a share of the rows each
    if (ck > 1) cluster.sync();
    else __syncthreads();
    const int share = rows / ck;
    for (int e = threadIdx.x; e < share * count; e += kThreads) {
        const int tk = e / share, r = rank * share + e - tk * share;
        const int64_t i = (int64_t)block * rows + r;
        if (i >= a.m) continue;
        float v = 0.f;
        for (int c = 0; c < ck; ++c)
            v += (ck > 1 ? cluster.map_shared_rank(part, c) : part)[tk * rows + r];
        v = v * a.out1 * a.out2;
        if (K == kI8 || K == kF16Book)
            if (a.Gx == 1 && a.xs) v *= a.xs[t0 + tk];
        const int64_t o = (int64_t)(t0 + tk) * a.ldy + i;
        if (a.y_dtype == BAKRON_F32) static_cast<float*>(a.y)[o] = v;
        else if (a.y_dtype == BAKRON_F16) from_f32(v, static_cast<__half*>(a.y)[o]);
        else from_f32(v, static_cast<__nv_bfloat16*>(a.y)[o]);
    }
    if (ck > 1) cluster.sync();
}

// ------------------------------------------------------------------------------------- host
template <int K, int NT, bool HALF>
int launch(const Args& a, int ck, size_t smem, cudaStream_t st) {
    auto kern = matvec4_kernel<K, NT, HALF>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess)
        return BAKRON_ERR_CUDA;
    const int rows = kWarps * a.tpw * 16, tok = NT * tile_tokens(K);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.m + (long long)rows - 1) / rows * ck),
                       (unsigned)((a.tokens + tok - 1) / tok));
    cfg.blockDim = dim3(kThreads);
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

template <int K>
int plan(Args& a, cudaStream_t st) {
    const Pack4Shape P(a.m, a.n, a.G);
    const int blocks = (P.mt + kWarps - 1) / kWarps;
    // Slices of the columns: as many as keep four tiles a warp, until there are 4 blocks an SM.
    int ck = 1;
    while (ck < 8 && P.kt >= 8 * ck && blocks * ck < 4 * 148) ck *= 2;
    // or as many as bring the staged activations of one product tile into shared memory
    while (ck < 8 && (P.kt + ck - 1) / ck > 64) ck *= 2;
    a.slice = (P.kt + ck - 1) / ck;
    a.tpw = 1;
    const int row_bytes = a.slice * 64 * (K == kI8 ? 1 : 2);
    a.pitch = row_bytes % 128 ? row_bytes : row_bytes + 64;    // odd multiple of 64: no conflicts
    const int rows = kWarps * a.tpw * 16;
    const auto bytes = [&](int nt) {
        const size_t tok = (size_t)nt * tile_tokens(K);
        size_t b = tok * token_rows(K) * a.pitch + tok * rows * 4;
        if (is_book(K)) b += planes(K) * 32768;
        if (a.Gx > 1) b += tok * 4 * ((size_t)a.slice * 64 / a.gx + 2);
        return b;
    };
    int nt = a.tokens <= tile_tokens(K) ? 1 : a.tokens <= 2 * tile_tokens(K) ? 2 : 4;
    while (nt > 1 && bytes(nt) > 110 * 1024) nt /= 2;
    const size_t smem = bytes(nt);
    if (smem > 227 * 1024) return BAKRON_ERR_INVALID_ARG;
    const bool half = (a.G > 1 && a.gs % 64) || (a.Gx > 1 && a.gx % 64);
    if (half)
        return nt == 1 ? launch<K, 1, true>(a, ck, smem, st)
             : nt == 2 ? launch<K, 2, true>(a, ck, smem, st)
                       : launch<K, 4, true>(a, ck, smem, st);
    return nt == 1 ? launch<K, 1, false>(a, ck, smem, st)
         : nt == 2 ? launch<K, 2, false>(a, ck, smem, st)
                   : launch<K, 4, false>(a, ck, smem, st);
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
// the largest. bf16: upper bits, then the rounding of what is left: 16 bits; fp32 takes three parts.
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
    Args a{};
    a.packed = static_cast<const uint8_t*>(packed);
    a.m = m, a.n = n;
    a.G = group_count(group_size, n);
    a.gs = a.G > 1 ? group_size : 64 * ((n + 63) / 64);
    a.x = x, a.x_dtype = x_dtype, a.ldx = ldx, a.xs = x_scales;
    a.Gx = i8 ? group_count(x_group_size, n) : 1;
    a.gx = a.Gx > 1 ? x_group_size : 64 * ((n + 63) / 64);
    a.tokens = tokens, a.y = y, a.y_dtype = y_dtype, a.ldy = ldy;
    a.out1 = a.out2 = 1.f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (codebook) {
        if (x_dtype == BAKRON_F32) {
            split_book<kF32Book>(codebook, 1 << bits, a);
            return plan<kF32Book>(a, st);
        }
        if (x_dtype == BAKRON_BF16) {
            split_book<kBf16Book>(codebook, 1 << bits, a);
            return plan<kBf16Book>(a, st);
        }
        split_book<kF16Book>(codebook, 1 << bits, a);
        return plan<kF16Book>(a, st);
    }
    switch (x_dtype) {
        case BAKRON_F32: return plan<kF32>(a, st);
        case BAKRON_F16: return plan<kF16>(a, st);
        case BAKRON_BF16: return plan<kBf16>(a, st);
        default:
            a.out1 = 1.f / 16.f;      // the codes stand in the upper halves of their bytes
            return plan<kI8>(a, st);
    }
}
