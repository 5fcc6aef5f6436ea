// norm_q8.cu -- bakron_rms_norm_q8: residual addition, root-mean-square norm, 8-bit codes.
//
//   h = x + residual, rho = 1 / sqrt(mean h^2 + eps), v = h * weight,
//   scale_g = max_g |v| rho / 127, q = round_half_even(127 v / max_g |v|)
//
// Bound by bytes: x and the residual read once, the sum and the codes written once. One block a row;
// a thread keeps its elements as they were read (one or two chunks of 8, in registers), so that the
// codes need no second read. Rows that do not fit (above 16384 elements, 8192 of fp32) are read
// again, from L2. The blocks of an SM (1024 threads) overlap each other's barriers.
//
// rho cancels in the codes, which are those of the real quotient: v and the quotient are fp32 first
// (relative error below 5 2^-24), and where that leaves the code open -- an element next to its
// group's maximum, a quotient within 2^-14 of the border of two codes -- fp64 decides, in which the
// products of 16-bit inputs are exact. One element in 8000 takes the second way.
#include <cmath>

#include "lowp.cuh"

namespace bakron {
namespace {

constexpr float kNear = 1.f - 0x1p-20f;      // of the maximum: candidates for it
constexpr float kBorder = 0.5f - 0x1p-14f;   // from the nearest code: the other one is as near
constexpr float kTiny = 0x1p-90f;            // below it fp32 quotients lose their relative error

struct Args {
    const void* x; int64_t ldx; const void* r; int64_t ldr; const void* w; int wd;
    int n; float eps; int gs, G, lanes;   // lanes: of a warp that share a group, a power of two
    int8_t* q; float* scales; void* sum; int64_t lds; int* status;
    int wide_x, wide_r, wide_w, wide_sum, wide_q;
};

// 8 elements from column j on; what lies behind the row is zero.
template <class X>
__device__ __forceinline__ void load8(const X* row, int j, int n, bool wide, X (&v)[8]) {
    if (wide && j + 8 <= n) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(X) / 2; ++k)
            reinterpret_cast<uint4*>(v)[k] = reinterpret_cast<const uint4*>(row + j)[k];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            from_f32(0.f, v[k]);
            if (j + k < n) v[k] = row[j + k];
        }
    }
}

template <class W>
__device__ __forceinline__ void weights8(const Args& a, int j, float (&f)[8]) {
    W w[8];
    load8<W>(static_cast<const W*>(a.w), j, a.n, a.wide_w, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = to_f32(w[k]);
}
__device__ __forceinline__ void weights8(const Args& a, int j, float (&f)[8]) {
    if (!a.w) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = 1.f;
    } else if (a.wd == BAKRON_F32) {
        weights8<float>(a, j, f);
    } else if (a.wd == BAKRON_F16) {
        weights8<__half>(a, j, f);
    } else {
        weights8<__nv_bfloat16>(a, j, f);
    }
}

// C: chunks that a thread keeps (0: none, the row is read again).
template <class X, int C, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
norm_q8_kernel(const __grid_constant__ Args a) {
    constexpr int K = C > 0 ? C : 1;
    extern __shared__ __align__(8) char smem[];
    unsigned long long* gmax = reinterpret_cast<unsigned long long*>(smem);   // of doubles >= 0
    unsigned* gmax32 = reinterpret_cast<unsigned*>(gmax + a.G);              // of floats >= 0
    __shared__ double part[THREADS / 32];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, n = a.n;
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    const X* r = a.r ? static_cast<const X*>(a.r) + row * a.ldr : nullptr;
    const int rounds = C > 0 ? C : (n + 8 * THREADS - 1) / (8 * THREADS);

    X xv[K][8], rv[K][8];
    const auto load = [&](int c, X (&xc)[8], X (&rc)[8]) {
        const int j = (c * THREADS + tid) * 8;
        load8<X>(x, j, n, a.wide_x, xc);
        if (r) load8<X>(r, j, n, a.wide_r, rc);
    };
    const auto value = [&](const X (&xc)[8], const X (&rc)[8], const float (&w)[8], float (&h)[8],
                           float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            h[k] = r ? to_f32(xc[k]) + to_f32(rc[k]) : to_f32(xc[k]);
            v[k] = h[k] * w[k];
        }
    };
    const auto exact = [&](X xe, X re, float w) {
        const double h = r ? (double)to_f32(xe) + (double)to_f32(re) : (double)to_f32(xe);
        return h * (double)w;
    };

    if (C > 0) {
#pragma unroll
        for (int c = 0; c < K; ++c) load(c, xv[c], rv[c]);
    }
    for (int g = tid; g < a.G; g += THREADS) gmax[g] = 0, gmax32[g] = 0;
    __syncthreads();

    // sum of squares and the fp32 maxima of the groups
    float ss = 0.f;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < rounds; ++c) {
        const int b = C > 0 ? c : 0, j = (c * THREADS + tid) * 8;
        if (C == 0) load(c, xv[b], rv[b]);
        float w[8], h[8], v[8], top = 0.f;
        weights8(a, j, w);
        value(xv[b], rv[b], w, h, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            ss = fmaf(h[k], h[k], ss);
            top = fmaxf(top, fabsf(v[k]));
            bad |= !(fabsf(h[k]) < INFINITY) || !(fabsf(v[k]) < INFINITY);
        }
        for (int o = 1; o < a.lanes; o <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((tid & (a.lanes - 1)) == 0 && j < n) atomicMax(&gmax32[j / a.gs], __float_as_uint(top));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 31) == 0) part[tid / 32] = ss;
    bad = __syncthreads_or(bad);
    double total = 0.0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) total += part[k];
    if (bad) {
        for (int c = 0; c < rounds; ++c) {
            const int b = C > 0 ? c : 0, j = (c * THREADS + tid) * 8;
            if (C == 0) load(c, xv[b], rv[b]);
            for (int k = 0; k < 8; ++k) {
                if (j + k >= n) break;
                const float h = r ? to_f32(xv[b][k]) + to_f32(rv[b][k]) : to_f32(xv[b][k]);
                a.q[row * n + j + k] = 0;
                if (a.sum) from_f32(h, static_cast<X*>(a.sum)[row * a.lds + j + k]);
            }
        }
        for (int g = tid; g < a.G; g += THREADS) a.scales[row * a.G + g] = NAN;
        if (tid == 0 && a.status) set_status(a.status, BAKRON_ERR_NONFINITE);
        return;
    }
    // squares that leave the range of fp32 are added again in fp64
    if (!(total < 0x1p120) || total < 0x1p-60) {
        double s = 0.0;
        for (int c = 0; c < rounds; ++c) {
            const int b = C > 0 ? c : 0;
            if (C == 0) load(c, xv[b], rv[b]);
            for (int k = 0; k < 8; ++k) {
                const double h = exact(xv[b][k], rv[b][k], 1.f);
                s += h * h;
            }
        }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        __syncthreads();
        if ((tid & 31) == 0) part[tid / 32] = s;
        __syncthreads();
        total = 0.0;
        for (int k = 0; k < THREADS / 32; ++k) total += part[k];
    }

    // the maxima in fp64, from the elements that may be them
#pragma unroll
    for (int c = 0; c < rounds; ++c) {
        const int b = C > 0 ? c : 0, j = (c * THREADS + tid) * 8;
        if (j >= n) break;
        if (C == 0) load(c, xv[b], rv[b]);
        float w[8], h[8], v[8];
        weights8(a, j, w);
        value(xv[b], rv[b], w, h, v);
        const float top = __uint_as_float(gmax32[j / a.gs]);
        const float from = top < kTiny ? 0.f : top * kNear;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (fabsf(v[k]) >= from)
                atomicMax(&gmax[j / a.gs], (unsigned long long)__double_as_longlong(
                                               fabs(exact(xv[b][k], rv[b][k], w[k]))));
    }
    __syncthreads();

    // codes, and the sum
#pragma unroll
    for (int c = 0; c < rounds; ++c) {
        const int b = C > 0 ? c : 0, j = (c * THREADS + tid) * 8;
        if (j >= n) break;
        if (C == 0) load(c, xv[b], rv[b]);
        float w[8], h[8], v[8];
        weights8(a, j, w);
        value(xv[b], rv[b], w, h, v);
        const double top = __longlong_as_double((long long)gmax[j / a.gs]);
        const float inv = (float)(127.0 / top);
        uint32_t out[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float t = v[k] * inv;
            float code = rintf(t);
            if (!(fabsf(t - code) < kBorder) || top < (double)kTiny)
                code = top > 0.0 ? (float)rint(exact(xv[b][k], rv[b][k], w[k]) * 127.0 / top) : 0.f;
            out[k / 4] |= ((uint32_t)(int)code & 0xFFu) << (8 * (k % 4));
        }
        int8_t* q = a.q + row * n + j;
        if (a.wide_q && j + 8 <= n) {
            *reinterpret_cast<uint2*>(q) = make_uint2(out[0], out[1]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (j + k < n) q[k] = (int8_t)(out[k / 4] >> (8 * (k % 4)));
        }
        if (a.sum) {
            X* s = static_cast<X*>(a.sum) + row * a.lds + j;
            __align__(16) X o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) from_f32(h[k], o[k]);
            if (a.wide_sum && j + 8 <= n) {
#pragma unroll
                for (int k = 0; k < (int)sizeof(X) / 2; ++k)
                    reinterpret_cast<uint4*>(s)[k] = reinterpret_cast<const uint4*>(o)[k];
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (j + k < n) s[k] = o[k];
            }
        }
    }
    const double rho = 1.0 / sqrt(total / n + (double)a.eps);
    for (int g = tid; g < a.G; g += THREADS)
        a.scales[row * a.G + g] = (float)(__longlong_as_double((long long)gmax[g]) * rho / 127.0);
}

template <class X, int C, int THREADS>
int launch(const Args& a, int rows, cudaStream_t st) {
    norm_q8_kernel<X, C, THREADS><<<rows, THREADS, (size_t)a.G * 12, st>>>(a);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}

// Threads and chunks by the row's length: one chunk a thread as long as blocks stay small, two where
// they are 16-bit values (8 registers a chunk; fp32 takes 16), nothing kept above 1024 threads' worth.
template <int D>
int plan(const Args& a, int rows, cudaStream_t st) {
    using X = typename Elem<D>::T;
    constexpr bool half = sizeof(X) == 2;
    const int chunks = (a.n + 7) / 8;
    if (chunks <= 64) return launch<X, 1, 64>(a, rows, st);
    if (chunks <= 128) return launch<X, 1, 128>(a, rows, st);
    if (chunks <= 256) return launch<X, 1, 256>(a, rows, st);
    if (chunks <= 512) return half ? launch<X, half ? 2 : 0, 256>(a, rows, st) : launch<X, 1, 512>(a, rows, st);
    if (chunks <= 1024) return half ? launch<X, half ? 2 : 0, 512>(a, rows, st) : launch<X, 1, 1024>(a, rows, st);
    if (half && chunks <= 2048) return launch<X, half ? 2 : 0, 1024>(a, rows, st);
    return launch<X, 0, 1024>(a, rows, st);
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" int bakron_rms_norm_q8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                  int dtype, const void* weight, int weight_dtype, int rows,
                                  int n, float eps, int group_size, int8_t* q, float* scales,
                                  void* sum, int64_t lds, int* dev_status, void* stream) {
    if (!float_dtype(dtype) || (weight && !float_dtype(weight_dtype)) || rows < 0 || n < 1 ||
        n > 65536 || !(eps > 0.f) || !std::isfinite(eps) || !group_ok(group_size, n) ||
        ldx < n || (residual && ldr < n) || (sum && lds < n))
        return BAKRON_ERR_INVALID_ARG;
    if (rows == 0) return BAKRON_OK;
    const size_t b = dtype_bytes(dtype);
    if (!x || !q || !scales || !aligned_to(x, b) || !aligned_to(residual, b) ||
        !aligned_to(sum, b) || (weight && !aligned_to(weight, dtype_bytes(weight_dtype))))
        return BAKRON_ERR_INVALID_ARG;
    Args a{x, ldx, residual, ldr, weight, weight_dtype, n, eps, 0, 0, 0, q, scales, sum, lds,
           dev_status};
    a.G = group_count(group_size, n);
    a.gs = a.G > 1 ? group_size : n;
    // lanes of a warp whose chunks lie in one group: the power of two in the group's chunks
    a.lanes = 32;
    while (a.G > 1 && (a.gs / 8) % a.lanes) a.lanes /= 2;
    const auto rows16 = [&](const void* p, int64_t ld) {
        return p && aligned_to(p, 16) && ld * (int64_t)b % 16 == 0;
    };
    a.wide_x = rows16(x, ldx);
    a.wide_r = rows16(residual, ldr);
    a.wide_sum = rows16(sum, lds);
    a.wide_w = weight && aligned_to(weight, 16);
    a.wide_q = n % 8 == 0 && aligned_to(q, 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case BAKRON_F32: return plan<BAKRON_F32>(a, rows, st);
        case BAKRON_F16: return plan<BAKRON_F16>(a, rows, st);
        default: return plan<BAKRON_BF16>(a, rows, st);
    }
}
