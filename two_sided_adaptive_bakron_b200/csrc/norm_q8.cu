// norm_q8.cu -- bakron_rms_norm_q8: residual addition, root-mean-square norm, 8-bit codes.
//
//   h = x + residual, rho = 1 / sqrt(mean h^2 + eps), v = h * weight,
//   scale_g = max_g |v| rho / 127, q = round_half_even(127 v / max_g |v|)
//
// Bound by bytes: x and the residual read once, the sum and the codes written once; 7 bytes of a
// 16-bit element leave about 38 instruction slots of a lane. One block a row, 8 elements (a chunk) a
// thread and round.
//
// rho cancels in the codes, which are those of the real quotient for the given inputs. So where a
// group's maximum is known, its codes are: groups of 32, 64, 128 or 256 columns lie within a warp's
// round, and a row is one pass without a barrier, but for the sum of squares, which only the scales
// need. Other groups (a whole row) meet in shared memory after a first pass; their elements stay in
// registers (one or two chunks a thread; longer rows are read again, from L2).
//
// v, its maximum and the quotient are fp32 (two roundings each of v and the maximum, two for the
// reciprocal, two products: 8 2^-24, 6.1e-5 of a code at most). Where that leaves the code open --
// within 2^-14 of the border of two codes, one element in 8000 -- fp64 decides, with the group's
// maximum in fp64; the products of 16-bit inputs are exact there.
//
// Measured: 2048 x 8192 bf16 with a residual, groups of 128: 34.0 us (3.5 TB/s; issue 62%, DRAM 30%: no
// unit is at its limit, but a block has only one round of loads on its way ahead), one group a row 42.8;
// fp32 45.8 (4.8 TB/s). Blocks of 128 threads for groups within a warp: 33.3 us, of 256 35.1, of 384
// 41.3, of 512 54.6.
#include <cmath>

#include "lowp.cuh"
#include "tcgemm_host.cuh"

namespace bakron {
namespace {

constexpr float kNear = 1.f - 0x1p-20f;      // of the fp32 maximum: candidates for the exact one
constexpr float kBorder = 0.5f - 0x1p-14f;   // from the nearest code: the next one may be as near
constexpr float kTiny = 0x1p-90f;            // below it fp32 products lose their relative error,
constexpr float kHuge = 0x1p120f;            // above it reciprocals do
constexpr float kMagic = 12582912.f;         // 1.5 2^23: adding it leaves the nearest integer (ties
                                             // to even) in the lowest bits

struct Args {
    const void* x; int64_t ldx; const void* r; int64_t ldr; const void* w; int wd;
    int n; float eps; int gs, G, lanes;   // lanes: of a warp that share a group, a power of two
    int8_t* q; float* scales; void* sum; int64_t lds; int* status;
    int wide_x, wide_r, wide_w, wide_sum, wide_q, same_w;
};

// 8 neighbouring elements as they stand in memory. WIDE: rows of whole, aligned chunks.
template <class X, bool WIDE> struct Elements {
    static constexpr int V = sizeof(X) / 2;
    uint4 v[V];
    // from column j on; what lies behind the row is zero
    __device__ __forceinline__ void load(const X* row, int j, int n, bool wide) {
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[k] = j < n ? reinterpret_cast<const uint4*>(row + j)[k] : make_uint4(0, 0, 0, 0);
        } else if (wide && j + 8 <= n) {
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = reinterpret_cast<const uint4*>(row + j)[k];
        } else {
            __align__(16) X e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                from_f32(0.f, e[k]);
                if (j + k < n) e[k] = row[j + k];
            }
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = reinterpret_cast<const uint4*>(e)[k];
        }
    }
    __device__ __forceinline__ void store(X* row, int j, int n, bool wide) const {
        if (WIDE || (wide && j + 8 <= n)) {
#pragma unroll
            for (int k = 0; k < V; ++k) reinterpret_cast<uint4*>(row + j)[k] = v[k];
        } else {
            __align__(16) X e[8];
#pragma unroll
            for (int k = 0; k < V; ++k) reinterpret_cast<uint4*>(e)[k] = v[k];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (j + k < n) row[j + k] = e[k];
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float part[8 / V];
            Vec<X>::get(v[k], part);
#pragma unroll
            for (int c = 0; c < 8 / V; ++c) f[k * (8 / V) + c] = part[c];
        }
    }
    __device__ __forceinline__ void put(const float (&f)[8]) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float part[8 / V];
#pragma unroll
            for (int c = 0; c < 8 / V; ++c) part[c] = f[k * (8 / V) + c];
            v[k] = Vec<X>::put(part);
        }
    }
};

template <class W>
__device__ __forceinline__ void weights8(const Args& a, int j, float (&f)[8]) {
    Elements<W, false> w;
    w.load(static_cast<const W*>(a.w), j, a.n, a.wide_w);
    w.get(f);
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

// Weights of x's type are loaded ahead as they stand, others where they are used.
template <class X, bool WIDE>
__device__ __forceinline__ void weights_ahead(const Args& a, int j, Elements<X, WIDE>& w) {
    if (WIDE || a.same_w) w.load(static_cast<const X*>(a.w), j, a.n, a.wide_w);
}
template <class X, bool WIDE>
__device__ __forceinline__ void weights8(const Args& a, int j, const Elements<X, WIDE>& w,
                                         float (&f)[8]) {
    if (WIDE || a.same_w) w.get(f);
    else weights8(a, j, f);
}

// One row, as a block's threads see it.
template <class X, bool WIDE> struct Row {
    using Chunk = Elements<X, WIDE>;
    const Args& a;
    int64_t row;
    const X *x, *r;
    __device__ __forceinline__ explicit Row(const Args& args, int64_t i)
        : a(args), row(i), x(static_cast<const X*>(args.x) + i * args.ldx),
          r(args.r ? static_cast<const X*>(args.r) + i * args.ldr : nullptr) {}
    __device__ __forceinline__ void load(int j, Chunk& xc, Chunk& rc) const {
        xc.load(x, j, a.n, a.wide_x);
        if (r) rc.load(r, j, a.n, a.wide_r);
    }
    __device__ __forceinline__ void sums(const Chunk& xc, const Chunk& rc,
                                         float (&h)[8]) const {
        xc.get(h);
        if (r) {
            float f[8];
            rc.get(f);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] += f[k];
        }
    }
    __device__ __forceinline__ void put_sum(int j, const float (&h)[8]) const {
        if (!a.sum || j >= a.n) return;
        Chunk o;
        o.put(h);
        o.store(static_cast<X*>(a.sum) + row * a.lds, j, a.n, a.wide_sum);
    }
    // v of the chunk's elements in fp64, one after another: f(k, v)
    template <class F>
    __device__ __forceinline__ void exact(int j, const Chunk& xc, const Chunk& rc, F f) const {
        float xf[8], rf[8], w[8];
        xc.get(xf);
        if (r) rc.get(rf);
        weights8(a, j, w);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            f(k, (r ? (double)xf[k] + (double)rf[k] : (double)xf[k]) * (double)w[k]);
    }
    // Adds the squares of a chunk: in fp32, or in fp64 where they leave its range.
    __device__ __forceinline__ void squares(const Chunk& xc, const Chunk& rc,
                                            const float (&h)[8], float& ss, double& far) const {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(h[k], h[k], s);
        if (s < 0x1p100f && s >= 0x1p-60f) {
            ss += s;
        } else {
            float xf[8], rf[8];
            xc.get(xf);
            if (r) rc.get(rf);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const double d = r ? (double)xf[k] + (double)rf[k] : (double)xf[k];
                far += d * d;
            }
        }
    }
    // Codes of a chunk for its group's maximum: packed, and whether fp64 has to decide one (also
    // where a v is not finite: NaN wins in `far`).
    static __device__ __forceinline__ bool codes(const float (&v)[8], float top, uint2& out) {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(top));
        inv *= 127.f;
        const bool usual = top >= kTiny && top <= kHuge;
        if (!usual) inv = top * 0.f;
        uint32_t bits[8];
        float far = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float t = v[k] * inv, u = t + kMagic;
            bits[k] = __float_as_uint(u);
            const float d = fabsf(t - (u - kMagic));
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(far) : "f"(d));
        }
        out.x = __byte_perm(__byte_perm(bits[0], bits[1], 0x0040),
                            __byte_perm(bits[2], bits[3], 0x0040), 0x5410);
        out.y = __byte_perm(__byte_perm(bits[4], bits[5], 0x0040),
                            __byte_perm(bits[6], bits[7], 0x0040), 0x5410);
        return !(far <= kBorder) || !usual;
    }
    __device__ __forceinline__ uint2 exact_codes(int j, const Chunk& xc, const Chunk& rc,
                                                 double top) const {
        uint32_t out[2] = {0, 0};
        if (top > 0.0)
            exact(j, xc, rc, [&](int k, double v) {
                out[k / 4] |= ((uint32_t)(int)rint(v * 127.0 / top) & 0xFFu) << (8 * (k % 4));
            });
        return make_uint2(out[0], out[1]);
    }
    __device__ __forceinline__ void put_codes(int j, uint2 c) const {
        int8_t* q = a.q + row * a.n + j;
        if (WIDE || (a.wide_q && j + 8 <= a.n)) {
            *reinterpret_cast<uint2*>(q) = c;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (j + k < a.n) q[k] = (int8_t)((k < 4 ? c.x : c.y) >> (8 * (k % 4)));
        }
    }
};

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The end of a row, by all threads: the sum of squares (fp32 parts, fp64 ones where there are any)
// and the scales from the groups' maxima, or a row that is not finite: codes 0, scales NaN.
template <int THREADS, class F>
__device__ __forceinline__ void finish(const Args& a, int64_t row, bool nan, float ss, double far,
                                       double* part64, float* part, F vmax) {
    const int tid = threadIdx.x;
    ss = warp_sum(ss);
    if ((tid & 31) == 0) part[tid / 32] = ss;
    const bool odd = __syncthreads_or(nan || far != 0.0 || !(ss < INFINITY));
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) t += part[k];
    if (!odd) {
        const float s = 127.f * sqrtf(t / (float)a.n + a.eps);
        for (int g = tid; g < a.G; g += THREADS) {
            const double v = vmax(g);
            a.scales[row * a.G + g] = v < (double)kTiny ? (float)(v / (double)s) : (float)v / s;
        }
        return;
    }
    far = warp_sum(far);
    if ((tid & 31) == 0) part64[tid / 32] = far;
    nan = __syncthreads_or(nan);
    double total = t;
    for (int k = 0; k < THREADS / 32; ++k) total += part64[k];
    if (nan || !(total < INFINITY)) {
        for (int j = tid; j < a.n; j += THREADS) a.q[row * a.n + j] = 0;
        for (int g = tid; g < a.G; g += THREADS) a.scales[row * a.G + g] = NAN;
        if (tid == 0 && a.status) set_status(a.status, BAKRON_ERR_NONFINITE);
        return;
    }
    for (int g = tid; g < a.G; g += THREADS)
        a.scales[row * a.G + g] = (float)(vmax(g) / (127.0 * sqrt(total / a.n + (double)a.eps)));
}

__device__ __forceinline__ bool any_not_finite(const float (&v)[8]) {
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) bad |= !(fabsf(v[k]) < INFINITY);
    return bad;
}

// Groups within a warp's round.
template <class X, int THREADS, bool WIDE>
__global__ void __launch_bounds__(THREADS, THREADS > 512 ? 1 : 768 / THREADS)
norm_q8_groups_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(8) char smem[];
    double* vmax = reinterpret_cast<double*>(smem);      // of the groups
    __shared__ double part64[THREADS / 32];
    __shared__ float part[THREADS / 32];
    using Rw = Row<X, WIDE>;
    const Rw R(a, blockIdx.x);
    const int tid = threadIdx.x;
    bool nan = false;                // whether a v is not finite
    float ss = 0.f;
    double far = 0.0;
    typename Rw::Chunk x0, r0, w0, x1, r1, w1;
    R.load(tid * 8, x0, r0);
    weights_ahead(a, tid * 8, w0);
    for (int j0 = 0; j0 < a.n; j0 += THREADS * 8) {
        const int j = j0 + tid * 8;
        if (j0 + THREADS * 8 < a.n) {
            R.load(j + THREADS * 8, x1, r1);
            weights_ahead(a, j + THREADS * 8, w1);
        }
        float h[8], w[8], v[8], top = 0.f;
        R.sums(x0, r0, h);
        weights8(a, j, w0, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = h[k] * w[k];
            top = fmaxf(top, fabsf(v[k]));
        }
        R.squares(x0, r0, h, ss, far);
        R.put_sum(j, h);
        for (int o = 1; o < a.lanes; o <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        uint2 c;
        const bool doubt = Rw::codes(v, top, c);
        double exact_top = (double)top;
        if (__any_sync(0xffffffffu, doubt && j < a.n)) {
            // the maximum in fp64, from the elements that may be it
            const float from = top < kTiny ? 0.f : top * kNear;
            exact_top = 0.0;
            R.exact(j, x0, r0, [&](int k, double e) {
                if (fabsf(v[k]) >= from) exact_top = fmax(exact_top, fabs(e));
            });
            for (int o = 1; o < a.lanes; o <<= 1)
                exact_top = fmax(exact_top, __shfl_xor_sync(0xffffffffu, exact_top, o));
            if (doubt) nan |= any_not_finite(v), c = R.exact_codes(j, x0, r0, exact_top);
        }
        if (j < a.n) {
            R.put_codes(j, c);
            if ((tid & (a.lanes - 1)) == 0) vmax[j / a.gs] = exact_top;
        }
        x0 = x1, r0 = r1, w0 = w1;
    }
    finish<THREADS>(a, R.row, nan, ss, far, part64, part, [&](int g) { return vmax[g]; });
}

// Any groups. C: chunks that a thread keeps (0: none, the row is read again).
template <class X, int C, int THREADS, bool WIDE>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
norm_q8_kernel(const __grid_constant__ Args a) {
    constexpr int K = C > 0 ? C : 1;      // (indices of kept chunks are constants)
    extern __shared__ __align__(8) char smem[];
    unsigned long long* gmax = reinterpret_cast<unsigned long long*>(smem);   // of doubles >= 0
    unsigned* gmax32 = reinterpret_cast<unsigned*>(gmax + a.G);              // of floats >= 0
    __shared__ double part64[THREADS / 32];
    __shared__ float part[THREADS / 32];
    using Rw = Row<X, WIDE>;
    const Rw R(a, blockIdx.x);
    const int tid = threadIdx.x, n = a.n;
    const int rounds = C > 0 ? C : (n + 8 * THREADS - 1) / (8 * THREADS);
    typename Rw::Chunk xc[K], rc[K];
    float v[K][8], most[K];
    const auto column = [&](int c) { return (c * THREADS + tid) * 8; };

    if (C > 0) {
#pragma unroll
        for (int c = 0; c < K; ++c) R.load(column(c), xc[c], rc[c]);
    }
    for (int g = tid; g < a.G; g += THREADS) gmax[g] = 0, gmax32[g] = 0;
    __syncthreads();

    bool nan = false;                // whether a v is not finite
    float ss = 0.f;
    double far = 0.0;
    const auto values = [&](int c, int b, float (&h)[8]) {
        float w[8];
        if (C == 0) R.load(column(c), xc[b], rc[b]);
        weights8(a, column(c), w);
        R.sums(xc[b], rc[b], h);
        most[b] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[b][k] = h[k] * w[k];
            most[b] = fmaxf(most[b], fabsf(v[b][k]));
        }
    };
#pragma unroll(K)
    for (int c = 0; c < rounds; ++c) {
        const int b = C > 0 ? c : 0, j = column(c);
        float h[8];
        values(c, b, h);
        R.squares(xc[b], rc[b], h, ss, far);
        if (C > 0) R.put_sum(j, h);       // (the elements of this row are all in registers)
        float top = most[b];
        for (int o = 1; o < a.lanes; o <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((tid & (a.lanes - 1)) == 0 && j < n) atomicMax(&gmax32[j / a.gs], __float_as_uint(top));
    }
    __syncthreads();

    // codes; the maxima in fp64 meanwhile, from the elements that may be them
    unsigned doubt = 0;              // chunks with a code that fp64 decides
#pragma unroll(K)
    for (int c = 0; c < rounds; ++c) {
        const int b = C > 0 ? c : 0, j = column(c);
        if (j >= n) break;
        float h[8];
        if (C == 0) values(c, b, h);
        const int g = a.G > 1 ? j / a.gs : 0;
        const float top = __uint_as_float(gmax32[g]), from = top < kTiny ? 0.f : top * kNear;
        if (most[b] >= from) {
            double e = 0.0;
            R.exact(j, xc[b], rc[b], [&](int k, double d) {
                if (fabsf(v[b][k]) >= from) e = fmax(e, fabs(d));
            });
            atomicMax(&gmax[g], (unsigned long long)__double_as_longlong(e));
        }
        uint2 q;
        if (Rw::codes(v[b], top, q)) doubt |= 1u << c, nan |= any_not_finite(v[b]);
        R.put_codes(j, q);
    }
    __syncthreads();
#pragma unroll(K)
    for (int c = 0; c < rounds; ++c) {
        if (!(doubt >> c & 1)) continue;
        const int b = C > 0 ? c : 0, j = column(c);
        if (C == 0) R.load(j, xc[b], rc[b]);
        R.put_codes(j, R.exact_codes(j, xc[b], rc[b],
                                     __longlong_as_double((long long)gmax[j / a.gs])));
    }
    if (C == 0 && a.sum) {
        // last, for the sum may take the place of what was read
        for (int c = 0; c < rounds; ++c) {
            float h[8];
            R.load(column(c), xc[0], rc[0]);
            R.sums(xc[0], rc[0], h);
            R.put_sum(column(c), h);
        }
    }
    finish<THREADS>(a, R.row, nan, ss, far, part64, part,
                    [&](int g) { return __longlong_as_double((long long)gmax[g]); });
}

template <class X, int C, int THREADS, bool WIDE>
int launch(const Args& a, int rows, cudaStream_t st) {
    norm_q8_kernel<X, C, THREADS, WIDE><<<rows, THREADS, (size_t)a.G * 12, st>>>(a);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}
template <class X, int THREADS, bool WIDE>
int launch_groups(const Args& a, int rows, cudaStream_t st) {
    norm_q8_groups_kernel<X, THREADS, WIDE><<<rows, THREADS, (size_t)a.G * 8, st>>>(a);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}

// Threads by the row's length: a block goes over a row of groups in rounds, with the next one's loads
// ahead. Where a row meets in shared memory, one chunk a thread as long as
// blocks stay small, two where they are 16-bit values (fp32 takes twice the registers), nothing kept
// above 1024 threads' worth.
template <class X, bool WIDE>
int plan(const Args& a, int rows, int sms, cudaStream_t st) {
    constexpr bool half = sizeof(X) == 2;
    const int chunks = (a.n + 7) / 8;
    if (a.G > 1 && 256 % a.gs == 0) {
        // many rows: long rounds of small blocks; few rows: as many threads as help one row
        if (chunks <= 64) return launch_groups<X, 64, WIDE>(a, rows, st);
        if (chunks <= 128 || rows >= 4 * sms) return launch_groups<X, 128, WIDE>(a, rows, st);
        return launch_groups<X, 512, WIDE>(a, rows, st);
    }
    if (chunks <= 64) return launch<X, 1, 64, WIDE>(a, rows, st);
    if (chunks <= 128) return launch<X, 1, 128, WIDE>(a, rows, st);
    if (chunks <= 256) return launch<X, 1, 256, WIDE>(a, rows, st);
    if (half) {
        if (chunks <= 512) return launch<X, half ? 2 : 0, 256, WIDE>(a, rows, st);
        if (chunks <= 1024) return launch<X, half ? 2 : 0, 512, WIDE>(a, rows, st);
        if (chunks <= 2048) return launch<X, half ? 2 : 0, 1024, WIDE>(a, rows, st);
    } else {
        if (chunks <= 512) return launch<X, half ? 0 : 1, 512, WIDE>(a, rows, st);
        if (chunks <= 1024) return launch<X, half ? 0 : 1, 1024, WIDE>(a, rows, st);
    }
    return launch<X, 0, 1024, WIDE>(a, rows, st);
}

template <int D>
int plan(const Args& a, int rows, cudaStream_t st) {
    using X = typename Elem<D>::T;
    const bool wide = a.n % 8 == 0 && a.wide_x && (!a.r || a.wide_r) && a.wide_w && a.same_w &&
                      (!a.sum || a.wide_sum) && a.wide_q;
    const int sms = tc::sm_count();
    if (sms <= 0) return BAKRON_ERR_CUDA;
    return wide ? plan<X, true>(a, rows, sms, st) : plan<X, false>(a, rows, sms, st);
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
        ldx < n || (residual && ldr < n) || (sum && lds < n) ||
        (rows > 1 && sum && ((sum == x && lds != ldx) || (sum == residual && lds != ldr))))
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
    a.same_w = weight && weight_dtype == dtype;
    a.wide_q = n % 8 == 0 && aligned_to(q, 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case BAKRON_F32: return plan<BAKRON_F32>(a, rows, st);
        case BAKRON_F16: return plan<BAKRON_F16>(a, rows, st);
        default: return plan<BAKRON_BF16>(a, rows, st);
    }
}
