// distill.cu -- bakron_distill: the distillation loss from a teacher's top logits and its gradient.
//
//   q = softmax(z / tau),  p_j = exp(t_j / tau - T),
//   loss = w sum_j p_j (log p_j - log q_{i_j}),   dz_i = (w / tau) (M q_i - sum_{j: i_j = i} p_j)
//
// One block per row: one pass with the running maximum and sum of each thread, the block's total,
// then the gradient from a second look at the row. All statistics are fp32.
#include <cmath>

#include "lowp.cuh"

namespace bakron {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxK = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -INFINITY;

// Joins the pairs (m, s) and (m2, s2) that stand for s 2^(c m) and s2 2^(c m2).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float c) {
    const float top = fmaxf(m, m2);
    if (top == kNegInf) {           // two empty parts (or NaN)
        s += s2;
        return;
    }
    s = s * exp2f((m - top) * c) + s2 * exp2f((m2 - top) * c);
    m = top;
}

struct Teacher {
    const void* idx; int idx64; const void* t; int td; int k;
    const float* lse; const float* w; float inv_tau;
};

__device__ __forceinline__ long long index_at(const Teacher& T, size_t e) {
    return T.idx64 ? static_cast<const long long*>(T.idx)[e] : static_cast<const int*>(T.idx)[e];
}
__device__ __forceinline__ float logit_at(const Teacher& T, size_t e) {
    if (T.td == BAKRON_F32) return static_cast<const float*>(T.t)[e];
    if (T.td == BAKRON_F16) return to_f32(static_cast<const __half*>(T.t)[e]);
    return to_f32(static_cast<const __nv_bfloat16*>(T.t)[e]);
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
    for (int k = 0; k < kThreads / 32; ++k) s += red[k];
    return s;
}
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = kNegInf;
    for (int k = 0; k < kThreads / 32; ++k) s = fmaxf(s, red[k]);
    return s;
}

template <class X>
__global__ void __launch_bounds__(kThreads)
distill_kernel(const X* z, int V, int64_t ld, Teacher T, float* __restrict__ loss,
               float* __restrict__ lse, X* dz, int64_t ldd, int* __restrict__ status) {
    __shared__ float red[2][kThreads / 32];
    __shared__ float p[kMaxK], zt[kMaxK];
    __shared__ int at[kMaxK];
    const int row = blockIdx.x, tid = threadIdx.x;
    const float w = T.w ? T.w[row] : 1.f;
    z += (int64_t)row * ld;
    if (dz) dz += (int64_t)row * ldd;
    if (w == 0.f) {
        if (tid == 0) loss[row] = 0.f, lse[row] = 0.f;
        if (dz)
            for (int i = tid; i < V; i += kThreads) from_f32(0.f, dz[i]);
        return;
    }
    // the teacher's list; differences from a maximum are taken before they are scaled, so that
    // nothing large cancels in log p - log q
    float tmax = kNegInf;
    for (int j = tid; j < T.k; j += kThreads) {
        const size_t e = (size_t)row * T.k + j;
        const long long i = index_at(T, e);
        const float t = logit_at(T, e);
        if (i >= V) set_status(status, BAKRON_ERR_INVALID_ARG);
        const bool there = i >= 0 && i < V && t != kNegInf;
        at[j] = there ? (int)i : -1;
        p[j] = t;
        zt[j] = there ? to_f32(z[i]) : 0.f;
        if (there) tmax = fmaxf(tmax, t);
    }
    float tl = 0.f;      // log p_j = (t_j - tmax) / tau - tl
    if (T.lse) {
        tmax = 0.f;
        tl = T.lse[row];
    } else {
        tmax = block_max(tmax, red[0]);
        float s = 0.f;
        for (int j = tid; j < T.k; j += kThreads)
            if (at[j] >= 0) s += expf((p[j] - tmax) * T.inv_tau);
        tl = logf(block_sum(s, red[0]));
    }
    // the row: its maximum m and s = sum 2^(c (z - m))
    const float c = T.inv_tau * kLog2e;
    float m = kNegInf, s = 0.f;
    for (int i = tid; i < V; i += kThreads) {
        const float v = to_f32(z[i]);
        if (v > m) {
            s = s * exp2f((m - v) * c) + 1.f;
            m = v;
        } else if (v != kNegInf) {
            s += exp2f((v - m) * c);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o), c);
    __syncthreads();
    if ((tid & 31) == 0) red[0][tid / 32] = m, red[1][tid / 32] = s;
    __syncthreads();
    m = red[0][0], s = red[1][0];
    for (int k = 1; k < kThreads / 32; ++k) join(m, s, red[0][k], red[1][k], c);
    if (fabsf(m) == INFINITY) s = NAN;      // +inf, or nothing but -inf
    const float l = logf(s);
    float kl = 0.f, mass = 0.f;
    for (int j = tid; j < T.k; j += kThreads) {
        float pj = 0.f;
        if (at[j] >= 0) {
            const float lp = (p[j] - tmax) * T.inv_tau - tl;
            pj = expf(lp);
            if (pj != 0.f) kl += pj * (lp - ((zt[j] - m) * T.inv_tau - l));
        }
        p[j] = pj;
        mass += pj;
    }
    kl = block_sum(kl, red[0]);
    mass = block_sum(mass, red[0]);
    if (tid == 0) loss[row] = w * kl, lse[row] = m * T.inv_tau + l;
    if (!dz) return;
    const float f = w * T.inv_tau;
    const float fq = mass == 0.f ? 0.f : f * mass / s;
    for (int i = tid; i < V; i += kThreads)
        from_f32(mass == 0.f ? 0.f : fq * exp2f((to_f32(z[i]) - m) * c), dz[i]);
    __syncthreads();
    for (int j = tid; j < T.k; j += kThreads) {
        if (at[j] < 0 || mass == 0.f) continue;
        float pj = 0.f;
        for (int k = 0; k < T.k; ++k) pj += at[k] == at[j] ? p[k] : 0.f;
        from_f32(fq * exp2f((zt[j] - m) * c) - f * pj, dz[at[j]]);
    }
}

template <int D>
int launch(const void* z, int rows, int V, int64_t ld, const Teacher& T, float* loss, float* lse,
           void* dz, int64_t ldd, int* status, cudaStream_t st) {
    using X = typename Elem<D>::T;
    distill_kernel<X><<<rows, kThreads, 0, st>>>(static_cast<const X*>(z), V, ld, T, loss, lse,
                                                 static_cast<X*>(dz), ldd, status);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" int bakron_distill(const void* logits, int dtype, int rows, int vocab, int64_t ld,
                              const void* top_idx, int idx_dtype, const void* top_logits,
                              int top_dtype, int k, const float* teacher_lse,
                              const float* row_weights, float temperature, float* loss,
                              float* lse, void* dlogits, int64_t ldd, int* dev_status,
                              void* stream) {
    if (!float_dtype(dtype) || !float_dtype(top_dtype) ||
        (idx_dtype != BAKRON_I32 && idx_dtype != BAKRON_I64) || rows < 0 || vocab < 1 ||
        ld < vocab || (dlogits && ldd < vocab) || (dlogits == logits && dlogits && ldd != ld) ||
        k < 1 || k > kMaxK || !(temperature > 0.f) || !std::isfinite(temperature) ||
        !std::isfinite(1.f / temperature))
        return BAKRON_ERR_INVALID_ARG;
    if (rows == 0) return BAKRON_OK;
    if (!logits || !top_idx || !top_logits || !loss || !lse || !dev_status ||
        !aligned_to(logits, dtype_bytes(dtype)) || !aligned_to(dlogits, dtype_bytes(dtype)) ||
        !aligned_to(top_idx, dtype_bytes(idx_dtype)) ||
        !aligned_to(top_logits, dtype_bytes(top_dtype)))
        return BAKRON_ERR_INVALID_ARG;
    const Teacher T{top_idx, idx_dtype == BAKRON_I64, top_logits, top_dtype, k, teacher_lse,
                    row_weights, 1.f / temperature};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case BAKRON_F32:
            return launch<BAKRON_F32>(logits, rows, vocab, ld, T, loss, lse, dlogits, ldd,
                                      dev_status, st);
        case BAKRON_F16:
            return launch<BAKRON_F16>(logits, rows, vocab, ld, T, loss, lse, dlogits, ldd,
                                      dev_status, st);
        default:
            return launch<BAKRON_BF16>(logits, rows, vocab, ld, T, loss, lse, dlogits, ldd,
                                       dev_status, st);
    }
}
