// norm_q8.cu -- bakron_rms_norm_q8: residual addition, root-mean-square norm, 8-bit codes.
//
//   h = x + residual, rho = 1 / sqrt(mean h^2 + eps), v = h * weight,
//   scale_g = max_g |v| rho / 127, q = round_half_even(127 v / max_g |v|)
//
// rho cancels in the codes, which are therefore those of the inputs alone: v, its maximum and the
// quotient in fp64. One block per row.
#include <cmath>

#include "lowp.cuh"

namespace bakron {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 65536 / 32;

template <class X>
__device__ __forceinline__ double weight_at(const void* w, int wd, int j) {
    if (!w) return 1.0;
    if (wd == BAKRON_F32) return (double)static_cast<const float*>(w)[j];
    if (wd == BAKRON_F16) return (double)to_f32(static_cast<const __half*>(w)[j]);
    return (double)to_f32(static_cast<const __nv_bfloat16*>(w)[j]);
}

template <class X>
__global__ void __launch_bounds__(kThreads)
norm_q8_kernel(const X* x, int64_t ldx, const X* r, int64_t ldr, const void* __restrict__ w,
               int wd, int n, float eps, int gs, int G, int8_t* __restrict__ q,
               float* __restrict__ scales, X* sum, int64_t lds, int* __restrict__ status) {
    __shared__ unsigned long long gmax[kMaxGroups];   // bit patterns of doubles >= 0: ordered
    __shared__ double part[kThreads];
    __shared__ int bad;
    const int64_t row = blockIdx.x;
    for (int g = threadIdx.x; g < G; g += kThreads) gmax[g] = 0;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    x += row * ldx;
    if (r) r += row * ldr;
    double s = 0.0;
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const float xv = to_f32(x[j]), rv = r ? to_f32(r[j]) : 0.f;
        const double h = (double)xv + (double)rv, v = h * weight_at<X>(w, wd, j);
        const float h32 = xv + rv;
        if (!isfinite(h32) || !isfinite((float)v)) bad = 1;
        else atomicMax(&gmax[j / gs], (unsigned long long)__double_as_longlong(fabs(v)));
        s += h * h;
    }
    part[threadIdx.x] = s;
    __syncthreads();
    for (int k = kThreads / 2; k > 0; k >>= 1) {
        if (threadIdx.x < k) part[threadIdx.x] += part[threadIdx.x + k];
        __syncthreads();
    }
    const double rho = 1.0 / sqrt(part[0] / n + (double)eps);
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const float xv = to_f32(x[j]), rv = r ? to_f32(r[j]) : 0.f;
        const double v = ((double)xv + (double)rv) * weight_at<X>(w, wd, j);
        const double top = __longlong_as_double((long long)gmax[j / gs]);
        q[row * n + j] = bad || !(top > 0.0) ? 0 : (int8_t)(int)rint(v * 127.0 / top);
        if (sum) from_f32(xv + rv, sum[row * lds + j]);
    }
    for (int g = threadIdx.x; g < G; g += kThreads)
        scales[row * G + g] =
            bad ? __int_as_float(0x7fc00000)
                : (float)(__longlong_as_double((long long)gmax[g]) * rho / 127.0);
    if (bad && status && threadIdx.x == 0) set_status(status, BAKRON_ERR_NONFINITE);
}

template <int D>
int launch(const void* x, int64_t ldx, const void* r, int64_t ldr, const void* w, int wd,
           int rows, int n, float eps, int gs, int G, int8_t* q, float* scales, void* sum,
           int64_t lds, int* status, cudaStream_t st) {
    using X = typename Elem<D>::T;
    norm_q8_kernel<X><<<rows, kThreads, 0, st>>>(
        static_cast<const X*>(x), ldx, static_cast<const X*>(r), ldr, w, wd, n, eps, gs, G, q,
        scales, static_cast<X*>(sum), lds, status);
    count_launches(1);
    return cuda_err(cudaGetLastError());
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
        !aligned_to(sum, b) || !aligned_to(weight, dtype_bytes(weight_dtype)))
        return BAKRON_ERR_INVALID_ARG;
    const int G = group_count(group_size, n), gs = group_size < n ? group_size : n;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case BAKRON_F32:
            return launch<BAKRON_F32>(x, ldx, residual, ldr, weight, weight_dtype, rows, n, eps,
                                      gs, G, q, scales, sum, lds, dev_status, st);
        case BAKRON_F16:
            return launch<BAKRON_F16>(x, ldx, residual, ldr, weight, weight_dtype, rows, n, eps,
                                      gs, G, q, scales, sum, lds, dev_status, st);
        default:
            return launch<BAKRON_BF16>(x, ldx, residual, ldr, weight, weight_dtype, rows, n, eps,
                                       gs, G, q, scales, sum, lds, dev_status, st);
    }
}
