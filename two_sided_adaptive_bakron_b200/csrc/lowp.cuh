// lowp.cuh -- element types of the 16-bit and 8-bit entry points (matvec4, norm_q8, distill).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace bakron {

// The C type of a bakron_dtype.
template <int DT> struct Elem;
template <> struct Elem<BAKRON_F32> { using T = float; };
template <> struct Elem<BAKRON_F16> { using T = __half; };
template <> struct Elem<BAKRON_BF16> { using T = __nv_bfloat16; };
template <> struct Elem<BAKRON_I8> { using T = int8_t; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(int8_t v) { return (float)v; }

// Round to nearest even, once.
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// The elements of 16 bytes as fp32 and back, the larger ones of two vectors, the largest of one (NaN
// loses).
template <class X> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ uint4 top(const uint4& a, const uint4& b) {
        const auto f = [](uint32_t x, uint32_t y) {
            return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
        };
        return make_uint4(f(a.x, b.x), f(a.y, b.y), f(a.z, b.z), f(a.w, b.w));
    }
    static __device__ __forceinline__ float most(const uint4& a) {
        return fmaxf(fmaxf(__uint_as_float(a.x), __uint_as_float(a.y)),
                     fmaxf(__uint_as_float(a.z), __uint_as_float(a.w)));
    }
    static __device__ __forceinline__ uint4 fill_low() {
        return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
    }
};
template <> struct Vec<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
            f[2 * k] = p.x, f[2 * k + 1] = p.y;
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 p = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    static __device__ __forceinline__ uint4 top(const uint4& a, const uint4& b) {
        const auto f = [](uint32_t x, uint32_t y) {
            const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&x),
                                      *reinterpret_cast<const __half2*>(&y));
            return *reinterpret_cast<const uint32_t*>(&m);
        };
        return make_uint4(f(a.x, b.x), f(a.y, b.y), f(a.z, b.z), f(a.w, b.w));
    }
    static __device__ __forceinline__ float most(const uint4& a) {
        const __half2 *p = reinterpret_cast<const __half2*>(&a);
        const float2 f = __half22float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ uint4 fill_low() {
        return make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = __uint_as_float(u[k] << 16);
            f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    static __device__ __forceinline__ uint4 top(const uint4& a, const uint4& b) {
        const auto f = [](uint32_t x, uint32_t y) {
            const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                      *reinterpret_cast<const __nv_bfloat162*>(&y));
            return *reinterpret_cast<const uint32_t*>(&m);
        };
        return make_uint4(f(a.x, b.x), f(a.y, b.y), f(a.z, b.z), f(a.w, b.w));
    }
    static __device__ __forceinline__ float most(const uint4& a) {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162*>(&a);
        const float2 f = __bfloat1622float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ uint4 fill_low() {
        return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
    }
};

inline bool float_dtype(int d) { return d == BAKRON_F32 || d == BAKRON_F16 || d == BAKRON_BF16; }
inline int dtype_bytes(int d) {
    return d == BAKRON_F32 || d == BAKRON_I32 ? 4 : d == BAKRON_I64 ? 8 : d == BAKRON_I8 ? 1 : 2;
}
inline bool aligned_to(const void* p, size_t a) {
    return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// Columns per step, as the entry points take it: a multiple of 32, or one step per row.
inline bool group_ok(int group, int n) { return group >= 1 && (group >= n || group % 32 == 0); }
inline int group_count(int group, int n) { return group >= n ? 1 : (n + group - 1) / group; }

}  // namespace bakron
