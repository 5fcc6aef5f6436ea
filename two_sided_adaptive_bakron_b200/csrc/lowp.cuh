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
