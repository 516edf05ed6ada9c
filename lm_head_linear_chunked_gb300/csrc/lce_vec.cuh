// Element types and vector access of the operators beside the head (layer
// norm, balance loss, beam selection): bf16, fp16 and fp32 values read and
// written in vectors, with all arithmetic in FP32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lce.h"

namespace lce {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// Round to nearest even, the rounding of torch's casts.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// VEC elements read or written at once; the address is a multiple of the size.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T v[VEC];
    __device__ __forceinline__ float f(int i) const { return to_f32(v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_f32<T>(x); }
};

// Elements of T in a 16-byte vector.
template <typename T>
constexpr int vec16() { return 16 / static_cast<int>(sizeof(T)); }

inline size_t dtype_bytes(int dtype) { return dtype == LCE_F32 ? 4 : 2; }
inline bool dtype_known(int dtype) { return dtype == LCE_BF16 || dtype == LCE_F16 || dtype == LCE_F32; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

__device__ __forceinline__ bool aligned_dev(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Calls f with a value of the element type that `dtype` names.
template <typename F>
auto with_dtype(int dtype, F f) {
    if (dtype == LCE_BF16) return f(__nv_bfloat16{});
    if (dtype == LCE_F16) return f(__half{});
    return f(float{});
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

}  // namespace lce
