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

// VEC elements read or written at once; the address is a multiple of the size,
// or of 16 bytes for larger ones.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Vec {
    T v[VEC];
    __device__ __forceinline__ float f(int i) const { return to_f32(v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_f32<T>(x); }
};

// Two FP32 values in one 64-bit register: sm_100's packed add, multiply and
// fused multiply-add round each half as the scalar instruction does, at one
// issue slot for the two.
struct F2 {
    uint64_t u;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float lo(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.u)); }
__device__ __forceinline__ float hi(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.u >> 32)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
    return r;
}

// 2^x by the hardware's approximation (relative error 2^-22), 0 below 2^-126.
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / x by the hardware's approximation (one unit in the last place).
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two neighbouring elements as a pair, and back (rounded to nearest even).
__device__ __forceinline__ F2 pair_of(const float* v) { return f2(v[0], v[1]); }
__device__ __forceinline__ F2 pair_of(const __nv_bfloat16* v) {
    uint32_t u;
    __builtin_memcpy(&u, v, 4);
    return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ F2 pair_of(const __half* v) { return f2(__half2float(v[0]), __half2float(v[1])); }
__device__ __forceinline__ void set_pair(float* v, F2 a) {
    v[0] = lo(a);
    v[1] = hi(a);
}
__device__ __forceinline__ void set_pair(__nv_bfloat16* v, F2 a) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo(a), hi(a));
    __builtin_memcpy(v, &r, 4);
}
__device__ __forceinline__ void set_pair(__half* v, F2 a) {
    const __half2 r = __floats2half2_rn(lo(a), hi(a));
    __builtin_memcpy(v, &r, 4);
}

template <typename T>
struct Pair16 {  // fp32 has no such pair; the type only has to exist
    using type = __half2;
};
template <>
struct Pair16<__nv_bfloat16> {
    using type = __nv_bfloat162;
};

// A thread's vectors of a row, seen as pairs: two neighbours of a vector, or
// with single elements (VEC = 1) the elements 2p and 2p + 1 of the thread.
template <typename T, int VEC, int ITEMS>
struct RowVectors {
    static constexpr int PAIRS = ITEMS * VEC / 2;
    Vec<T, VEC> v[ITEMS];
    __device__ __forceinline__ F2 pair(int p) const {
        if constexpr (VEC == 1)
            return f2(to_f32(v[2 * p].v[0]), to_f32(v[2 * p + 1].v[0]));
        else
            return pair_of(v[2 * p / VEC].v + 2 * p % VEC);
    }
    // The largest value (NaN only if all are), without unpacking.
    __device__ __forceinline__ float max() const {
        using T2 = typename Pair16<T>::type;
        T2 m;
        __builtin_memcpy(&m, v[0].v, 4);
#pragma unroll
        for (int p = 1; p < PAIRS; ++p) {
            T2 x;
            __builtin_memcpy(&x, v[2 * p / VEC].v + 2 * p % VEC, 4);
            m = __hmax2(m, x);
        }
        return fmaxf(to_f32(m.x), to_f32(m.y));
    }
    __device__ __forceinline__ void set(int p, F2 x) {
        if constexpr (VEC == 1) {
            v[2 * p].v[0] = from_f32<T>(lo(x));
            v[2 * p + 1].v[0] = from_f32<T>(hi(x));
        } else {
            set_pair(v[2 * p / VEC].v + 2 * p % VEC, x);
        }
    }
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

// 4, 8 or 16 bytes from global to shared memory without a register, in groups
// that the thread that started them waits for.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the thread's last N groups have arrived.
template <int N>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A kernel that reads what the one before it in the stream wrote, launched
// while that one still runs: its blocks may start once every block of the first
// has called launch_dependents() or ended, and wait_for_primary() returns when
// the first has ended and its writes are visible.  The first is launched the
// usual way, after all that came before it.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename K, typename A>
cudaError_t launch_after(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const A& args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = s;
    config.attrs = attr;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, args);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

}  // namespace lce
