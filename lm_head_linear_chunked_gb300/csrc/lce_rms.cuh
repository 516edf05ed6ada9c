// RMS norm with the residual's addition, forward (in the rows' type or in 8
// bits with scales) and backward.
//
//   s = x + r, rounded to the rows' type;  rstd = 1 / sqrt(sum_h s^2 / H + eps)
//   y = s rstd w
//   8 bits: a = max |y| of a group of columns, scale = max(a, 2^-100) / 448,
//     q = e4m3(y / scale)
//   xh = s rstd,  g = dy w,  dx = rstd (g - xh mean_h(g xh)) + ds
//   dw = sum_r dy xh
//
// The sum is rounded before it is normed: the rounded one is what the next
// block adds to and what the backward reads, so all three see the same s.
// All sums are FP32.
#pragma once

#include "lce_internal.cuh"
#include "lce_rows.cuh"

namespace lce {

constexpr float E4M3_MAX = 448.f;
constexpr float RMS_LEAST_AMAX = 0x1p-100f;  // keeps 1 / scale finite where a group is zero

// What a launch needs, by the element type (one translation unit each).
struct RmsCall {
    const void *x, *r, *w, *dy, *ds;
    int64_t ldx, ldr, ldd, ldds, lds, ldy;
    bool w32;
    float eps;
    void *sum, *y;       // y: the output, or dx
    uint8_t* q;
    int64_t ldq;
    float* scales;
    int32_t group;       // columns to a scale (H: one for the row)
    float* rstd_out;
    const float* rstd;
    void* dw;
    float* parts;        // [NORM_PARTS, H]
    int64_t rows;
    int32_t H;
    cudaStream_t s;
};
lce_status_t rms_forward_bf16(const RmsCall& c);
lce_status_t rms_forward_f16(const RmsCall& c);
lce_status_t rms_forward_f32(const RmsCall& c);
lce_status_t rms_backward_bf16(const RmsCall& c);
lce_status_t rms_backward_f16(const RmsCall& c);
lce_status_t rms_backward_f32(const RmsCall& c);

namespace {

// The larger of two, NaN if one is: a row that holds one shows it in its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Two values as e4m3, rounded to nearest even, the first in the low byte.
__device__ __forceinline__ uint16_t to_e4m3x2(float first, float second) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(second), "f"(first));
    return r;
}

__device__ __forceinline__ float group_scale(float amax) { return max_nan(amax, RMS_LEAST_AMAX) / E4M3_MAX; }

template <typename T>
struct RmsFwd {
    const T *x, *r;  // r nullable
    int64_t ldx, ldr;
    const void* w;   // nullable; fp32 with w32, else T
    bool w32;
    float eps;
    T* sum;          // written where r is given
    int64_t lds;
    T* y;            // or q and scales
    int64_t ldy;
    uint8_t* q;
    int64_t ldq;
    float* scales;   // [rows, groups]
    int32_t group, groups;
    float* rstd;     // nullable
    int64_t rows;
    int32_t H;
};

// A block per row, any width: the row is read again for the output (and, in 8
// bits, for the largest magnitude), from L1 or L2.
template <typename T, bool QUANT>
__global__ void __launch_bounds__(512) rms_fwd_any(RmsFwd<T> a) {
    __shared__ float part[2][32];
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        float v = to_f32(x[i]);
        if (a.r) {
            const T t = from_f32<T>(v + to_f32(a.r[r * a.ldr + i]));
            a.sum[r * a.lds + i] = t;
            v = to_f32(t);
        }
        s = fmaf(v, v, s);
    }
    const float rstd = rsqrtf(block_sum(s, part[0]) / static_cast<float>(a.H) + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    if (a.r) x = a.sum + r * a.lds;
    auto normed = [&](int i) { return to_f32(x[i]) * rstd * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f); };
    if constexpr (!QUANT) {
        for (int i = threadIdx.x; i < a.H; i += blockDim.x) a.y[r * a.ldy + i] = from_f32<T>(normed(i));
    } else if (a.groups == 1) {
        float m = 0.f;
        for (int i = threadIdx.x; i < a.H; i += blockDim.x) m = max_nan(m, fabsf(normed(i)));
        m = warp_max_nan(m);
        if ((threadIdx.x & 31) == 0) part[1][threadIdx.x >> 5] = m;
        __syncthreads();
        m = warp_max_nan((threadIdx.x & 31) < (blockDim.x >> 5) ? part[1][threadIdx.x & 31] : 0.f);
        const float scale = group_scale(m), inv = 1.f / scale;
        if (threadIdx.x == 0) a.scales[r] = scale;
        for (int i = threadIdx.x; i < a.H; i += blockDim.x)
            a.q[r * a.ldq + i] = static_cast<uint8_t>(to_e4m3x2(normed(i) * inv, 0.f));
    } else {
        for (int g = threadIdx.x >> 5; g < a.groups; g += blockDim.x >> 5) {
            const int first = g * a.group + (threadIdx.x & 31);
            const int end = a.H - g * a.group < a.group ? a.H : (g + 1) * a.group;
            float m = 0.f;
            for (int i = first; i < end; i += 32) m = max_nan(m, fabsf(normed(i)));
            m = warp_max_nan(m);
            const float scale = group_scale(m), inv = 1.f / scale;
            if ((threadIdx.x & 31) == 0) a.scales[r * a.groups + g] = scale;
            for (int i = first; i < end; i += 32)
                a.q[r * a.ldq + i] = static_cast<uint8_t>(to_e4m3x2(normed(i) * inv, 0.f));
        }
    }
}

template <typename T>
struct RmsBwd {
    const T *dy, *x, *ds;  // ds nullable
    int64_t ldd, ldx, ldds;
    const void* w;
    bool w32;
    const float* rstd;
    T* dx;                 // nullable
    int64_t lddx;
    float* part_w;         // [parts, H], nullable
    int64_t rows, rows_per_part;
    int32_t H;
};

// dx of a block's row, any width.
template <typename T>
__global__ void __launch_bounds__(512) rms_dx_any(RmsBwd<T> a) {
    __shared__ float part[32];
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    const T* dy = a.dy + r * a.ldd;
    const float rstd = a.rstd[r];
    float q = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x)
        q += to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f) * (to_f32(x[i]) * rstd);
    q = block_sum(q, part) / static_cast<float>(a.H);
    T* dx = a.dx + r * a.lddx;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f);
        float v = rstd * (g - to_f32(x[i]) * rstd * q);
        if (a.ds) v += to_f32(a.ds[r * a.ldds + i]);
        dx[i] = from_f32<T>(v);
    }
}

// Column sums of a block of rows: 32 columns per block, 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) rms_dw_any(RmsBwd<T> a) {
    __shared__ float sw[8][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    const int64_t r0 = blockIdx.y * a.rows_per_part;
    const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
    float w = 0.f;
    if (col < a.H)
        for (int64_t r = r0 + k; r < r1; r += 8)
            w += to_f32(a.dy[r * a.ldd + col]) * (to_f32(a.x[r * a.ldx + col]) * a.rstd[r]);
    sw[k][c] = w;
    __syncthreads();
    if (k == 0 && col < a.H) {
#pragma unroll
        for (int j = 1; j < 8; ++j) w += sw[j][c];
        a.part_w[static_cast<int64_t>(blockIdx.y) * a.H + col] = w;
    }
}

template <typename T, typename W>
lce_status_t rms_forward(const RmsCall& c) {
    const RmsFwd<T> a{static_cast<const T*>(c.x), static_cast<const T*>(c.r), c.ldx, c.ldr, c.w, c.w32, c.eps,
                      static_cast<T*>(c.sum), c.lds, static_cast<T*>(c.y), c.ldy, c.q, c.ldq, c.scales, c.group,
                      (c.H + c.group - 1) / c.group, c.rstd_out, c.rows, c.H};
    cudaStream_t s = c.s;
    const unsigned blocks = static_cast<unsigned>(c.rows);
    if (c.q)
        LCE_PROFILED(rms_fwd_any<T, true><<<blocks, 512, 0, s>>>(a));
    else
        LCE_PROFILED(rms_fwd_any<T, false><<<blocks, 512, 0, s>>>(a));
    return LCE_OK;
}

template <typename T, typename W>
lce_status_t rms_backward(const RmsCall& c) {
    RmsBwd<T> a{static_cast<const T*>(c.dy), static_cast<const T*>(c.x), static_cast<const T*>(c.ds), c.ldd, c.ldx, c.ldds,
                c.w, c.w32, c.rstd, static_cast<T*>(c.y), c.ldy, c.parts, c.rows, 0, c.H};
    cudaStream_t s = c.s;
    if (c.y) LCE_PROFILED(rms_dx_any<T><<<static_cast<unsigned>(c.rows), 512, 0, s>>>(a));
    if (!c.dw) return LCE_OK;
    a.rows_per_part = (c.rows + NORM_PARTS - 1) / NORM_PARTS;
    if (a.rows_per_part < 32) a.rows_per_part = 32;
    const int parts = static_cast<int>((c.rows + a.rows_per_part - 1) / a.rows_per_part);
    LCE_PROFILED(rms_dw_any<T><<<dim3((c.H + 31) / 32, parts), 256, 0, s>>>(a));
    LCE_PROFILED(launch_after(norm_dw_join<W>, dim3((c.H + 31) / 32), 1024, 0, s,
                              JoinArgs{a.part_w, nullptr, parts, c.H, c.dw, nullptr}));
    return LCE_OK;
}

}  // namespace
}  // namespace lce
