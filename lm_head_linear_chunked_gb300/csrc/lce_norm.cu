// Layer norm of the rows that the head reads, forward and backward.
//
//   mean = sum_h x / H,  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - mean_h(g) - xh mean_h(g xh))
//   dw = sum_r dy xh,  db = sum_r dy
//
// All sums are FP32; the variance is summed from the centred values, so an
// offset of the row costs no digits.
#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {
namespace {

// One value for the whole block: the sum of v over its threads, added in a
// fixed order.  `part` holds 32 floats and may be reused after the next
// barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5, l = threadIdx.x & 31;
    return warp_sum(l < warps ? part[l] : 0.f);
}

template <typename T>
struct NormFwd {
    const T* x;
    int64_t ldx;
    const void *w, *b;  // each nullable; fp32 with w32, else T
    bool w32;
    float eps;
    T* y;
    int64_t ldy;
    float *mean, *rstd;  // nullable
    int64_t rows;
    int32_t H;
};

template <typename T>
__device__ __forceinline__ float load_w(const void* w, bool w32, int64_t i) {
    return w32 ? static_cast<const float*>(w)[i] : to_f32(static_cast<const T*>(w)[i]);
}

// A block per row, any width: the row is read three times (mean, variance,
// output), the later times from L1 or L2.
template <typename T>
__global__ void __launch_bounds__(512) norm_fwd_any(NormFwd<T> a) {
    __shared__ float part[2][32];
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) s += to_f32(x[i]);
    const float mean = block_sum(s, part[0]) / static_cast<float>(a.H);
    float q = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float d = to_f32(x[i]) - mean;
        q += d * d;
    }
    const float rstd = 1.f / sqrtf(block_sum(q, part[1]) / static_cast<float>(a.H) + a.eps);
    T* y = a.y + r * a.ldy;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        float v = (to_f32(x[i]) - mean) * rstd;
        if (a.w) v *= load_w<T>(a.w, a.w32, i);
        if (a.b) v += load_w<T>(a.b, a.w32, i);
        y[i] = from_f32<T>(v);
    }
    if (threadIdx.x == 0 && a.mean) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
    }
}

template <typename T>
struct NormBwd {
    const T *dy, *x;
    int64_t ldd, ldx;
    const void* w;
    bool w32;
    const float *mean, *rstd;
    T* dx;  // nullable
    int64_t lddx;
    float* part_w;  // [parts, H], nullable
    float* part_b;
    int64_t rows, rows_per_part;
    int32_t H;
};

// dx of a block's row, any width.
template <typename T>
__global__ void __launch_bounds__(512) norm_dx_any(NormBwd<T> a) {
    __shared__ float part[2][32];
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    const T* dy = a.dy + r * a.ldd;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s = 0.f, q = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f);
        s += g;
        q += g * (to_f32(x[i]) - mean) * rstd;
    }
    s = block_sum(s, part[0]) / static_cast<float>(a.H);
    q = block_sum(q, part[1]) / static_cast<float>(a.H);
    T* dx = a.dx + r * a.lddx;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f);
        dx[i] = from_f32<T>(rstd * (g - s - (to_f32(x[i]) - mean) * rstd * q));
    }
}

// Column sums of a block of rows: 32 columns per block, 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_any(NormBwd<T> a) {
    __shared__ float sw[8][33], sb[8][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    const int64_t r0 = blockIdx.y * a.rows_per_part;
    const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
    float w = 0.f, b = 0.f;
    if (col < a.H)
        for (int64_t r = r0 + k; r < r1; r += 8) {
            const float d = to_f32(a.dy[r * a.ldd + col]);
            w += d * (to_f32(a.x[r * a.ldx + col]) - a.mean[r]) * a.rstd[r];
            b += d;
        }
    sw[k][c] = w;
    sb[k][c] = b;
    __syncthreads();
    if (k == 0 && col < a.H) {
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            w += sw[j][c];
            b += sb[j][c];
        }
        if (a.part_w) a.part_w[static_cast<int64_t>(blockIdx.y) * a.H + col] = w;
        if (a.part_b) a.part_b[static_cast<int64_t>(blockIdx.y) * a.H + col] = b;
    }
}

// Adds the parts' column sums in a fixed order: 32 columns per block, 8
// threads a column.
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_join(const float* part_w, const float* part_b, int parts, int32_t H,
                                                    bool w32, void* dw, void* db) {
    __shared__ float s[8][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    const float* p = blockIdx.y ? part_b : part_w;
    void* out = blockIdx.y ? db : dw;
    if (!out) return;
    float v = 0.f;
    if (col < H)
        for (int j = k; j < parts; j += 8) v += p[static_cast<int64_t>(j) * H + col];
    s[k][c] = v;
    __syncthreads();
    if (k == 0 && col < H) {
#pragma unroll
        for (int j = 1; j < 8; ++j) v += s[j][c];
        if (w32)
            static_cast<float*>(out)[col] = v;
        else
            static_cast<T*>(out)[col] = from_f32<T>(v);
    }
}

// Parts of the weight gradient's row sum.
constexpr int64_t NORM_PARTS = 608;

}  // namespace
}  // namespace lce

using namespace lce;

namespace {

lce_status_t norm_args(int64_t rows, int64_t H, int dtype, int wtype) {
    if (rows < 0 || H <= 0 || !dtype_known(dtype) || !dtype_known(wtype)) return LCE_ERR_INVALID_ARG;
    if (wtype != dtype && wtype != LCE_F32) return LCE_ERR_UNSUPPORTED;
    if (rows > INT32_MAX || H > LCE_NORM_MAX_H) return LCE_ERR_UNSUPPORTED;
    return LCE_OK;
}

bool norm_ptr(const void* p, size_t bytes, bool needed) { return p ? aligned_to(p, bytes) : !needed; }

}  // namespace

extern "C" lce_status_t lce_layer_norm_forward(int64_t rows, int64_t H, int dtype, int wtype, const void* x,
                                               int64_t ldx, const void* weight, const void* bias, float eps, void* y,
                                               int64_t ldy, float* mean, float* rstd, lce_stream_t stream) {
    const lce_status_t st = norm_args(rows, H, dtype, wtype);
    if (st != LCE_OK) return st;
    const size_t es = dtype_bytes(dtype), ws = dtype_bytes(wtype);
    if (!(eps >= 0.f) || ldx < H || ldy < H || (mean != nullptr) != (rstd != nullptr)) return LCE_ERR_INVALID_ARG;
    if (!norm_ptr(weight, ws, false) || !norm_ptr(bias, ws, false) || !norm_ptr(mean, 4, false) ||
        !norm_ptr(rstd, 4, false))
        return LCE_ERR_INVALID_ARG;
    if (rows == 0) return LCE_OK;
    if (!norm_ptr(x, es, true) || !norm_ptr(y, es, true)) return LCE_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        NormFwd<T> a{static_cast<const T*>(x), ldx, weight, bias, wtype == LCE_F32, eps, static_cast<T*>(y), ldy,
                     mean, rstd, rows, static_cast<int32_t>(H)};
        LCE_PROFILED(norm_fwd_any<T><<<static_cast<unsigned>(rows), 256, 0, s>>>(a));
        return LCE_OK;
    });
}

extern "C" lce_status_t lce_layer_norm_workspace_size(int64_t rows, int64_t H, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = norm_args(rows, H, LCE_F32, LCE_F32);
    if (st != LCE_OK) return st;
    const int64_t parts = rows < 1 ? 1 : (rows < NORM_PARTS ? rows : NORM_PARTS);
    *bytes = static_cast<size_t>(parts) * H * 2 * 4;
    return LCE_OK;
}

extern "C" lce_status_t lce_layer_norm_backward(int64_t rows, int64_t H, int dtype, int wtype, const void* grad_y,
                                                int64_t ldg, const void* x, int64_t ldx, const void* weight,
                                                const float* mean, const float* rstd, void* grad_x, int64_t ldgx,
                                                void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes,
                                                lce_stream_t stream) {
    size_t need = 0;
    lce_status_t st = norm_args(rows, H, dtype, wtype);
    if (st != LCE_OK) return st;
    st = lce_layer_norm_workspace_size(rows, H, &need);
    if (st != LCE_OK) return st;
    const size_t es = dtype_bytes(dtype), wb = dtype_bytes(wtype);
    if (ldg < H || ldx < H || (grad_x && ldgx < H)) return LCE_ERR_INVALID_ARG;
    if (!norm_ptr(weight, wb, false) || !norm_ptr(grad_weight, wb, false) || !norm_ptr(grad_bias, wb, false) ||
        !norm_ptr(grad_x, es, false))
        return LCE_ERR_INVALID_ARG;
    const bool sums = grad_weight || grad_bias;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {  // no rows: the sums over them are zero
        if (grad_weight && cudaMemsetAsync(grad_weight, 0, H * wb, s) != cudaSuccess) return LCE_ERR_CUDA;
        if (grad_bias && cudaMemsetAsync(grad_bias, 0, H * wb, s) != cudaSuccess) return LCE_ERR_CUDA;
        return LCE_OK;
    }
    if (!norm_ptr(grad_y, es, true) || !norm_ptr(x, es, true) || !norm_ptr(mean, 4, true) || !norm_ptr(rstd, 4, true))
        return LCE_ERR_INVALID_ARG;
    if (sums && (!ws || !aligned_to(ws, 256))) return LCE_ERR_INVALID_ARG;
    if (sums && ws_bytes < need) return LCE_ERR_WORKSPACE;
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        NormBwd<T> a{static_cast<const T*>(grad_y), static_cast<const T*>(x), ldg, ldx, weight, wtype == LCE_F32,
                     mean, rstd, static_cast<T*>(grad_x), ldgx, nullptr, nullptr, rows, 0, static_cast<int32_t>(H)};
        if (grad_x) LCE_PROFILED(norm_dx_any<T><<<static_cast<unsigned>(rows), 256, 0, s>>>(a));
        if (sums) {
            const int64_t parts_max = static_cast<int64_t>(need / (static_cast<size_t>(H) * 8));
            a.rows_per_part = (rows + parts_max - 1) / parts_max;
            if (a.rows_per_part < 32) a.rows_per_part = 32;
            const int parts = static_cast<int>((rows + a.rows_per_part - 1) / a.rows_per_part);
            a.part_w = static_cast<float*>(ws);
            a.part_b = a.part_w + static_cast<int64_t>(parts) * H;
            const unsigned tiles = static_cast<unsigned>((H + 31) / 32);
            LCE_PROFILED(norm_dw_any<T><<<dim3(tiles, parts), 256, 0, s>>>(a));
            LCE_PROFILED(norm_dw_join<T><<<dim3(tiles, 2), 256, 0, s>>>(a.part_w, a.part_b, parts, a.H, a.w32,
                                                                         grad_weight, grad_bias));
        }
        return LCE_OK;
    });
}
