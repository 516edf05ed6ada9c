// Layer norm's C entry points: the checks of their arguments (the kernels:
// lce_norm.cuh).
#include "lce_norm.cuh"

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
    NormCall c{};
    c.x = x;
    c.ldx = ldx;
    c.w = weight;
    c.b = bias;
    c.w32 = wtype == LCE_F32;
    c.eps = eps;
    c.y = y;
    c.ldy = ldy;
    c.mean_out = mean;
    c.rstd_out = rstd;
    c.rows = rows;
    c.H = static_cast<int32_t>(H);
    c.s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == LCE_BF16 ? norm_forward_bf16(c) : dtype == LCE_F16 ? norm_forward_f16(c) : norm_forward_f32(c);
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
    NormCall c{};
    c.x = x;
    c.ldx = ldx;
    c.dy = grad_y;
    c.ldd = ldg;
    c.w = weight;
    c.w32 = wtype == LCE_F32;
    c.y = grad_x;
    c.ldy = grad_x ? ldgx : ldx;
    c.mean = mean;
    c.rstd = rstd;
    c.dw = grad_weight;
    c.db = grad_bias;
    c.parts = static_cast<float*>(ws);
    c.rows = rows;
    c.H = static_cast<int32_t>(H);
    c.s = s;
    return dtype == LCE_BF16 ? norm_backward_bf16(c) : dtype == LCE_F16 ? norm_backward_f16(c) : norm_backward_f32(c);
}
