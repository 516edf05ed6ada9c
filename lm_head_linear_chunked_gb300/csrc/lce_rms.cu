// RMS norm's C entry points: the checks of their arguments (the kernels:
// lce_rms.cuh).
#include "lce_rms.cuh"

using namespace lce;

namespace {

lce_status_t rms_args(int64_t rows, int64_t H, int dtype, int wtype) {
    if (rows < 0 || H <= 0 || !dtype_known(dtype) || !dtype_known(wtype)) return LCE_ERR_INVALID_ARG;
    if (wtype != dtype && wtype != LCE_F32) return LCE_ERR_UNSUPPORTED;
    if (rows > INT32_MAX || H > LCE_NORM_MAX_H) return LCE_ERR_UNSUPPORTED;
    return LCE_OK;
}

bool at(const void* p, size_t bytes, bool needed) { return p ? aligned_to(p, bytes) : !needed; }

// The inputs of the two forward calls.
lce_status_t rms_in(int64_t rows, int64_t H, int dtype, int wtype, const void* x, int64_t ldx, const void* residual,
                    int64_t ldr, const void* weight, float eps, void* sum, int64_t lds, lce_stream_t stream, RmsCall* c) {
    const lce_status_t st = rms_args(rows, H, dtype, wtype);
    if (st != LCE_OK) return st;
    const size_t es = dtype_bytes(dtype);
    if (!(eps >= 0.f) || ldx < H || (residual && ldr < H) || (sum && lds < H)) return LCE_ERR_INVALID_ARG;
    if (!at(weight, dtype_bytes(wtype), false) || (rows && !at(x, es, true))) return LCE_ERR_INVALID_ARG;
    if (rows && ((residual != nullptr) != (sum != nullptr) || !at(residual, es, false) || !at(sum, es, false)))
        return LCE_ERR_INVALID_ARG;
    *c = RmsCall{};
    c->x = x;
    c->ldx = ldx;
    c->r = residual;
    c->ldr = residual ? ldr : ldx;
    c->w = weight;
    c->w32 = wtype == LCE_F32;
    c->eps = eps;
    c->sum = sum;
    c->lds = sum ? lds : ldx;
    c->rows = rows;
    c->H = static_cast<int32_t>(H);
    c->group = c->H;
    c->s = reinterpret_cast<cudaStream_t>(stream);
    return LCE_OK;
}

lce_status_t rms_forward_any(const RmsCall& c, int dtype) {
    if (c.rows == 0) return LCE_OK;
    return dtype == LCE_BF16 ? rms_forward_bf16(c) : dtype == LCE_F16 ? rms_forward_f16(c) : rms_forward_f32(c);
}

}  // namespace

extern "C" lce_status_t lce_rms_norm_forward(int64_t rows, int64_t H, int dtype, int wtype, const void* x, int64_t ldx,
                                             const void* residual, int64_t ldr, const void* weight, float eps,
                                             void* sum, int64_t lds, void* y, int64_t ldy, float* rstd,
                                             lce_stream_t stream) {
    RmsCall c;
    const lce_status_t st = rms_in(rows, H, dtype, wtype, x, ldx, residual, ldr, weight, eps, sum, lds, stream, &c);
    if (st != LCE_OK) return st;
    if (ldy < H || !at(y, dtype_bytes(dtype), rows > 0) || !at(rstd, 4, false)) return LCE_ERR_INVALID_ARG;
    c.y = y;
    c.ldy = ldy;
    c.rstd_out = rstd;
    return rms_forward_any(c, dtype);
}

extern "C" lce_status_t lce_rms_norm_fp8(int64_t rows, int64_t H, int dtype, int wtype, const void* x, int64_t ldx,
                                         const void* residual, int64_t ldr, const void* weight, float eps, void* sum,
                                         int64_t lds, uint8_t* q, int64_t ldq, float* scales, int64_t group,
                                         lce_stream_t stream) {
    RmsCall c;
    const lce_status_t st = rms_in(rows, H, dtype, wtype, x, ldx, residual, ldr, weight, eps, sum, lds, stream, &c);
    if (st != LCE_OK) return st;
    if (group < 0 || ldq < H || (rows && !q) || !at(scales, 4, rows > 0)) return LCE_ERR_INVALID_ARG;
    if (group != 0 && group != LCE_FP8_GROUP) return LCE_ERR_UNSUPPORTED;
    c.q = q;
    c.ldq = ldq;
    c.scales = scales;
    if (group && group < H) c.group = static_cast<int32_t>(group);
    return rms_forward_any(c, dtype);
}

extern "C" lce_status_t lce_rms_norm_workspace_size(int64_t rows, int64_t H, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = rms_args(rows, H, LCE_F32, LCE_F32);
    if (st != LCE_OK) return st;
    const int64_t parts = rows < 1 ? 1 : (rows < NORM_PARTS ? rows : NORM_PARTS);
    *bytes = static_cast<size_t>(parts) * H * 4;
    return LCE_OK;
}

extern "C" lce_status_t lce_rms_norm_backward(int64_t rows, int64_t H, int dtype, int wtype, const void* grad_y,
                                              int64_t ldg, const void* x, int64_t ldx, const void* weight,
                                              const float* rstd, const void* grad_sum, int64_t ldgs, void* grad_x,
                                              int64_t ldgx, void* grad_weight, void* ws, size_t ws_bytes,
                                              lce_stream_t stream) {
    size_t need = 0;
    lce_status_t st = rms_args(rows, H, dtype, wtype);
    if (st != LCE_OK) return st;
    st = lce_rms_norm_workspace_size(rows, H, &need);
    if (st != LCE_OK) return st;
    const size_t es = dtype_bytes(dtype), wb = dtype_bytes(wtype);
    if (ldg < H || ldx < H || (grad_x && ldgx < H) || (grad_sum && ldgs < H)) return LCE_ERR_INVALID_ARG;
    if (!at(weight, wb, false) || !at(grad_weight, wb, false) || !at(grad_x, es, false) || !at(grad_sum, es, false))
        return LCE_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {  // no rows: the sum over them is zero
        if (grad_weight && cudaMemsetAsync(grad_weight, 0, H * wb, s) != cudaSuccess) return LCE_ERR_CUDA;
        return LCE_OK;
    }
    if (!at(grad_y, es, true) || !at(x, es, true) || !at(rstd, 4, true)) return LCE_ERR_INVALID_ARG;
    if (grad_weight && (!ws || !aligned_to(ws, 256))) return LCE_ERR_INVALID_ARG;
    if (grad_weight && ws_bytes < need) return LCE_ERR_WORKSPACE;
    RmsCall c{};
    c.x = x;
    c.ldx = ldx;
    c.dy = grad_y;
    c.ldd = ldg;
    c.ds = grad_sum;
    c.ldds = grad_sum ? ldgs : ldx;
    c.w = weight;
    c.w32 = wtype == LCE_F32;
    c.y = grad_x;
    c.ldy = grad_x ? ldgx : ldx;
    c.rstd = rstd;
    c.dw = grad_weight;
    c.parts = grad_weight ? static_cast<float*>(ws) : nullptr;
    c.rows = rows;
    c.H = static_cast<int32_t>(H);
    c.s = s;
    return dtype == LCE_BF16 ? rms_backward_bf16(c) : dtype == LCE_F16 ? rms_backward_f16(c) : rms_backward_f32(c);
}
