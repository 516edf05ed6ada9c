// RMS norm of bf16 rows (the kernels and their choice: lce_rms.cuh).
#include "lce_rms.cuh"

namespace lce {
lce_status_t rms_forward_bf16(const RmsCall& c) {
    return c.w32 ? rms_forward<__nv_bfloat16, float>(c) : rms_forward<__nv_bfloat16, __nv_bfloat16>(c);
}
lce_status_t rms_backward_bf16(const RmsCall& c) {
    return c.w32 ? rms_backward<__nv_bfloat16, float>(c) : rms_backward<__nv_bfloat16, __nv_bfloat16>(c);
}
}  // namespace lce
