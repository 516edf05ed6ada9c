// Layer norm of bf16 rows (the kernels and their choice: lce_norm.cuh).
#include "lce_norm.cuh"

namespace lce {
lce_status_t norm_forward_bf16(const NormCall& c) {
    return c.w32 ? norm_forward<__nv_bfloat16, float>(c) : norm_forward<__nv_bfloat16, __nv_bfloat16>(c);
}
lce_status_t norm_backward_bf16(const NormCall& c) {
    return c.w32 ? norm_backward<__nv_bfloat16, float>(c) : norm_backward<__nv_bfloat16, __nv_bfloat16>(c);
}
}  // namespace lce
