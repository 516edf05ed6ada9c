// Layer norm of f16 rows (the kernels and their choice: lce_norm.cuh).
#include "lce_norm.cuh"

namespace lce {
lce_status_t norm_forward_f16(const NormCall& c) {
    return c.w32 ? norm_forward<__half, float>(c) : norm_forward<__half, __half>(c);
}
lce_status_t norm_backward_f16(const NormCall& c) {
    return c.w32 ? norm_backward<__half, float>(c) : norm_backward<__half, __half>(c);
}
}  // namespace lce
