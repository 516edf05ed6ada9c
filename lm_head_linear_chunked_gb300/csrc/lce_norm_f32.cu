// Layer norm of f32 rows (the kernels and their choice: lce_norm.cuh).
#include "lce_norm.cuh"

namespace lce {
lce_status_t norm_forward_f32(const NormCall& c) { return norm_forward<float, float>(c); }
lce_status_t norm_backward_f32(const NormCall& c) { return norm_backward<float, float>(c); }
}  // namespace lce
