// RMS norm of f32 rows (the kernels and their choice: lce_rms.cuh).
#include "lce_rms.cuh"

namespace lce {
lce_status_t rms_forward_f32(const RmsCall& c) { return rms_forward<float, float>(c); }
lce_status_t rms_backward_f32(const RmsCall& c) { return rms_backward<float, float>(c); }
}  // namespace lce
