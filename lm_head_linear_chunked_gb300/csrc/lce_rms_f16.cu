// RMS norm of f16 rows (the kernels and their choice: lce_rms.cuh).
#include "lce_rms.cuh"

namespace lce {
lce_status_t rms_forward_f16(const RmsCall& c) {
    return c.w32 ? rms_forward<__half, float>(c) : rms_forward<__half, __half>(c);
}
lce_status_t rms_backward_f16(const RmsCall& c) {
    return c.w32 ? rms_backward<__half, float>(c) : rms_backward<__half, __half>(c);
}
}  // namespace lce
