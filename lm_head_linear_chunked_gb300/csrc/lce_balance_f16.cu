// The balance loss's pass over f16 logits (the kernel: lce_balance.cuh).
#include "lce_balance.cuh"

namespace lce {
lce_status_t bal_pass_f16(const BalArgs& a, BalMode mode, cudaStream_t s) { return bal_pass<__half>(a, mode, s); }
}  // namespace lce
