// The balance loss's pass over bf16 logits (the kernel: lce_balance.cuh).
#include "lce_balance.cuh"

namespace lce {
lce_status_t bal_pass_bf16(const BalArgs& a, BalMode mode, cudaStream_t s) { return bal_pass<__nv_bfloat16>(a, mode, s); }
}  // namespace lce
