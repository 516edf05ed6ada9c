// The balance loss's counting and its C entry points (the
// mathematics and the pass over the logits: lce_balance.cuh).
#include "lce_balance.cuh"

namespace lce {
namespace {

// Counts, before the pass over the logits.
__global__ void __launch_bounds__(BAL_THREADS) bal_count_kernel(BalArgs a) {
    extern __shared__ int32_t hist[];
    launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.done = 0;
    const int64_t t0 = blockIdx.x * a.per_count;
    count_tokens(a, blockIdx.y, blockIdx.x, t0, t0 + a.per_count < a.T ? t0 + a.per_count : a.T, hist);
}

lce_status_t bal_pass_any(const BalArgs& a, int dtype, BalMode mode, cudaStream_t s) {
    return dtype == LCE_BF16  ? bal_pass_bf16(a, mode, s)
           : dtype == LCE_F16 ? bal_pass_f16(a, mode, s)
                              : bal_pass_f32(a, mode, s);
}

int64_t bal_parts(int64_t G, int64_t T) {
    const int64_t most = (T + BAL_MIN_TOKENS - 1) / BAL_MIN_TOKENS;
    const int64_t p = BAL_BLOCKS / G > 1 ? BAL_BLOCKS / G : 1;
    return p < most ? p : most;
}

lce_status_t bal_sizes(int64_t G, int64_t T, int64_t E, int64_t k) {
    if (G <= 0 || T <= 0 || E <= 0 || k <= 0) return LCE_ERR_INVALID_ARG;
    if (G > 65535 || T > INT32_MAX || E > LCE_BALANCE_MAX_E || k > E) return LCE_ERR_UNSUPPORTED;
    return LCE_OK;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t bal_ws(int64_t G, int64_t T, int64_t E, BalArgs* a, void* ws) {
    int64_t parts = bal_parts(G, T);
    const bool alone = G == 1 && T <= BAL_ALONE_TOKENS;
    if (alone) parts = 1;
    const int64_t counting = parts < BAL_COUNT_PARTS ? parts : BAL_COUNT_PARTS;
    const size_t c = 1024, n = c + align256(static_cast<size_t>(G * counting * E) * 4);
    const size_t q = n + align256(static_cast<size_t>(G * counting) * 4);
    if (a) {
        uint8_t* w = static_cast<uint8_t*>(ws);
        a->parts = static_cast<int32_t>(parts);
        a->count_parts = static_cast<int32_t>(counting);
        a->per_count = (T + counting - 1) / counting;
        a->inline_count = alone;
        a->hdr = reinterpret_cast<WsHeader*>(w);
        a->done = reinterpret_cast<unsigned*>(w + 256);
        a->part_c = reinterpret_cast<int32_t*>(w + c);
        a->part_n = reinterpret_cast<int32_t*>(w + n);
        a->part_q = reinterpret_cast<float*>(w + q);
    }
    return q + align256(static_cast<size_t>(G * parts) * 4);
}

struct BalIn {
    int64_t G, T, E, k;
    int dtype;
    const void* z;
    int64_t zg, zt;
    const uint8_t* mask;
    int64_t mask_g;
    uint32_t flags;
};

lce_status_t bal_in(const BalIn& in, BalArgs* a) {
    const lce_status_t st = bal_sizes(in.G, in.T, in.E, in.k);
    if (st != LCE_OK) return st;
    if (!dtype_known(in.dtype) || !in.z || !aligned_to(in.z, dtype_bytes(in.dtype))) return LCE_ERR_INVALID_ARG;
    if (in.zt < in.E || in.zg < 0 || in.mask_g < 0 || (in.flags & ~LCE_REDUCTION_SUM)) return LCE_ERR_INVALID_ARG;
    *a = BalArgs{};
    a->z = in.z;
    a->zg = in.zg;
    a->zt = in.zt;
    a->mask = in.mask;
    a->mask_g = in.mask_g;
    a->T = in.T;
    a->G = static_cast<int32_t>(in.G);
    a->E = static_cast<int32_t>(in.E);
    a->k = static_cast<int32_t>(in.k);
    a->groups = (in.flags & LCE_REDUCTION_SUM) ? 1 : in.G;
    return LCE_OK;
}

lce_status_t bal_loss(const BalIn& in, const void* idx, int idx_bytes, bool grad, float grad_scale,
                      const float* d_grad_output, float* loss, float* group_loss, int64_t* counts, int64_t* n_valid,
                      void* dz, void* ws, size_t ws_bytes, cudaStream_t s) {
    BalArgs a;
    const lce_status_t st = bal_in(in, &a);
    if (st != LCE_OK) return st;
    if (idx_bytes != 4 && idx_bytes != 8) return LCE_ERR_INVALID_ARG;
    if (!idx || !aligned_to(idx, idx_bytes) || !loss || !aligned_to(loss, 4) || !aligned_to(group_loss, 4))
        return LCE_ERR_INVALID_ARG;
    if (!counts || !n_valid || !aligned_to(counts, 8) || !aligned_to(n_valid, 8)) return LCE_ERR_INVALID_ARG;
    if (!ws || !aligned_to(ws, 256) || !aligned_to(d_grad_output, 4)) return LCE_ERR_INVALID_ARG;
    if (grad && (!dz || !aligned_to(dz, dtype_bytes(in.dtype)))) return LCE_ERR_INVALID_ARG;
    if (ws_bytes < bal_ws(in.G, in.T, in.E, &a, ws)) return LCE_ERR_WORKSPACE;
    a.idx = idx;
    a.idx64 = idx_bytes == 8;
    a.grad_scale = grad_scale;
    a.d_grad_output = d_grad_output;
    a.dz = dz;
    a.loss = loss;
    a.group_loss = group_loss;
    a.counts_out = counts;
    a.n_out = n_valid;
    if (!a.inline_count)
        LCE_PROFILED(bal_count_kernel<<<dim3(a.count_parts, a.G), BAL_THREADS,
                                        static_cast<size_t>(a.E) * 4 * BAL_WARPS, s>>>(a));
    return bal_pass_any(a, in.dtype, grad ? BAL_FUSED : BAL_FORWARD, s);
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status_t lce_balance_workspace_size(int64_t groups, int64_t T, int64_t E, int64_t k, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = bal_sizes(groups, T, E, k);
    if (st == LCE_OK) *bytes = bal_ws(groups, T, E, nullptr, nullptr);
    return st;
}

lce_status_t lce_balance_forward(int64_t groups, int64_t T, int64_t E, int64_t k, int dtype, const void* logits,
                                 int64_t group_stride, int64_t token_stride, const void* experts, int index_bytes,
                                 const uint8_t* mask, int64_t mask_group_stride, float* loss, float* group_loss,
                                 int64_t* counts, int64_t* n_valid, void* ws, size_t ws_bytes, lce_stream_t stream,
                                 uint32_t flags) {
    const BalIn in{groups, T, E, k, dtype, logits, group_stride, token_stride, mask, mask_group_stride, flags};
    return bal_loss(in, experts, index_bytes, false, 1.f, nullptr, loss, group_loss, counts, n_valid, nullptr, ws,
                    ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

lce_status_t lce_balance_fused(int64_t groups, int64_t T, int64_t E, int64_t k, int dtype, const void* logits,
                               int64_t group_stride, int64_t token_stride, const void* experts, int index_bytes,
                               const uint8_t* mask, int64_t mask_group_stride, float grad_scale,
                               const float* d_grad_output, float* loss, float* group_loss, int64_t* counts,
                               int64_t* n_valid, void* grad_logits, void* ws, size_t ws_bytes, lce_stream_t stream,
                               uint32_t flags) {
    const BalIn in{groups, T, E, k, dtype, logits, group_stride, token_stride, mask, mask_group_stride, flags};
    return bal_loss(in, experts, index_bytes, true, grad_scale, d_grad_output, loss, group_loss, counts, n_valid,
                    grad_logits, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

lce_status_t lce_balance_backward(int64_t groups, int64_t T, int64_t E, int64_t k, int dtype, const void* logits,
                                  int64_t group_stride, int64_t token_stride, const int64_t* counts,
                                  const int64_t* n_valid, const uint8_t* mask, int64_t mask_group_stride,
                                  float grad_scale, const float* d_grad_output, void* grad_logits,
                                  lce_stream_t stream, uint32_t flags) {
    const BalIn in{groups, T, E, k, dtype, logits, group_stride, token_stride, mask, mask_group_stride, flags};
    BalArgs a;
    const lce_status_t st = bal_in(in, &a);
    if (st != LCE_OK) return st;
    if (!counts || !n_valid || !aligned_to(counts, 8) || !aligned_to(n_valid, 8) || !grad_logits ||
        !aligned_to(grad_logits, dtype_bytes(dtype)) || !aligned_to(d_grad_output, 4))
        return LCE_ERR_INVALID_ARG;
    a.parts = static_cast<int32_t>(bal_parts(groups, T));
    a.per_part = (T + a.parts - 1) / a.parts;
    a.counts = counts;
    a.n_valid = n_valid;
    a.grad_scale = grad_scale;
    a.d_grad_output = d_grad_output;
    a.dz = grad_logits;
    return bal_pass_any(a, dtype, BAL_BACKWARD, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
