// The balance loss's counting and finish, and its C entry points (the
// mathematics and the pass over the logits: lce_balance.cuh).
#include "lce_balance.cuh"

namespace lce {
namespace {

// Counts by themselves, before the fused call's pass.
__global__ void __launch_bounds__(BAL_THREADS) bal_count_kernel(BalArgs a) {
    extern __shared__ int32_t hist[];
    open_finish(a);
    const int64_t t0 = blockIdx.x * a.per_count;
    count_tokens(a, blockIdx.y, blockIdx.x, t0, t0 + a.per_count < a.T ? t0 + a.per_count : a.T, hist);
}

// Adds the parts up.  A block takes 32 experts of a group, a row of 32 threads
// each 1/32 of the parts; the last block to end adds the blocks' shares of the
// loss, in order.  The sums are FP32 (at most 24 terms in sequence; this GPU's
// FP64 adds run at 1/64 of their rate, and took 8 of 11 us here) and only the
// last few scalars FP64.
__global__ void __launch_bounds__(1024) bal_finish_kernel(BalArgs a) {
    __shared__ float sp[32][33];
    __shared__ long long sc[32][33];
    __shared__ int32_t sn[32];
    __shared__ int bad;
    __shared__ bool last;
    const int g = blockIdx.y, lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    float p = 0.f;
    long long c = 0;
    int32_t n = 0;
    if (e < a.E) {
#pragma unroll 4
        for (int q = row; q < a.parts; q += 32) p += a.part_p[(static_cast<int64_t>(g) * a.parts + q) * a.E + e];
#pragma unroll 4
        for (int q = row; q < a.count_parts; q += 32) c += a.part_c[(static_cast<int64_t>(g) * a.count_parts + q) * a.E + e];
    }
    sp[row][lane] = p;
    sc[row][lane] = c;
    for (int q = threadIdx.x; q < a.count_parts; q += 1024) {
        const int32_t m = a.part_n[static_cast<int64_t>(g) * a.count_parts + q];
        n += m < 0 ? -1 - m : m;
        if (m < 0) bad = 1;
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) sn[row] = n;
    __syncthreads();
    p = warp_sum(sp[lane][row]);  // expert `row` of the block
    c = sc[lane][row];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
    __syncthreads();
    if (lane == 0) {
        const int at = blockIdx.x * 32 + row;
        if (at < a.E) a.counts_out[static_cast<int64_t>(g) * a.E + at] = c;
        sp[0][row] = at < a.E ? static_cast<float>(c) * p : 0.f;
    }
    __syncthreads();
    if (row == 0) {
        const float v = warp_sum(sp[0][lane]);
        n = __reduce_add_sync(0xFFFFFFFFu, sn[lane]);
        if (lane == 0) {
            a.part_l[static_cast<int64_t>(g) * gridDim.x + blockIdx.x] =
                n > 0 ? static_cast<double>(v) * a.E / (static_cast<double>(a.k) * n * n) : 0.0;
            if (blockIdx.x == 0) a.n_out[g] = n;
            if (bad) atomicOr(&a.hdr->status, STATUS_INDEX);
            __threadfence();
            last = atomicAdd(a.done, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!last || row != 0) return;
    __threadfence();
    double total = 0.0;
    for (int k = lane; k < a.G; k += 32) {
        double v = 0.0;
        for (unsigned i = 0; i < gridDim.x; ++i) v += __ldcg(a.part_l + static_cast<int64_t>(k) * gridDim.x + i);
        if (a.group_loss) a.group_loss[k] = static_cast<float>(v);
        total += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    const bool wrong = (__ldcg(&a.hdr->status) & STATUS_INDEX) != 0;
    if (lane == 0) *a.loss = wrong ? __int_as_float(0x7FC00000) : static_cast<float>(total / a.groups);
}

lce_status_t bal_pass_any(BalArgs& a, int dtype, BalMode mode, cudaStream_t s) {
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

size_t bal_ws(int64_t G, int64_t T, int64_t E, bool fused, BalArgs* a, void* ws) {
    const int64_t parts = bal_parts(G, T);
    const int64_t counting = fused && parts > BAL_COUNT_PARTS ? BAL_COUNT_PARTS : parts;
    const size_t c = 1024, n = c + align256(static_cast<size_t>(G * parts * E) * 4);
    const size_t p = n + align256(static_cast<size_t>(G * parts) * 4);
    const size_t l = p + align256(static_cast<size_t>(G * parts * E) * 4);
    if (a) {
        uint8_t* w = static_cast<uint8_t*>(ws);
        a->parts = static_cast<int32_t>(parts);
        a->per_part = (T + parts - 1) / parts;
        a->count_parts = static_cast<int32_t>(counting);
        a->per_count = (T + counting - 1) / counting;
        a->hdr = reinterpret_cast<WsHeader*>(w);
        a->done = reinterpret_cast<unsigned*>(w + 256);
        a->part_c = reinterpret_cast<int32_t*>(w + c);
        a->part_n = reinterpret_cast<int32_t*>(w + n);
        a->part_p = reinterpret_cast<float*>(w + p);
        a->part_l = reinterpret_cast<double*>(w + l);
    }
    return l + align256(static_cast<size_t>(G * ((E + 31) / 32)) * 8);
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
    if (ws_bytes < bal_ws(in.G, in.T, in.E, grad, &a, ws)) return LCE_ERR_WORKSPACE;
    a.idx = idx;
    a.idx64 = idx_bytes == 8;
    a.grad_scale = grad_scale;
    a.d_grad_output = d_grad_output;
    a.dz = dz;
    a.loss = loss;
    a.group_loss = group_loss;
    a.counts_out = counts;
    a.n_out = n_valid;
    if (grad)
        LCE_PROFILED(bal_count_kernel<<<dim3(a.count_parts, a.G), BAL_THREADS,
                                        static_cast<size_t>(a.E) * 4 * BAL_WARPS, s>>>(a));
    const lce_status_t pt = bal_pass_any(a, in.dtype, grad ? BAL_FUSED : BAL_FORWARD, s);
    if (pt != LCE_OK) return pt;
    LCE_PROFILED(bal_finish_kernel<<<dim3((a.E + 31) / 32, a.G), 1024, 0, s>>>(a));
    return LCE_OK;
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status_t lce_balance_workspace_size(int64_t groups, int64_t T, int64_t E, int64_t k, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = bal_sizes(groups, T, E, k);
    if (st == LCE_OK) *bytes = bal_ws(groups, T, E, false, nullptr, nullptr);
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
