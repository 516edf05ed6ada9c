// The balance loss of a mixture of experts, its per-expert counts and its
// gradient.  For each group g (a layer or a sequence) of T tokens, E experts
// and k slots per token, over the n_g tokens that the mask keeps:
//
//   p = softmax_e(z),  c_e = slots that name e,  f_e = c_e E / (k n_g)
//   L_g = sum_e f_e P_e,  P_e = sum_t p_te / n_g        (0 when n_g = 0)
//   dL_g/dz_te = p_te (f_e - sum_j f_j p_tj) / n_g
//
// A row of p adds up to 1, so f - 1 in place of f gives the same gradient,
// without the cancellation of two numbers near 1 when the load is even.
//
// The counts need only the expert indices, which are k/E of the logits'
// size, so the loss and its gradient together take one pass over the logits.
// Nothing is added by atomics on floats: each block writes its own sums, and
// they are added in a fixed order.
#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int BAL_WARPS = 8;
constexpr int BAL_THREADS = 32 * BAL_WARPS;
// Blocks over all groups (a group's blocks share its tokens out), and the
// fewest tokens that are worth one.
constexpr int64_t BAL_BLOCKS = 1216;
constexpr int64_t BAL_MIN_TOKENS = 32;

struct BalArgs {
    const void* z;
    int64_t zg, zt;  // strides of a group and of a token, in elements
    const void* idx;  // [G, T, k]
    bool idx64;
    const uint8_t* mask;  // nullable; [T] with group stride 0, or [G, T]
    int64_t mask_g;
    int64_t T, per_part;
    int32_t G, E, k, parts;
    // workspace: per (group, part) the counts, the kept tokens and the sums of p
    WsHeader* hdr;
    int32_t* part_c;   // [G, parts, E]
    int32_t* part_n;   // [G, parts]: kept tokens, or -1 - kept if an index is out of range
    float* part_p;     // [G, parts, E]
    // finished counts (read by the backward)
    const int64_t* counts;
    const int64_t* n_valid;
    float grad_scale;
    const float* d_grad_output;
    float inv_groups;  // 1 / G, or 1 for the sum over groups
    void* dz;          // [G, T, E], contiguous
};

__device__ __forceinline__ bool kept(const BalArgs& a, int g, int64_t t) {
    return !a.mask || a.mask[g * a.mask_g + t] != 0;
}

// Counts of one part of a group's tokens.
__global__ void __launch_bounds__(BAL_THREADS) bal_count_kernel(BalArgs a) {
    extern __shared__ int32_t cnt[];  // [E]
    __shared__ int32_t total, bad;
    const int g = blockIdx.y, part = blockIdx.x;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
    if (threadIdx.x == 0) total = bad = 0;
    __syncthreads();
    const int64_t t0 = part * a.per_part, t1 = t0 + a.per_part < a.T ? t0 + a.per_part : a.T;
    const int64_t n = (t1 - t0) * a.k;
    const int64_t base = (static_cast<int64_t>(g) * a.T + t0) * a.k;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
        const int64_t t = i / a.k;
        if (!kept(a, g, t0 + t)) continue;
        const int64_t e = a.idx64 ? static_cast<const int64_t*>(a.idx)[base + i]
                                  : static_cast<const int32_t*>(a.idx)[base + i];
        if (e >= 0 && e < a.E)
            atomicAdd(cnt + e, 1);
        else if (e != -1)
            bad = 1;
    }
    int32_t mine = 0;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += blockDim.x) mine += kept(a, g, t);
    if (mine) atomicAdd(&total, mine);
    __syncthreads();
    const int64_t slot = static_cast<int64_t>(g) * a.parts + part;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.part_c[slot * a.E + e] = cnt[e];
    if (threadIdx.x == 0) a.part_n[slot] = bad ? -1 - total : total;
}

// One pass over a part's logits: with SUM the column sums of p, with GRAD the
// gradient.  A warp per token, lane l holds the experts l, l + 32, ...
template <typename T, int PER, bool SUM, bool GRAD>
__global__ void __launch_bounds__(BAL_THREADS) bal_pass_kernel(BalArgs a) {
    extern __shared__ float sm[];  // f [E] with GRAD, then the warps' sums [BAL_WARPS, E] with SUM
    float* fs = sm;
    float* ps = sm + (GRAD ? a.E : 0);
    __shared__ float scale_s;
    const int g = blockIdx.y, part = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (GRAD) {
        // the group's counts: finished (the backward), or the sums of its parts
        int64_t n = 0;
        if (a.counts) {
            n = a.n_valid[g];
        } else {
            for (int q = 0; q < a.parts; ++q) {
                const int32_t m = a.part_n[static_cast<int64_t>(g) * a.parts + q];
                n += m < 0 ? -1 - m : m;
            }
        }
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            int64_t c = 0;
            if (a.counts) {
                c = a.counts[static_cast<int64_t>(g) * a.E + e];
            } else {
                for (int q = 0; q < a.parts; ++q) c += a.part_c[(static_cast<int64_t>(g) * a.parts + q) * a.E + e];
            }
            fs[e] = n > 0 ? static_cast<float>(static_cast<double>(c) * a.E / (static_cast<double>(a.k) * n) - 1.0) : 0.f;
        }
        if (threadIdx.x == 0) {
            const float go = a.d_grad_output ? *a.d_grad_output : 1.f;
            scale_s = n > 0 ? static_cast<float>(static_cast<double>(a.grad_scale) * go * a.inv_groups / n) : 0.f;
        }
        __syncthreads();
    }
    float f[PER], sum[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        f[i] = GRAD && e < a.E ? fs[e] : 0.f;
        sum[i] = 0.f;
    }
    const float scale = GRAD ? scale_s : 0.f;
    const int64_t t0 = part * a.per_part, t1 = t0 + a.per_part < a.T ? t0 + a.per_part : a.T;
    for (int64_t t = t0 + warp; t < t1; t += BAL_WARPS) {
        const bool ok = kept(a, g, t);
        T* dz = GRAD ? static_cast<T*>(a.dz) + (static_cast<int64_t>(g) * a.T + t) * a.E : nullptr;
        if (!ok) {
            if (GRAD)
                for (int e = lane; e < a.E; e += 32) dz[e] = from_f32<T>(0.f);
            continue;
        }
        const T* z = static_cast<const T*>(a.z) + g * a.zg + t * a.zt;
        float v[PER], m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            v[i] = e < a.E ? to_f32(z[e]) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float s = 0.f, fp = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            // the max's product rounds the same way for every expert of the row and cancels in p
            v[i] = e < a.E ? exp2f(fmaf(v[i], LOG2E, -m * LOG2E)) : 0.f;
            s += v[i];
            if (GRAD) fp = fmaf(f[i], v[i], fp);
        }
        s = warp_sum(s);
        if (GRAD) fp = warp_sum(fp);
        const float r = 1.f / s;
        fp *= r;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            const float p = v[i] * r;
            if (SUM) sum[i] += p;
            if (GRAD && e < a.E) dz[e] = from_f32<T>(scale * p * (f[i] - fp));
        }
    }
    if (SUM) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            if (e < a.E) ps[warp * a.E + e] = sum[i];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < BAL_WARPS; ++w) v += ps[w * a.E + e];
            a.part_p[(static_cast<int64_t>(g) * a.parts + part) * a.E + e] = v;
        }
    }
}

// Adds the parts up: counts, kept tokens, each group's loss, and the loss.
// One block; the groups one after the other.
__global__ void __launch_bounds__(256) bal_finish_kernel(BalArgs a, float* loss, float* group_loss, int64_t* counts,
                                                         int64_t* n_valid) {
    __shared__ double part[8];
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    double total = 0.0;
    for (int g = 0; g < a.G; ++g) {
        int64_t n = 0;
        for (int q = 0; q < a.parts; ++q) {
            const int32_t m = a.part_n[static_cast<int64_t>(g) * a.parts + q];
            n += m < 0 ? -1 - m : m;
            if (m < 0) bad = 1;
        }
        double v = 0.0;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            int64_t c = 0;
            double p = 0.0;
            for (int q = 0; q < a.parts; ++q) {
                const int64_t at = (static_cast<int64_t>(g) * a.parts + q) * a.E + e;
                c += a.part_c[at];
                p += a.part_p[at];
            }
            counts[static_cast<int64_t>(g) * a.E + e] = c;
            v += static_cast<double>(c) * p;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
            double s = 0.0;
            for (int w = 0; w < 8; ++w) s += part[w];
            s = n > 0 ? s * a.E / (static_cast<double>(a.k) * n * n) : 0.0;
            if (group_loss) group_loss[g] = static_cast<float>(s);
            n_valid[g] = n;
            total += s;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.hdr->status = bad ? STATUS_INDEX : 0u;
        *loss = bad ? __int_as_float(0x7FC00000) : static_cast<float>(total * a.inv_groups);
    }
}

template <bool SUM, bool GRAD>
lce_status_t bal_pass(const BalArgs& a, int dtype, cudaStream_t s) {
    const size_t smem = static_cast<size_t>(a.E) * 4 * ((GRAD ? 1 : 0) + (SUM ? BAL_WARPS : 0));
    const dim3 grid(a.parts, a.G);
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        if (a.E <= 64)
            LCE_PROFILED(bal_pass_kernel<T, 2, SUM, GRAD><<<grid, BAL_THREADS, smem, s>>>(a));
        else if (a.E <= 256)
            LCE_PROFILED(bal_pass_kernel<T, 8, SUM, GRAD><<<grid, BAL_THREADS, smem, s>>>(a));
        else
            LCE_PROFILED(bal_pass_kernel<T, 32, SUM, GRAD><<<grid, BAL_THREADS, smem, s>>>(a));
        return LCE_OK;
    });
}

int64_t bal_parts(int64_t G, int64_t T) {
    const int64_t most = (T + BAL_MIN_TOKENS - 1) / BAL_MIN_TOKENS;
    int64_t p = (BAL_BLOCKS + G - 1) / G;
    return p < most ? p : most;
}

lce_status_t bal_sizes(int64_t G, int64_t T, int64_t E, int64_t k) {
    if (G <= 0 || T <= 0 || E <= 0 || k <= 0) return LCE_ERR_INVALID_ARG;
    if (G > 65535 || T > INT32_MAX || E > LCE_BALANCE_MAX_E || k > E) return LCE_ERR_UNSUPPORTED;
    return LCE_OK;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t bal_ws(int64_t G, int64_t T, int64_t E, BalArgs* a, void* ws) {
    const int64_t parts = bal_parts(G, T);
    const size_t c = 1024, n = c + align256(static_cast<size_t>(G * parts * E) * 4);
    const size_t p = n + align256(static_cast<size_t>(G * parts) * 4);
    if (a) {
        uint8_t* w = static_cast<uint8_t*>(ws);
        a->parts = static_cast<int32_t>(parts);
        a->per_part = (T + parts - 1) / parts;
        a->hdr = reinterpret_cast<WsHeader*>(w);
        a->part_c = reinterpret_cast<int32_t*>(w + c);
        a->part_n = reinterpret_cast<int32_t*>(w + n);
        a->part_p = reinterpret_cast<float*>(w + p);
    }
    return p + align256(static_cast<size_t>(G * parts * E) * 4);
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
    a->inv_groups = (in.flags & LCE_REDUCTION_SUM) ? 1.f : 1.f / static_cast<float>(in.G);
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
    const dim3 grid(a.parts, a.G);
    LCE_PROFILED(bal_count_kernel<<<grid, BAL_THREADS, static_cast<size_t>(a.E) * 4, s>>>(a));
    const lce_status_t pt = grad ? bal_pass<true, true>(a, in.dtype, s) : bal_pass<true, false>(a, in.dtype, s);
    if (pt != LCE_OK) return pt;
    LCE_PROFILED(bal_finish_kernel<<<1, 256, 0, s>>>(a, loss, group_loss, counts, n_valid));
    return LCE_OK;
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
    return bal_pass<false, true>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
