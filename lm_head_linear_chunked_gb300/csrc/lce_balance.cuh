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
// size.  With them first, one pass over the logits gives loss and gradient:
// per token both need q = sum_j (f_j - 1) p_tj, and
//
//   L_g = 1 + sum_t q_t / n_g.
//
// Nothing is added by atomics on floats: each block writes its own sum, and
// the last block to end adds them in a fixed order.
//
// A row of logits is short (8 to 1024 values), so a token takes only as many
// lanes of a warp as it has 16-byte vectors, and its sums as many shuffles.
#pragma once

#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {

constexpr int BAL_WARPS = 8;
constexpr int BAL_THREADS = 32 * BAL_WARPS;
// Tokens of a lane group in the ring of the pass: one in work, the others on their way.
constexpr int BAL_STAGES = 4;
// Blocks of the pass over all groups (a group's blocks share its tokens out):
// at most four on each of 152 SMs, which all run at once (one more a group
// takes a second round: 24 x 16384 x 128 63 us, not 51.5); and the fewest
// tokens that are worth one.
constexpr int64_t BAL_SMS = 152;
constexpr int64_t BAL_BLOCKS = 4 * BAL_SMS;
// Whether the tokens read ahead wait in shared memory (24 x 16384 x 128 bf16,
// loss and gradient with the counting: 51.5 us, against 62.6 from registers,
// where the waits could not be hidden) or, with several vectors a lane, in
// registers (gradient of 2^25 fp32 logits of 256: 44.7 us against 46.0).
constexpr bool bal_ring(size_t vec, int items) { return vec >= 4 && items == 1; }
// Blocks of the pass on an SM, by the experts of a lane (which it keeps in registers).
constexpr int bal_resident(int experts) { return experts <= 8 ? 4 : experts <= 16 ? 2 : 1; }
constexpr int64_t BAL_MIN_TOKENS = 32;
// Blocks per group of the counting: every block of the pass adds their counts
// up, so they are few.
constexpr int64_t BAL_COUNT_PARTS = 32;

// Up to so many tokens of a single group, one block counts and passes over
// them: one launch, not two.  Device time in us, one block against two
// launches, forward of fp32 logits:
//    experts \ tokens      64          128          512
//         8            5.9  6.4     5.5  7.1     6.3  6.9
//        64            6.7  6.9     7.7  7.9    14.0  7.1
//       256            8.3  7.9    10.8  8.4    25.0  8.2
// so the two launches are faster for many experts; the rule does not look at
// them yet.
constexpr int64_t BAL_ALONE_TOKENS = 512;

struct BalArgs {
    const void* z;
    int64_t zg, zt;  // strides of a group and of a token, in elements
    const void* idx;  // [G, T, k]
    bool idx64;
    const uint8_t* mask;  // nullable; [T] with group stride 0, or [G, T]
    int64_t mask_g;
    int64_t T, per_part, per_count;
    int32_t G, E, k, parts, count_parts;  // the pass may take fewer parts than these
    uint32_t ring_at;   // byte offset of the pass's ring in its shared memory
    bool inline_count;  // one block in all: the pass counts by itself
    // workspace
    WsHeader* hdr;
    unsigned* done;    // blocks of the pass that are through
    int32_t* part_c;   // [G, count_parts, E] counts
    int32_t* part_n;   // [G, count_parts]: kept tokens, or -1 - kept if an index is out of range
    float* part_q;     // [G, parts] sums of q
    // finished counts (read by the backward)
    const int64_t* counts;
    const int64_t* n_valid;
    float grad_scale;
    const float* d_grad_output;
    int64_t groups;    // that the loss is divided by: G, or 1 for the sum over groups
    void* dz;          // [G, T, E], contiguous
    // outputs of the forward
    float *loss, *group_loss;
    int64_t *counts_out, *n_out;
};

enum BalMode { BAL_FORWARD, BAL_BACKWARD, BAL_FUSED };

lce_status_t bal_pass_bf16(const BalArgs& a, BalMode mode, cudaStream_t s);
lce_status_t bal_pass_f16(const BalArgs& a, BalMode mode, cudaStream_t s);
lce_status_t bal_pass_f32(const BalArgs& a, BalMode mode, cudaStream_t s);

namespace {

__device__ __forceinline__ bool kept(const BalArgs& a, int g, int64_t t) {
    return !a.mask || a.mask[g * a.mask_g + t] != 0;
}

// Counts of the tokens t0 .. t1 of a group, by the whole block: a histogram
// per warp in shared memory (`hist`, [BAL_WARPS, E]), then one of the block.
__device__ __forceinline__ void count_tokens(const BalArgs& a, int g, int part, int64_t t0, int64_t t1, int32_t* hist) {
    __shared__ int32_t total, bad;
    for (int e = threadIdx.x; e < BAL_WARPS * a.E; e += BAL_THREADS) hist[e] = 0;
    if (threadIdx.x == 0) total = bad = 0;
    __syncthreads();
    int32_t* mine = hist + (threadIdx.x >> 5) * a.E;
    int32_t n = 0;
    auto count = [&](int64_t e) {
        if (e >= 0 && e < a.E)
            atomicAdd(mine + e, 1);
        else if (e != -1)
            bad = 1;
    };
    // 16 bytes of indices at a time where a token's begin on such a boundary
    const int per = a.idx64 ? 2 : 4;
    const bool vec = a.k % per == 0 && aligned_dev(a.idx);
    for (int64_t t = t0 + threadIdx.x; t < t1; t += BAL_THREADS) {
        const int64_t at = (static_cast<int64_t>(g) * a.T + t) * a.k;
        if (vec && a.idx64 && a.k <= 8) {  // the mask and all indices are read together
            const longlong2* p = reinterpret_cast<const longlong2*>(static_cast<const int64_t*>(a.idx) + at);
            longlong2 e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (2 * j < a.k) e[j] = p[j];
            if (!kept(a, g, t)) continue;
            ++n;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (2 * j < a.k) {
                    count(e[j].x);
                    count(e[j].y);
                }
            continue;
        }
        if (!kept(a, g, t)) continue;
        ++n;
        if (vec && a.idx64) {
            const longlong2* p = reinterpret_cast<const longlong2*>(static_cast<const int64_t*>(a.idx) + at);
#pragma unroll 4
            for (int j = 0; j < a.k / 2; ++j) {
                const longlong2 e = p[j];
                count(e.x);
                count(e.y);
            }
        } else if (vec) {
            const int4* p = reinterpret_cast<const int4*>(static_cast<const int32_t*>(a.idx) + at);
#pragma unroll 2
            for (int j = 0; j < a.k / 4; ++j) {
                const int4 e = p[j];
                count(e.x);
                count(e.y);
                count(e.z);
                count(e.w);
            }
        } else {
#pragma unroll 4
            for (int j = 0; j < a.k; ++j)
                count(a.idx64 ? static_cast<const int64_t*>(a.idx)[at + j]
                              : static_cast<const int32_t*>(a.idx)[at + j]);
        }
    }
    if (n) atomicAdd(&total, n);
    __syncthreads();
    const int64_t slot = static_cast<int64_t>(g) * a.count_parts + part;
    for (int e = threadIdx.x; e < a.E; e += BAL_THREADS) {
        int32_t c = 0;
#pragma unroll
        for (int w = 0; w < BAL_WARPS; ++w) c += hist[w * a.E + e];
        a.part_c[slot * a.E + e] = c;
    }
    if (threadIdx.x == 0) a.part_n[slot] = bad ? -1 - total : total;
}

// The last block of the pass adds the loss up: a warp over a group's parts,
// then the groups in order.
__device__ __forceinline__ void finish_loss(const BalArgs& a) {
    __shared__ int bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    bool wrong = false;
    for (int64_t k = threadIdx.x; k < static_cast<int64_t>(a.G) * a.count_parts; k += BAL_THREADS)
        wrong |= __ldcg(a.part_n + k) < 0;
    if (wrong) bad = 1;
    for (int g = warp; g < a.G; g += BAL_WARPS) {
        const float* from = a.part_q + static_cast<int64_t>(g) * a.parts;
        const int64_t n = __ldcg(a.n_out + g);
        float q = 0.f;
        for (int k0 = lane; k0 < a.parts; k0 += 8 * 32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k0 + i * 32 < a.parts ? __ldcg(from + k0 + i * 32) : 0.f;
            q += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        q = warp_sum(q);
        // the group's loss takes the place of its first part's sum
        if (lane == 0) {
            q = n > 0 ? 1.f + q / static_cast<float>(n) : 0.f;
            if (a.group_loss) a.group_loss[g] = q;
            a.part_q[static_cast<int64_t>(g) * a.parts] = q;
        }
    }
    __syncthreads();
    if (warp != 0) return;
    float total = 0.f;
    for (int g = lane; g < a.G; g += 32) total += a.part_q[static_cast<int64_t>(g) * a.parts];
    total = warp_sum(total);
    if (lane == 0) {
        a.hdr->status = bad ? STATUS_INDEX : 0u;
        *a.loss = bad ? __int_as_float(0x7FC00000) : total / static_cast<float>(a.groups);
    }
}

// One pass over a part's logits: the loss, the gradient, or both.  INLINE: the
// only block counts first.
// Vector i of lane l holds the experts (i lanes + l) VEC + 0 .. VEC - 1; the
// next tokens' vectors are read while this one's are worked on.  A token that
// the mask leaves out counts as a row of zeros with a factor of zero, so what
// it holds is never used and the lanes of a warp stay together.
template <typename T, int VEC, int LANES, int ITEMS, int MODE>
__global__ void __launch_bounds__(BAL_THREADS, bal_resident(ITEMS * VEC)) bal_pass_kernel(BalArgs a) {
    constexpr bool LOSS = MODE != BAL_BACKWARD, GRAD = MODE != BAL_FORWARD;
    constexpr int PAIRS = ITEMS * VEC / 2;
    constexpr float LOG2E = 1.4426950408889634f;
    using V = Vec<T, VEC>;
    extern __shared__ __align__(16) float sm[];  // f [E]; with the counting inline, histograms [BAL_WARPS, E]; the ring
    __shared__ float warp_q[BAL_WARPS];
    __shared__ bool last;
    __shared__ float scale_s;
    __shared__ int64_t n_s;
    const int g = blockIdx.y, part = blockIdx.x;
    constexpr int tpw = 32 / LANES;                 // tokens of a warp at a time
    constexpr bool RING = bal_ring(sizeof(V), ITEMS);
    constexpr int AHEAD = RING ? BAL_STAGES - 1 : 1;  // tokens read ahead
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (LANES - 1), sub = lane / LANES;
    const int n = a.E / VEC;
    const bool whole = n == LANES * ITEMS;  // no lane has a vector outside the row
    const int64_t t0 = part * a.per_part, t1 = t0 + a.per_part < a.T ? t0 + a.per_part : a.T;
    // from here on tokens count from the part's first, in 32 bits
    const int tokens = t1 > t0 ? static_cast<int>(t1 - t0) : 0;
    constexpr int step = BAL_WARPS * tpw;
    int t = warp * tpw + sub;
    const V* src = reinterpret_cast<const V*>(static_cast<const T*>(a.z) + g * a.zg + (t0 + t) * a.zt) + l;
    const int64_t src_step = step * a.zt / VEC;
    V* dst = GRAD ? reinterpret_cast<V*>(static_cast<T*>(a.dz) + (static_cast<int64_t>(g) * a.T + t0 + t) * a.E) + l : nullptr;
    const uint8_t* keep = a.mask ? a.mask + g * a.mask_g + t0 : nullptr;
    // a thread's own vectors of the next tokens, in shared memory; or in registers
    // (RING); the mask's bytes wait as they were read
    V* ring = reinterpret_cast<V*>(reinterpret_cast<char*>(sm) + a.ring_at) + threadIdx.x;
    V next[RING ? 1 : ITEMS];
    uint32_t next_ok[AHEAD];
    auto fetch = [&](int at, int slot, uint32_t* valid) {
        *valid = at < tokens;
        if (at < tokens) {
            if (keep) *valid = keep[at];
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (whole || i * LANES + l < n) {
                    if constexpr (RING)
                        copy_async<sizeof(V)>(ring + (slot * ITEMS + i) * BAL_THREADS, src + i * LANES);
                    else
                        next[i] = src[i * LANES];
                }
        }
        if constexpr (RING) copy_async_commit();
        src += src_step;
    };
    // the first tokens are on their way while the counts are waited for and added up:
    // the logits and the mask were there before the counting began (24 x 16384 x 128
    // 53.5 -> 52.9 us, 131072 x 256 fp32 gradient 46.6 -> 46.0; small calls alike)
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) fetch(t + k * step, k, next_ok + k);
    if (LOSS && !a.inline_count) wait_for_primary();  // the counts
    if (LOSS && a.inline_count) {
        if (threadIdx.x == 0) *a.done = 0;
        count_tokens(a, g, part, t0, t1, reinterpret_cast<int32_t*>(sm));
        __syncthreads();
    }
    F2 f[PAIRS];
    float scale = 0.f, q_sum = 0.f;
    auto column = [&](int e) { return ((e / VEC) * LANES + l) * VEC + e % VEC; };
    {
        // f - 1 = (c E - k n) / (k n), the numerator exact in integers, from the group's
        // counts: finished (the backward), or the sums of their parts.  (In FP64, at 1/64
        // of the rate, 24 x 16384 x 128 took 80 us, not 76.)
        if (warp == 0) {
            int32_t m = 0;
            if (LOSS)
                for (int q = lane; q < a.count_parts; q += 32) {
                    const int32_t v = a.part_n[static_cast<int64_t>(g) * a.count_parts + q];
                    m += v < 0 ? -1 - v : v;
                }
            const int64_t kept_n = MODE == BAL_BACKWARD ? a.n_valid[g] : __reduce_add_sync(0xFFFFFFFFu, m);
            if (lane == 0) {
                const float go = a.d_grad_output ? *a.d_grad_output : 1.f;
                n_s = kept_n;
                if (LOSS && part == 0) a.n_out[g] = kept_n;
                if (GRAD) scale_s = kept_n > 0 ? a.grad_scale * go / static_cast<float>(a.groups * kept_n) : 0.f;
            }
        }
        int64_t c = 0;
        for (int e0 = 0; e0 < a.E; e0 += BAL_THREADS) {
            const int e = e0 + threadIdx.x;
            c = 0;
            if (e < a.E) {
                if (MODE == BAL_BACKWARD) {
                    c = a.counts[static_cast<int64_t>(g) * a.E + e];
                } else {
#pragma unroll 16
                    for (int q = 0; q < a.count_parts; ++q)
                        c += a.part_c[(static_cast<int64_t>(g) * a.count_parts + q) * a.E + e];
                }
            }
            if (e0 == 0) __syncthreads();  // n_s
            const int64_t all = a.k * n_s;
            if (LOSS && part == 0 && e < a.E) a.counts_out[static_cast<int64_t>(g) * a.E + e] = c;
            if (e < a.E) sm[e] = all > 0 ? static_cast<float>(c * a.E - all) / static_cast<float>(all) : 0.f;
        }
        __syncthreads();
        if (GRAD) scale = scale_s;
    }
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
        const int c0 = column(2 * p), c1 = column(2 * p + 1);
        f[p] = f2(c0 < a.E ? sm[c0] : 0.f, c1 < a.E ? sm[c1] : 0.f);
    }
    int slot = 0;
    // the warp's first subgroup has the lowest token: the warp goes on while that one has
    for (; t - sub < tokens; t += step) {
        RowVectors<T, VEC, ITEMS> z;
        const bool ok = next_ok[0] != 0;
#pragma unroll
        for (int k = 0; k + 1 < AHEAD; ++k) next_ok[k] = next_ok[k + 1];
        if constexpr (RING) {
            // into the stage that the last token was read from
            fetch(t + AHEAD * step, slot == 0 ? BAL_STAGES - 1 : slot - 1, next_ok + AHEAD - 1);
            copy_async_wait<AHEAD>();
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) z.v[i] = ok ? ring[(slot * ITEMS + i) * BAL_THREADS] : V{};
            if (++slot == BAL_STAGES) slot = 0;
        } else {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) z.v[i] = ok ? next[i] : V{};
            fetch(t + step, 0, next_ok);
        }
        F2 v[PAIRS];
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            v[p] = z.pair(p);
            if (!whole)
                v[p] = f2((2 * p / VEC) * LANES + l < n ? lo(v[p]) : -INFINITY,
                          ((2 * p + 1) / VEC) * LANES + l < n ? hi(v[p]) : -INFINITY);
        }
        float m = -INFINITY;
        if (sizeof(T) == 2 && VEC > 1 && whole) {
            m = z.max();  // two at a time in 16 bits: a maximum does not round
        } else {
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) m = fmaxf(m, fmaxf(lo(v[p]), hi(v[p])));
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        // The difference first, so that the largest has the exponent 0 whatever its size: a
        // row of the type's lowest value is as even as one of zeros.  (With m log2 e rounded
        // by itself, one fused multiply-add, rows beyond about 1e9 gave NaN; 24 x 16384 x 128
        // took 52.8 us, not 53.3, and 55.4 with this form for large rows only.)
        const F2 m2 = f2(-m), l2 = f2(LOG2E);
        F2 s2 = f2(0.f), q2 = f2(0.f);
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            const F2 y = mul2(add2(v[p], m2), l2);
            v[p] = f2(fast_exp2(lo(y)), fast_exp2(hi(y)));
            s2 = add2(s2, v[p]);
            q2 = fma2(f[p], v[p], q2);
        }
        float s = lo(s2) + hi(s2), q = lo(q2) + hi(q2);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
        }
        const float r = ok ? fast_rcp(s) : 0.f;
        q *= r;
        if (LOSS) q_sum += q;
        if (GRAD) {
            const F2 fq = f2(-q), sr = f2(scale * r);
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) z.set(p, mul2(mul2(v[p], sr), add2(f[p], fq)));
        }
        if (GRAD) {
            if (t < tokens)
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (whole || i * LANES + l < n) dst[i * LANES] = z.v[i];
            dst += step * n;
        }
    }
    if (!LOSS) return;
    // the subgroups of a warp (each of their lanes has their sum), then the warps
    q_sum = warp_sum(l == 0 ? q_sum : 0.f);
    if (lane == 0) warp_q[warp] = q_sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        q_sum = 0.f;
        for (int w = 0; w < BAL_WARPS; ++w) q_sum += warp_q[w];
        a.part_q[static_cast<int64_t>(g) * a.parts + part] = q_sum;
        __threadfence();  // with the counts of part 0, which the barrier put before this
        last = atomicAdd(a.done, 1u) == gridDim.x * gridDim.y - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    finish_loss(a);
}

template <typename T, int VEC, int LANES, int ITEMS>
lce_status_t bal_pass_form(BalArgs a, BalMode mode, cudaStream_t s) {
    const int64_t fit = BAL_SMS * bal_resident(ITEMS * VEC) / a.G;
    if (a.parts > fit) a.parts = static_cast<int32_t>(fit > 1 ? fit : 1);
    a.per_part = (a.T + a.parts - 1) / a.parts;
    const dim3 grid(a.parts, a.G);
    // at most 32 KB: histograms of 1024 experts without a ring, or of 256 beside one of 16 KB
    a.ring_at = (static_cast<uint32_t>(a.E) * 4 * (a.inline_count ? BAL_WARPS : 1) + 15u) / 16u * 16u;
    constexpr size_t vec = sizeof(Vec<T, VEC>);
    const size_t smem = a.ring_at + (bal_ring(vec, ITEMS) ? BAL_STAGES * BAL_THREADS * vec : 0);
    auto kernel = mode == BAL_FORWARD    ? bal_pass_kernel<T, VEC, LANES, ITEMS, BAL_FORWARD>
                  : mode == BAL_BACKWARD ? bal_pass_kernel<T, VEC, LANES, ITEMS, BAL_BACKWARD>
                                         : bal_pass_kernel<T, VEC, LANES, ITEMS, BAL_FUSED>;
    if (mode == BAL_BACKWARD || a.inline_count)
        LCE_PROFILED(kernel<<<grid, BAL_THREADS, smem, s>>>(a));
    else
        LCE_PROFILED(launch_after(kernel, grid, BAL_THREADS, smem, s, a));
    return LCE_OK;
}

// Rows that start on 16-byte boundaries are read in 16-byte vectors, else in
// 8-byte ones where that fits (60 experts in 16 bits), else by the element.
template <typename T>
lce_status_t bal_pass(const BalArgs& a, BalMode mode, cudaStream_t s) {
    auto fits = [&](int vec) {
        const size_t b = vec * sizeof(T);
        return a.E % vec == 0 && a.zt % vec == 0 && a.zg % vec == 0 && aligned_to(a.z, b) && aligned_to(a.dz, b);
    };
    constexpr int V16 = 16 / sizeof(T), V8 = 8 / sizeof(T);
    if (fits(V16)) {
        const int n = a.E / V16;
        return n <= 1    ? bal_pass_form<T, V16, 1, 1>(a, mode, s)
               : n <= 2  ? bal_pass_form<T, V16, 2, 1>(a, mode, s)
               : n <= 4  ? bal_pass_form<T, V16, 4, 1>(a, mode, s)
               : n <= 8  ? bal_pass_form<T, V16, 8, 1>(a, mode, s)
               : n <= 16 ? bal_pass_form<T, V16, 16, 1>(a, mode, s)
               : n <= 32 ? bal_pass_form<T, V16, 32, 1>(a, mode, s)
               : n <= 64 ? bal_pass_form<T, V16, 32, 2>(a, mode, s)
                         : bal_pass_form<T, V16, 32, LCE_BALANCE_MAX_E / (32 * V16)>(a, mode, s);
    }
    if (fits(V8)) {
        const int n = a.E / V8;
        return n <= 16   ? bal_pass_form<T, V8, 16, 1>(a, mode, s)
               : n <= 32 ? bal_pass_form<T, V8, 32, 1>(a, mode, s)
                         : bal_pass_form<T, V8, 32, LCE_BALANCE_MAX_E / (32 * V8)>(a, mode, s);
    }
    return a.E <= 16    ? bal_pass_form<T, 1, 8, 2>(a, mode, s)
           : a.E <= 64  ? bal_pass_form<T, 1, 32, 2>(a, mode, s)
           : a.E <= 256 ? bal_pass_form<T, 1, 32, 8>(a, mode, s)
                        : bal_pass_form<T, 1, 32, 32>(a, mode, s);
}

}  // namespace
}  // namespace lce
