// Beam search: selection over beams and vocabulary, and reordering of the
// beams' states.
//
// Selection, for item b with beams k, logits z and scores s:
//   candidate (k, v) has s_k + z_kv - lse_k,  lse_k = ln sum_v exp z_kv;
//   a finished beam has one candidate, its own score with the pad token.
// The M best leave in the order (score down, beam up, logit down, token up).
// Within a beam the scores are ordered as the logits are, so the scan keeps,
// for a part of a row, the M largest of 64-bit keys (the logit's bits made
// monotone, then the token's complement: all keys differ, and the lower token
// wins among equal logits), next to the part's maximum and sum of
// exponentials.  The join adds the parts of each beam up and merges the
// beams, comparing scores in FP64: two candidates of different beams compare
// as their exact scores do unless these are within a few 2^-24.
#include <float.h>

#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int SCAN_THREADS = 256;
constexpr int SCAN_WARPS = SCAN_THREADS / 32;
constexpr int SCAN_CAP = 1024;                        // keys the buffer holds beside the list
constexpr int SCAN_HIGH = 256;                        // keys that start a merge
constexpr int SCAN_SEGS_MAX = 32;                     // parts of a row (a lane each in the join)
constexpr int64_t SCAN_BLOCKS = 608;                  // blocks that fill the GPU
constexpr int JOIN_WARPS = 8;
constexpr int MAX_M = LCE_BEAM_MAX;
constexpr int JOIN_SMEM_MAX = MAX_M * 8 * (2 * MAX_M + JOIN_WARPS * SCAN_SEGS_MAX);
static_assert(JOIN_SMEM_MAX <= 224 * 1024, "dynamic shared memory of a block");

// Logits as the selection sees them: NaN as -inf, +inf as the largest finite.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ uint64_t logit_key(float x, uint32_t token) {
    const uint32_t b = __float_as_uint(clean(x) + 0.f);  // -0 becomes +0
    const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - token);
}

__device__ __forceinline__ float key_logit(uint64_t key) {
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

__device__ __forceinline__ uint32_t key_token(uint64_t key) { return 0xFFFFFFFFu - static_cast<uint32_t>(key); }

// The largest of the warp's keys, by its two halves.
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t h = static_cast<uint32_t>(v >> 32);
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, h);
    const uint32_t low = __reduce_max_sync(0xFFFFFFFFu, h == top ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(top) << 32) | low;
}

// A sum in two floats: the exact error of each addition of the first goes to
// the second.  FP64 adds run at 1/64 of the rate here.
struct Sum2 {
    float hi, lo;
    __device__ __forceinline__ void add(float x, float x_lo = 0.f) {
        const float t = hi + x, back = t - hi;
        lo += ((hi - (t - back)) + (x - back)) + x_lo;
        hi = t;
    }
    __device__ __forceinline__ void scale(float f) {
        const float h = hi * f;
        lo = fmaf(lo, f, fmaf(hi, f, -h));
        hi = h;
    }
    // The sum over the warp, in every lane.
    __device__ __forceinline__ void over_warp() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            add(__shfl_xor_sync(0xFFFFFFFFu, hi, o), __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    }
};

struct ScanArgs {
    const void* z;
    int64_t ld;
    const uint8_t* finished;  // [rows], nullable
    int32_t V, M, segs, per_seg;  // per_seg: chunks of a segment
    float* seg_m;      // [rows, segs]
    float2* seg_s;     // the sum relative to seg_m, in two floats
    uint64_t* seg_key;  // [rows, segs, M], sorted down; 0: no candidate
};

struct ScanShared {
    alignas(16) uint64_t buf[MAX_M + SCAN_CAP + 2];  // the list's keys, then the new ones
    float2 red_s[SCAN_WARPS];
    float red_m[SCAN_WARPS];
    uint64_t red_k[SCAN_WARPS];
    int n;
};

// Keeps the M largest of buf[0..n) at its front, sorted down; returns how many
// there are.  A key's place is the number of larger ones.
__device__ int keep_best(ScanShared& sh, int n, int M) {
    constexpr int PER = (MAX_M + SCAN_CAP + SCAN_THREADS - 1) / SCAN_THREADS;
    if (threadIdx.x == 0) sh.buf[n] = 0;  // read with the last key of an odd number
    __syncthreads();
    uint64_t key[PER];
    int rank[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int i = q * SCAN_THREADS + threadIdx.x;
        rank[q] = M;
        if (q * SCAN_THREADS < n && i < n) {
            key[q] = sh.buf[i];
            int r = 0;
#pragma unroll 4
            for (int j = 0; j < n; j += 2) {
                const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(sh.buf + j);
                r += (k.x > key[q]) + (k.y > key[q]);
            }
            rank[q] = r;
        }
    }
    __syncthreads();
    if (n > M) n = M;
#pragma unroll
    for (int q = 0; q < PER; ++q)
        if (rank[q] < M) sh.buf[rank[q]] = key[q];
    if (threadIdx.x == 0) sh.n = n;
    __syncthreads();
    return n;
}

// One thread's elements of a chunk: vector u holds the tokens
// first + (u * SCAN_THREADS + thread) * VEC + j.  The places do not depend on
// the alignment, so equal rows give equal sums.
template <typename T, int PER>
struct Chunk : RowVectors<T, vec16<T>(), PER / vec16<T>()> {
    static constexpr int VEC = vec16<T>(), N = PER / VEC;
    using Base = RowVectors<T, VEC, N>;
    using Base::v;

    static __device__ __forceinline__ uint32_t token(uint32_t first, int i) {
        return first + ((i / VEC) * SCAN_THREADS + threadIdx.x) * VEC + i % VEC;
    }
    __device__ __forceinline__ float at(int i) const { return v[i / VEC].f(i % VEC); }
    // A vector of a row that starts SHIFT bytes past a 16-byte boundary, cut
    // out of the two that it lies in.
    template <int SHIFT>
    static __device__ __forceinline__ Vec<T, VEC> cut(const char* p) {
        const uint4 a = *reinterpret_cast<const uint4*>(p - SHIFT);
        const uint4 b = *reinterpret_cast<const uint4*>(p - SHIFT + 16);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = SHIFT % 4 ? __funnelshift_r(w[k + SHIFT / 4], w[k + SHIFT / 4 + 1], SHIFT % 4 * 8) : w[k + SHIFT / 4];
        Vec<T, VEC> r;
        __builtin_memcpy(&r, o, 16);
        return r;
    }
    // The chunk's vectors; at the ends of an unaligned row, and past the end of
    // any (-inf), elements are read singly.
    template <int SHIFT>
    __device__ __forceinline__ void load_from(const T* row, uint32_t first, uint32_t V) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t t = token(first, u * VEC);
            const char* p = reinterpret_cast<const char*>(row + t);
            if (SHIFT == 0 && t + VEC <= V)
                v[u] = *reinterpret_cast<const Vec<T, VEC>*>(p);
            else if (SHIFT != 0 && t >= VEC && t + 2 * VEC <= V)
                v[u] = cut<SHIFT>(p);
            else
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[u].v[j] = t + j < V ? row[t + j] : from_f32<T>(-INFINITY);
        }
    }
    __device__ __forceinline__ void load(const T* row, uint32_t first, uint32_t V, uint32_t shift) {
        if (shift == 0) return load_from<0>(row, first, V);
        if (shift == 4) return load_from<4>(row, first, V);
        if (shift == 8) return load_from<8>(row, first, V);
        if (shift == 12) return load_from<12>(row, first, V);
        if constexpr (sizeof(T) == 2) {
            if (shift == 2) return load_from<2>(row, first, V);
            if (shift == 6) return load_from<6>(row, first, V);
            if (shift == 10) return load_from<10>(row, first, V);
            if (shift == 14) return load_from<14>(row, first, V);
        }
    }
    // The largest logit as read (NaN only if all are).
    __device__ __forceinline__ float largest() const {
        if constexpr (sizeof(T) == 2) {
            return this->max();
        } else {
            float m = v[0].v[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) m = fmaxf(m, at(i));
            return m;
        }
    }
    // The sum of e^(x - m).
    __device__ __forceinline__ float sum(float m) const {
        F2 s0 = f2(0.f), s1 = f2(0.f);
        const F2 m2 = f2(-m), l2 = f2(LOG2E);
#pragma unroll
        for (int p = 0; p < PER / 2; p += 2) {
            const F2 a = mul2(add2(this->pair(p), m2), l2), b = mul2(add2(this->pair(p + 1), m2), l2);
            s0 = add2(s0, f2(fast_exp2(lce::lo(a)), fast_exp2(lce::hi(a))));
            s1 = add2(s1, f2(fast_exp2(lce::lo(b)), fast_exp2(lce::hi(b))));
        }
        s0 = add2(s0, s1);
        const float s = lce::lo(s0) + lce::hi(s0);
        if (s < INFINITY) return s;
        float c = 0.f;  // a NaN or an infinity among them
#pragma unroll
        for (int i = 0; i < PER; ++i) c += fast_exp2((clean(at(i)) - m) * LOG2E);
        return c;
    }
};

// The M best of the chunk's own elements by rounds of a block-wide maximum,
// appended to the buffer: for chunks whose candidates overflow it.
template <typename T, int PER>
__device__ void best_by_rounds(ScanShared& sh, const Chunk<T, PER>& c, uint32_t first, uint32_t V, int M, int n) {
    uint64_t below = ~0ull;
    for (int r = 0; r < M; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t t = c.token(first, i);
            const uint64_t k = t < V ? logit_key(c.at(i), t) : 0;
            if (k < below && k > best) best = k;
        }
        best = warp_max(best);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh.red_k[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int w = 0; w < SCAN_WARPS; ++w) best = sh.red_k[w] > best ? sh.red_k[w] : best;
        if (threadIdx.x == 0) sh.buf[n + r] = best;
        below = best;
    }
    __syncthreads();
}

template <typename T, int PER>
__global__ void __launch_bounds__(SCAN_THREADS, 4) beam_scan_kernel(ScanArgs a) {
    constexpr uint32_t CHUNK = SCAN_THREADS * PER;
    __shared__ ScanShared sh;
    launch_dependents();
    const int64_t row = blockIdx.y;
    const int seg = blockIdx.x;
    if (a.finished && a.finished[row]) return;  // the join does not read its parts
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) & 15u);
    const uint32_t V = static_cast<uint32_t>(a.V);
    const uint64_t begin = static_cast<uint64_t>(seg) * a.per_seg * CHUNK;
    uint64_t end = begin + static_cast<uint64_t>(a.per_seg) * CHUNK;
    if (end > V) end = V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;         // keys in the buffer (all threads agree)
    uint64_t tau = 0;  // the M-th best so far, 0 while there are fewer
    float m = -INFINITY;
    Sum2 s{0.f, 0.f};
    if (threadIdx.x == 0) sh.n = 0;
    for (uint64_t first64 = begin; first64 < end; first64 += CHUNK) {
        const uint32_t first = static_cast<uint32_t>(first64);
        Chunk<T, PER> c;
        c.load(z, first, V, shift);
        const float raw = c.largest(), mx = clean(raw);
        const float m2 = fmaxf(m, mx);
        if (m2 > -INFINITY) {
            if (m2 > m) s.scale(fast_exp2((m - m2) * LOG2E));  // of nothing at first
            s.add(c.sum(m2));
            m = m2;
        }
        // candidates: in a part's first chunk those that are at least as large as the
        // r-th largest thread's maximum of every warp, r = M / 8 (M of them exist), later
        // those above the M-th best so far (a later token loses against an equal one)
        uint64_t limit = tau;
        if (tau == 0) {
            int at = 0;
            if (mx > -INFINITY)
#pragma unroll
                for (int i = PER - 1; i >= 0; --i) at = c.at(i) >= raw ? i : at;
            const uint32_t t = first + ((at / c.VEC) * SCAN_THREADS + threadIdx.x) * c.VEC + at % c.VEC;
            const uint64_t k = t < V ? logit_key(mx, t) : 0;
            const int r = (a.M + SCAN_WARPS - 1) / SCAN_WARPS;
            uint64_t below = k, rth = 0;
            for (int i = 0; i < r; ++i) {
                rth = warp_max(below);
                if (below == rth) below = 0;
            }
            if (lane == 0) sh.red_k[warp] = rth;
            __syncthreads();
            limit = sh.red_k[0];
#pragma unroll
            for (int w = 1; w < SCAN_WARPS; ++w) limit = sh.red_k[w] < limit ? sh.red_k[w] : limit;
            if (limit) --limit;  // 0, all pass: a warp with fewer than r threads that have elements
        }
        // (the barrier also puts the count of the chunk before it ahead of the pushes)
        const bool some = logit_key(mx, 0) > limit;
        if (!__syncthreads_or(some)) continue;
        if (some) {
            const float least = key_logit(limit + 1);
            uint32_t which = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) which |= static_cast<uint32_t>(c.at(i) >= least) << i;
            if (limit == 0) which = (1u << PER) - 1;
            for (; which; which &= which - 1) {
                const int i = __ffs(which) - 1;
                const uint32_t t = first + ((i / c.VEC) * SCAN_THREADS + threadIdx.x) * c.VEC + i % c.VEC;
                const uint64_t k = t < V ? logit_key(to_f32(z[t]), t) : 0;  // read again: the registers have no index
                if (k > limit) {
                    const int place = atomicAdd(&sh.n, 1);
                    if (place < MAX_M + SCAN_CAP) sh.buf[place] = k;
                }
            }
        }
        __syncthreads();
        const int total = sh.n;
        if (total > MAX_M + SCAN_CAP) {
            n = keep_best(sh, n, a.M);
            best_by_rounds<T, PER>(sh, c, first, V, a.M, n);
            n += a.M;
        } else {
            n = total;
        }
        if (total > MAX_M + SCAN_CAP || n > SCAN_HIGH || tau == 0) {
            n = keep_best(sh, n, a.M);
            if (n == a.M) tau = sh.buf[n - 1];
        }
    }
    __syncthreads();
    if (n > 0) n = keep_best(sh, n, a.M);
    const int64_t part = row * a.segs + seg;
    for (int i = threadIdx.x; i < a.M; i += SCAN_THREADS) a.seg_key[part * a.M + i] = i < n ? sh.buf[i] : 0;
    // the block's maximum and sum
    float bm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
    if (lane == 0) sh.red_m[warp] = bm;
    __syncthreads();
    for (int w = 0; w < SCAN_WARPS; ++w) bm = fmaxf(bm, sh.red_m[w]);
    if (m > -INFINITY && m < bm) s.scale(fast_exp2((m - bm) * LOG2E));
    s.over_warp();
    if (lane == 0) sh.red_s[warp] = make_float2(s.hi, s.lo);
    __syncthreads();
    if (threadIdx.x == 0) {
        Sum2 b{0.f, 0.f};
        for (int w = 0; w < SCAN_WARPS; ++w) b.add(sh.red_s[w].x, sh.red_s[w].y);
        a.seg_m[part] = bm;
        a.seg_s[part] = make_float2(b.hi, b.lo);
    }
}

struct JoinArgs {
    const float* seg_m;
    const float2* seg_s;
    const uint64_t* seg_key;
    const float* scores;      // [B, K]
    const uint8_t* finished;  // [B, K], nullable
    int32_t K, M, segs, V;
    int64_t pad, eos;         // eos < 0: none
    float* out_scores;        // [B, M]
    int64_t *out_tokens, *out_parents;
    uint8_t* out_finished;    // nullable
};

// Doubles as integers in the same order (no NaN comes here), and back.
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_ordered(uint64_t o) {
    return __longlong_as_double(static_cast<long long>((o >> 63) ? (o ^ 0x8000000000000000ull) : ~o));
}

// One block per item: a warp per beam adds its parts up and merges their
// lists; then all scores are computed, and the first warp merges the beams, a
// lane holding the beams l and l + 32.  A merge takes the largest head M times.
__global__ void __launch_bounds__(32 * JOIN_WARPS) beam_join_kernel(JoinArgs a) {
    extern __shared__ uint64_t dyn[];
    uint64_t* keys = dyn;                // [K, M] per beam, sorted down
    uint64_t* score = dyn + a.K * a.M;   // [K, M] as ordered integers, 0: no candidate
    uint64_t* lists = score + a.K * a.M;  // [JOIN_WARPS, segs, M]
    __shared__ double base[MAX_M];       // score - ln(sum)
    __shared__ float top[MAX_M];
    __shared__ float2 sums[MAX_M];
    __shared__ bool ended[MAX_M];
    const int64_t b = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_primary();
    for (int k = warp; k < a.K; k += JOIN_WARPS) {
        const int64_t row = b * a.K + k;
        const bool over = a.finished && a.finished[row];
        if (lane == 0) {
            ended[k] = over;
            top[k] = 0.f;
            sums[k] = make_float2(1.f, 0.f);
        }
        if (over) continue;
        uint64_t* list = lists + warp * a.segs * a.M;
        const uint64_t* from = a.seg_key + row * a.segs * a.M;
        for (int i = lane; i < a.segs * a.M; i += 32) list[i] = from[i];
        const bool have = lane < a.segs;
        const float m = have ? a.seg_m[row * a.segs + lane] : -INFINITY;
        const float2 ms = have ? a.seg_s[row * a.segs + lane] : make_float2(0.f, 0.f);
        float bm = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
        Sum2 s{ms.x, ms.y};
        if (!(m > -INFINITY))
            s = Sum2{0.f, 0.f};
        else if (m < bm)
            s.scale(fast_exp2((m - bm) * LOG2E));
        s.over_warp();
        if (lane == 0) {
            top[k] = bm;
            sums[k] = make_float2(s.hi, s.lo);
        }
        __syncwarp();
        int at = lane * a.M;
        const int stop = at + a.M;
        uint64_t head = have ? list[at] : 0;
        for (int r = 0; r < a.M; ++r) {
            const uint64_t best = warp_max(head);
            if (lane == 0) keys[k * a.M + r] = best;
            if (head == best && best) head = ++at < stop ? list[at] : 0;
        }
        __syncwarp();
    }
    __syncthreads();
    // one logarithm per beam, in FP64
    if (threadIdx.x < a.K) {
        float sc = a.scores[b * a.K + threadIdx.x];
        if (!(sc == sc)) sc = -INFINITY;
        const float2 v = sums[threadIdx.x];
        base[threadIdx.x] = ended[threadIdx.x]           ? static_cast<double>(sc)
                            : top[threadIdx.x] > -INFINITY ? sc - log(static_cast<double>(v.x) + v.y)
                                                           : -INFINITY;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.K * a.M; i += 32 * JOIN_WARPS) {
        const int k = i / a.M, r = i - k * a.M;
        uint64_t o = 0;
        if (ended[k]) {
            if (r < a.V) o = ordered(r == 0 ? base[k] : -INFINITY);
        } else if (const uint64_t key = keys[i]) {
            const float x = key_logit(key);
            o = ordered(x > -INFINITY ? base[k] + (static_cast<double>(x) - static_cast<double>(top[k])) : -INFINITY);
        }
        score[i] = o;
    }
    __syncthreads();
    if (warp != 0) return;
    int at0 = lane * a.M, at1 = (lane + 32) * a.M;
    const int stop0 = at0 + a.M, stop1 = at1 + a.M;
    uint64_t k0 = lane < a.K ? score[at0] : 0, k1 = lane + 32 < a.K ? score[at1] : 0;
    for (int r = 0; r < a.M; ++r) {
        const uint64_t best = warp_max(k1 > k0 ? k1 : k0);
        // the lowest beam among equals: the lanes' first beams before their second ones
        const unsigned has0 = __ballot_sync(0xFFFFFFFFu, k0 == best), has1 = __ballot_sync(0xFFFFFFFFu, k1 == best);
        const bool first = has0 != 0;
        if (lane == __ffs(first ? has0 : has1) - 1) {
            const int k = first ? lane : lane + 32, at = first ? at0 : at1;
            const int64_t token = ended[k] ? a.pad : static_cast<int64_t>(key_token(keys[at])), o = b * a.M + r;
            a.out_scores[o] = static_cast<float>(from_ordered(best));
            a.out_tokens[o] = token;
            a.out_parents[o] = k;
            if (a.out_finished) a.out_finished[o] = ended[k] || (a.eos >= 0 && token == a.eos);
            if (first)
                k0 = ++at0 < stop0 ? score[at0] : 0;
            else
                k1 = ++at1 < stop1 ? score[at1] : 0;
        }
    }
}

// ---------------------------------------------------------------- states

constexpr int MOVE_STATES = 24;  // tensors of one launch
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_PER = 4;      // vectors per thread

struct MoveState {
    const uint8_t* src;
    uint8_t* dst;
    int64_t s_row, d_row;                // bytes between rows
    int64_t s1, d1, s2, d2;              // bytes between the outer and the inner runs of a row
    uint32_t n2, run;                    // inner runs, vectors of a run
    uint32_t vectors, pieces;            // of a row
    uint32_t vec;                        // bytes of a vector: 16, 8, 4, 2 or 1
};

struct MoveArgs {
    MoveState st[MOVE_STATES];
    uint32_t end[MOVE_STATES];  // pieces before the next tensor, over all out rows
    int32_t n;
    const int64_t* parents;     // [items, out_beams]
    uint32_t out_beams, beams;
    unsigned* status;           // nullable
};

template <typename U>
__device__ __forceinline__ void move_piece(const MoveState& t, const uint8_t* src, uint8_t* dst, uint32_t first, bool ok) {
    U v[MOVE_PER];
    int64_t to[MOVE_PER];
#pragma unroll
    for (int q = 0; q < MOVE_PER; ++q) {
        const uint32_t i = first + q * MOVE_THREADS + threadIdx.x;
        to[q] = -1;
        if (i >= t.vectors) continue;
        const uint32_t o = i / t.run, off = i - o * t.run;
        const uint32_t i1 = o / t.n2, i2 = o - i1 * t.n2;
        const int64_t inner = static_cast<int64_t>(off) * sizeof(U);
        to[q] = i1 * t.d1 + i2 * t.d2 + inner;
        v[q] = U{};
        if (ok) v[q] = *reinterpret_cast<const U*>(src + i1 * t.s1 + i2 * t.s2 + inner);
    }
#pragma unroll
    for (int q = 0; q < MOVE_PER; ++q)
        if (to[q] >= 0) *reinterpret_cast<U*>(dst + to[q]) = v[q];
}

__global__ void __launch_bounds__(MOVE_THREADS) beam_move_kernel(const __grid_constant__ MoveArgs a) {
    int k = 0;
    while (blockIdx.x >= a.end[k]) ++k;
    const MoveState& t = a.st[k];
    const uint32_t piece = blockIdx.x - (k ? a.end[k - 1] : 0);
    const uint32_t out_row = piece / t.pieces, p = piece - out_row * t.pieces;
    const int64_t parent = a.parents[out_row];
    const bool ok = parent >= 0 && parent < a.beams;
    if (!ok && a.status && threadIdx.x == 0) atomicOr(a.status, STATUS_INDEX);
    const int64_t in_row = static_cast<int64_t>(out_row / a.out_beams) * a.beams + parent;
    const uint8_t* src = ok ? t.src + in_row * t.s_row : t.src;
    uint8_t* dst = t.dst + out_row * t.d_row;
    const uint32_t first = p * MOVE_THREADS * MOVE_PER;
    switch (t.vec) {
        case 16: move_piece<uint4>(t, src, dst, first, ok); break;
        case 8: move_piece<uint2>(t, src, dst, first, ok); break;
        case 4: move_piece<uint32_t>(t, src, dst, first, ok); break;
        case 2: move_piece<uint16_t>(t, src, dst, first, ok); break;
        default: move_piece<uint8_t>(t, src, dst, first, ok); break;
    }
}

// ---------------------------------------------------------------- host

lce_status_t beam_sizes(int64_t items, int64_t K, int64_t V, int64_t M) {
    if (items <= 0 || K <= 0 || V <= 0 || M <= 0) return LCE_ERR_INVALID_ARG;
    if (K > LCE_BEAM_MAX || M > LCE_BEAM_MAX || items > 65535 / K || V > INT32_MAX || M > K * V)
        return LCE_ERR_UNSUPPORTED;
    return LCE_OK;
}

struct BeamPlan {
    bool small;  // chunks of 2048 tokens, not 4096
    int32_t segs, per_seg;
    size_t off_m, off_key, total;
};

// A row's chunks and how they are shared out.  With few rows, chunks of 2048
// tokens spread the work over twice the blocks (one request of four beams over
// 32768 tokens: 64 blocks, not 32).
BeamPlan beam_plan(int64_t rows, int64_t V, int64_t M) {
    BeamPlan p;
    p.small = rows * ((V + 4095) / 4096) < SCAN_BLOCKS / 4;
    const int64_t chunk = p.small ? 2048 : 4096, chunks = (V + chunk - 1) / chunk;
    int64_t segs = rows < SCAN_BLOCKS ? SCAN_BLOCKS / rows : 1;  // one round of blocks
    if (segs > SCAN_SEGS_MAX) segs = SCAN_SEGS_MAX;
    if (segs > chunks) segs = chunks;
    p.per_seg = static_cast<int32_t>((chunks + segs - 1) / segs);
    p.segs = static_cast<int32_t>((chunks + p.per_seg - 1) / p.per_seg);
    const size_t n = static_cast<size_t>(rows) * p.segs;
    p.off_m = 1024 + n * 8;
    p.off_key = (p.off_m + n * 4 + 255) / 256 * 256;
    p.total = p.off_key + n * M * 8;
    return p;
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status_t lce_beam_workspace_size(int64_t items, int64_t beams, int64_t V, int64_t n_out, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = beam_sizes(items, beams, V, n_out);
    if (st == LCE_OK) *bytes = beam_plan(items * beams, V, n_out).total;
    return st;
}

lce_status_t lce_beam_select(int64_t items, int64_t beams, int64_t V, int64_t n_out, int dtype, const void* logits,
                             int64_t ld, const float* scores, const uint8_t* finished, int64_t pad_token,
                             int64_t eos_token, float* out_scores, int64_t* out_tokens, int64_t* out_parents,
                             uint8_t* out_finished, void* ws, size_t ws_bytes, lce_stream_t stream) {
    const lce_status_t st = beam_sizes(items, beams, V, n_out);
    if (st != LCE_OK) return st;
    if (!dtype_known(dtype) || !logits || !aligned_to(logits, dtype_bytes(dtype)) || ld < V) return LCE_ERR_INVALID_ARG;
    if (!scores || !out_scores || !out_tokens || !out_parents || !aligned_to(scores, 4) || !aligned_to(out_scores, 4) ||
        !aligned_to(out_tokens, 8) || !aligned_to(out_parents, 8))
        return LCE_ERR_INVALID_ARG;
    if (!ws || !aligned_to(ws, 256)) return LCE_ERR_INVALID_ARG;
    const BeamPlan p = beam_plan(items * beams, V, n_out);
    if (ws_bytes < p.total) return LCE_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(ws);
    float2* seg_s = reinterpret_cast<float2*>(w + 1024);
    float* seg_m = reinterpret_cast<float*>(w + p.off_m);
    uint64_t* seg_key = reinterpret_cast<uint64_t*>(w + p.off_key);
    const ScanArgs sa{logits, ld, finished, static_cast<int32_t>(V), static_cast<int32_t>(n_out), p.segs, p.per_seg,
                      seg_m, seg_s, seg_key};
    const dim3 grid(p.segs, static_cast<unsigned>(items * beams));
    const lce_status_t sc = with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        if (p.small)
            LCE_PROFILED(beam_scan_kernel<T, 8><<<grid, SCAN_THREADS, 0, s>>>(sa));
        else
            LCE_PROFILED(beam_scan_kernel<T, 16><<<grid, SCAN_THREADS, 0, s>>>(sa));
        return LCE_OK;
    });
    if (sc != LCE_OK) return sc;
    const JoinArgs ja{seg_m, seg_s, seg_key, scores, finished, static_cast<int32_t>(beams), static_cast<int32_t>(n_out),
                      p.segs, static_cast<int32_t>(V), pad_token, eos_token, out_scores, out_tokens, out_parents,
                      out_finished};
    const size_t smem = static_cast<size_t>(n_out) * 8 * (2 * beams + JOIN_WARPS * p.segs);
    if (smem > 40 * 1024 && cudaFuncSetAttribute(beam_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 JOIN_SMEM_MAX) != cudaSuccess)
        return LCE_ERR_CUDA;
    LCE_PROFILED(launch_after(beam_join_kernel, dim3(static_cast<unsigned>(items)), 32 * JOIN_WARPS, smem, s, ja));
    return LCE_OK;
}

lce_status_t lce_beam_reorder(int64_t items, int64_t beams, int64_t out_beams, const int64_t* parents,
                              const lce_beam_state_t* states, int64_t n_states, void* status, lce_stream_t stream) {
    if (items <= 0 || beams <= 0 || out_beams <= 0 || n_states < 0) return LCE_ERR_INVALID_ARG;
    if (items > INT32_MAX / beams || items > INT32_MAX / out_beams) return LCE_ERR_UNSUPPORTED;
    if (!parents || !aligned_to(parents, 8) || !aligned_to(status, 4) || (n_states && !states)) return LCE_ERR_INVALID_ARG;
    const int64_t rows = items * out_beams;
    for (int64_t i = 0; i < n_states; ++i) {
        const lce_beam_state_t& t = states[i];
        if (t.n1 < 0 || t.n2 < 0 || t.run_bytes < 0) return LCE_ERR_INVALID_ARG;
        if (!t.n1 || !t.n2 || !t.run_bytes) continue;
        if (!t.src || !t.dst) return LCE_ERR_INVALID_ARG;
        if (t.n1 > INT32_MAX || t.n2 > INT32_MAX || t.run_bytes > INT32_MAX || t.n1 * t.n2 > INT32_MAX / t.run_bytes)
            return LCE_ERR_UNSUPPORTED;  // a row of at most 2 GB
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    MoveArgs a;
    a.parents = parents;
    a.out_beams = static_cast<uint32_t>(out_beams);
    a.beams = static_cast<uint32_t>(beams);
    a.status = static_cast<unsigned*>(status);
    a.n = 0;
    uint64_t pieces = 0;
    auto flush = [&]() -> lce_status_t {
        if (a.n) LCE_PROFILED(beam_move_kernel<<<static_cast<unsigned>(pieces), MOVE_THREADS, 0, s>>>(a));
        a.n = 0;
        pieces = 0;
        return LCE_OK;
    };
    for (int64_t i = 0; i < n_states; ++i) {
        const lce_beam_state_t& t = states[i];
        if (!t.n1 || !t.n2 || !t.run_bytes) continue;
        // the widest vector that every address and length is a multiple of
        const uint64_t all = reinterpret_cast<uint64_t>(t.src) | reinterpret_cast<uint64_t>(t.dst) |
                             static_cast<uint64_t>(t.run_bytes) | static_cast<uint64_t>(t.src_row) |
                             static_cast<uint64_t>(t.dst_row) | static_cast<uint64_t>(t.src1) |
                             static_cast<uint64_t>(t.dst1) | static_cast<uint64_t>(t.src2) |
                             static_cast<uint64_t>(t.dst2) | 16u;
        const uint32_t vec = static_cast<uint32_t>(all & (~all + 1));
        MoveState m;
        m.src = static_cast<const uint8_t*>(t.src);
        m.dst = static_cast<uint8_t*>(t.dst);
        m.s_row = t.src_row;
        m.d_row = t.dst_row;
        m.s1 = t.src1;
        m.d1 = t.dst1;
        m.s2 = t.src2;
        m.d2 = t.dst2;
        m.vec = vec;
        m.run = static_cast<uint32_t>(t.run_bytes / vec);
        m.n2 = static_cast<uint32_t>(t.n2);
        m.vectors = static_cast<uint32_t>(t.n1 * t.n2 * m.run);
        m.pieces = (m.vectors + MOVE_THREADS * MOVE_PER - 1) / (MOVE_THREADS * MOVE_PER);
        const uint64_t more = static_cast<uint64_t>(m.pieces) * rows;
        if (more > INT32_MAX) return LCE_ERR_UNSUPPORTED;
        if (a.n == MOVE_STATES || pieces + more > INT32_MAX) {
            const lce_status_t st = flush();
            if (st != LCE_OK) return st;
        }
        pieces += more;
        a.st[a.n] = m;
        a.end[a.n++] = static_cast<uint32_t>(pieces);
    }
    return flush();
}

}  // extern "C"
