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
constexpr int SCAN_PER = 32;                          // elements of a chunk per thread
constexpr int SCAN_CHUNK = SCAN_THREADS * SCAN_PER;   // 8192
constexpr int SCAN_CAP = 1024;                        // keys the buffer holds beside the list
constexpr int SCAN_HIGH = 256;                        // keys that start a merge
constexpr int SCAN_SEGS_MAX = 32;                     // parts of a row (a lane each in the join)
constexpr int64_t SCAN_BLOCKS = 608;                  // blocks that fill the GPU
constexpr int MAX_M = LCE_BEAM_MAX;

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

struct ScanArgs {
    const void* z;
    int64_t ld;
    const uint8_t* finished;  // [rows], nullable
    int32_t V, M, segs, per_seg;  // per_seg: chunks of a segment
    float* seg_m;      // [rows, segs]
    double* seg_s;
    uint64_t* seg_key;  // [rows, segs, M], sorted down; 0: no candidate
};

struct ScanShared {
    uint64_t buf[MAX_M + SCAN_CAP];  // the list's keys, then the new ones
    uint64_t lane_key[SCAN_THREADS];
    uint64_t tau;
    double red_s[SCAN_THREADS / 32];
    float red_m[SCAN_THREADS / 32];
    uint64_t red_k[SCAN_THREADS / 32];
    int n;
};

// Keeps the M largest of buf[0..n) at its front, sorted down; returns how many
// there are.  A key's place is the number of larger ones.
__device__ int keep_best(ScanShared& sh, int n, int M) {
    constexpr int PER = (MAX_M + SCAN_CAP + SCAN_THREADS - 1) / SCAN_THREADS;
    uint64_t key[PER];
    int rank[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int i = q * SCAN_THREADS + threadIdx.x;
        rank[q] = M;
        if (q * SCAN_THREADS < n && i < n) {
            key[q] = sh.buf[i];
            int r = 0;
            for (int j = 0; j < n; ++j) r += sh.buf[j] > key[q];
            rank[q] = r;
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < PER; ++q)
        if (rank[q] < M) sh.buf[rank[q]] = key[q];
    __syncthreads();
    return n < M ? n : M;
}

__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = u > v ? u : v;
    }
    return v;
}

// One thread's elements of a chunk: vector u holds the tokens
// first + (u * SCAN_THREADS + thread) * VEC + j.  The places do not depend on
// the alignment, so equal rows give equal sums.
template <typename T>
struct Chunk {
    static constexpr int VEC = vec16<T>();
    static constexpr int N = SCAN_PER / VEC;
    Vec<T, VEC> v[N];

    static __device__ __forceinline__ uint32_t token(uint32_t first, int i) {
        return first + ((i / VEC) * SCAN_THREADS + threadIdx.x) * VEC + i % VEC;
    }
    __device__ __forceinline__ float at(int i) const { return v[i / VEC].f(i % VEC); }
    __device__ __forceinline__ void load(const T* row, uint32_t first, uint32_t V, bool vec) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t t = token(first, u * VEC);
            if (vec && t + VEC <= V) {
                v[u] = *reinterpret_cast<const Vec<T, VEC>*>(row + t);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[u].v[j] = t + j < V ? row[t + j] : from_f32<T>(-INFINITY);
            }
        }
    }
};

// The M best of the chunk's own elements by rounds of a block-wide maximum,
// appended to the buffer: for chunks whose candidates overflow it.
template <typename T>
__device__ void best_by_rounds(ScanShared& sh, const Chunk<T>& c, uint32_t first, uint32_t V, int M, int n) {
    uint64_t below = ~0ull;
    for (int r = 0; r < M; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < SCAN_PER; ++i) {
            const uint32_t t = Chunk<T>::token(first, i);
            const uint64_t k = t < V ? logit_key(c.at(i), t) : 0;
            if (k < below && k > best) best = k;
        }
        best = warp_max(best);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh.red_k[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int w = 0; w < SCAN_THREADS / 32; ++w) best = sh.red_k[w] > best ? sh.red_k[w] : best;
        if (threadIdx.x == 0) sh.buf[n + r] = best;
        below = best;
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(SCAN_THREADS) beam_scan_kernel(ScanArgs a) {
    __shared__ ScanShared sh;
    const int64_t row = blockIdx.y;
    const int seg = blockIdx.x;
    if (a.finished && a.finished[row]) return;  // the join does not read its parts
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    const bool vec = aligned_dev(z);
    const uint32_t V = static_cast<uint32_t>(a.V);
    const uint64_t begin = static_cast<uint64_t>(seg) * a.per_seg * SCAN_CHUNK;
    uint64_t end = begin + static_cast<uint64_t>(a.per_seg) * SCAN_CHUNK;
    if (end > V) end = V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;        // keys in the buffer (all threads agree)
    uint64_t tau = 0;  // the M-th best so far, 0 while there are fewer
    float m = -INFINITY;
    double s = 0.0;
    for (uint64_t first64 = begin; first64 < end; first64 += SCAN_CHUNK) {
        const uint32_t first = static_cast<uint32_t>(first64);
        Chunk<T> c;
        c.load(z, first, V, vec);
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < SCAN_PER; ++i) mx = fmaxf(mx, clean(c.at(i)));
        const float m2 = fmaxf(m, mx);
        if (m2 > -INFINITY) {
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < SCAN_PER; ++i) part += exp2f((clean(c.at(i)) - m2) * LOG2E);
            s = s * static_cast<double>(exp2f((m - m2) * LOG2E)) + static_cast<double>(part);
            m = m2;
        }
        // candidates: in a part's first chunk those not below the M-th largest of the
        // threads' maxima, later those above the M-th best so far (a later
        // token loses against an equal one)
        uint64_t limit = tau;
        if (tau == 0) {
            uint64_t k = 0;
#pragma unroll
            for (int i = 0; i < SCAN_PER; ++i) {
                const uint32_t t = Chunk<T>::token(first, i);
                const uint64_t q = t < V ? logit_key(c.at(i), t) : 0;
                k = q > k ? q : k;
            }
            sh.lane_key[threadIdx.x] = k;
            if (threadIdx.x == 0) sh.tau = 1;  // fewer than M threads with elements: all pass
            __syncthreads();
            int rank = 0;
            for (int j = 0; j < SCAN_THREADS; ++j) rank += sh.lane_key[j] > k;
            if (rank == a.M - 1 && k) sh.tau = k;
            __syncthreads();
            limit = sh.tau - 1;
        }
        if (threadIdx.x == 0) sh.n = n;
        __syncthreads();
        if (logit_key(mx, 0) > limit) {
#pragma unroll
            for (int i = 0; i < SCAN_PER; ++i) {
                const uint32_t t = Chunk<T>::token(first, i);
                const uint64_t k = t < V ? logit_key(c.at(i), t) : 0;
                if (k > limit) {
                    const int at = atomicAdd(&sh.n, 1);
                    if (at < MAX_M + SCAN_CAP) sh.buf[at] = k;
                }
            }
        }
        __syncthreads();
        const int total = sh.n;
        __syncthreads();
        if (total > MAX_M + SCAN_CAP) {
            n = keep_best(sh, n, a.M);
            best_by_rounds<T>(sh, c, first, V, a.M, n);
            n += a.M;
        } else {
            n = total;
        }
        if (n > SCAN_HIGH || tau == 0) {
            n = keep_best(sh, n, a.M);
            if (n == a.M) tau = sh.buf[n - 1];
        }
    }
    n = keep_best(sh, n, a.M);
    const int64_t part = row * a.segs + seg;
    for (int i = threadIdx.x; i < a.M; i += SCAN_THREADS) a.seg_key[part * a.M + i] = i < n ? sh.buf[i] : 0;
    // the block's maximum and sum
    float bm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
    if (lane == 0) sh.red_m[warp] = bm;
    __syncthreads();
    for (int w = 0; w < SCAN_THREADS / 32; ++w) bm = fmaxf(bm, sh.red_m[w]);
    double bs = m > -INFINITY ? s * static_cast<double>(exp2f((m - bm) * LOG2E)) : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bs += __shfl_xor_sync(0xFFFFFFFFu, bs, o);
    if (lane == 0) sh.red_s[warp] = bs;
    __syncthreads();
    if (threadIdx.x == 0) {
        bs = 0.0;
        for (int w = 0; w < SCAN_THREADS / 32; ++w) bs += sh.red_s[w];
        a.seg_m[part] = bm;
        a.seg_s[part] = bs;
    }
}

struct JoinArgs {
    const float* seg_m;
    const double* seg_s;
    const uint64_t* seg_key;
    const float* scores;      // [B, K]
    const uint8_t* finished;  // [B, K], nullable
    int32_t K, M, segs, V;
    int64_t pad, eos;         // eos < 0: none
    float* out_scores;        // [B, M]
    int64_t *out_tokens, *out_parents;
    uint8_t* out_finished;    // nullable
};

// Doubles as integers in the same order (no NaN comes here).
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}

// One block per item: a warp per beam adds its parts up and merges their
// lists, then the first warp merges the beams, a lane holding the beams l and
// l + 32.
__global__ void __launch_bounds__(256) beam_join_kernel(JoinArgs a) {
    extern __shared__ uint64_t keys[];  // [K, M] per beam, sorted down
    __shared__ double base[MAX_M];      // score - ln(sum)
    __shared__ float top[MAX_M];
    const int64_t b = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int k = warp; k < a.K; k += 8) {
        const int64_t row = b * a.K + k;
        float score = a.scores[row];
        if (!(score == score)) score = -INFINITY;
        if (a.finished && a.finished[row]) {
            if (lane == 0) base[k] = score;
            continue;
        }
        const int64_t part = row * a.segs + lane;
        const bool have = lane < a.segs;
        const float m = have ? a.seg_m[part] : -INFINITY;
        float bm = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
        double s = have && m > -INFINITY ? a.seg_s[part] * exp(static_cast<double>(m) - static_cast<double>(bm)) : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) {
            base[k] = bm > -INFINITY ? static_cast<double>(score) - log(s) : -INFINITY;
            top[k] = bm;
        }
        // each lane holds the head of its part's list; the largest leaves
        int at = 0;
        uint64_t head = have ? a.seg_key[part * a.M] : 0;
        for (int r = 0; r < a.M; ++r) {
            const uint64_t best = warp_max(head);
            if (lane == 0) keys[k * a.M + r] = best;
            if (head == best && best) {
                ++at;
                head = at < a.M ? a.seg_key[part * a.M + at] : 0;
            }
        }
    }
    __syncthreads();
    if (warp != 0) return;
    // (score as an integer, 0 when the beam has no more candidates)
    auto candidate = [&](int k, int r, double* score, int64_t* token) -> uint64_t {
        if (k >= a.K || r >= a.M) return 0;
        if (a.finished && a.finished[b * a.K + k]) {
            if (r >= a.V) return 0;
            *score = r == 0 ? base[k] : -INFINITY;
            *token = a.pad;
            return ordered(*score);
        }
        const uint64_t key = keys[k * a.M + r];
        if (!key) return 0;
        const float x = key_logit(key);
        *score = x > -INFINITY ? base[k] + (static_cast<double>(x) - static_cast<double>(top[k])) : -INFINITY;
        *token = key_token(key);
        return ordered(*score);
    };
    int at0 = 0, at1 = 0;
    double s0 = 0.0, s1 = 0.0;
    int64_t t0 = 0, t1 = 0;
    uint64_t k0 = candidate(lane, 0, &s0, &t0), k1 = candidate(lane + 32, 0, &s1, &t1);
    for (int r = 0; r < a.M; ++r) {
        const uint64_t mine = k1 > k0 ? k1 : k0;
        const uint64_t best = warp_max(mine);
        // the lowest beam among equals: the lanes' first beams before their second ones
        const unsigned has0 = __ballot_sync(0xFFFFFFFFu, k0 == best), has1 = __ballot_sync(0xFFFFFFFFu, k1 == best);
        const bool first = has0 != 0;
        const int winner = __ffs(first ? has0 : has1) - 1;
        if (lane == winner) {
            const int k = first ? lane : lane + 32;
            const int64_t token = first ? t0 : t1, o = b * a.M + r;
            a.out_scores[o] = static_cast<float>(first ? s0 : s1);
            a.out_tokens[o] = token;
            a.out_parents[o] = k;
            if (a.out_finished)
                a.out_finished[o] = (a.finished && a.finished[b * a.K + k]) || (a.eos >= 0 && token == a.eos);
            if (first)
                k0 = candidate(lane, ++at0, &s0, &t0);
            else
                k1 = candidate(lane + 32, ++at1, &s1, &t1);
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
    int32_t segs, per_seg;
    size_t off_s, off_m, off_key, total;
};

BeamPlan beam_plan(int64_t rows, int64_t V, int64_t M) {
    BeamPlan p;
    const int64_t chunks = (V + SCAN_CHUNK - 1) / SCAN_CHUNK;
    int64_t segs = (SCAN_BLOCKS + rows - 1) / rows;
    if (segs > SCAN_SEGS_MAX) segs = SCAN_SEGS_MAX;
    if (segs > chunks) segs = chunks;
    p.per_seg = static_cast<int32_t>((chunks + segs - 1) / segs);
    p.segs = static_cast<int32_t>((chunks + p.per_seg - 1) / p.per_seg);
    const size_t n = static_cast<size_t>(rows) * p.segs;
    p.off_s = 1024;
    p.off_m = p.off_s + n * 8;
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
    float* seg_m = reinterpret_cast<float*>(w + p.off_m);
    double* seg_s = reinterpret_cast<double*>(w + p.off_s);
    uint64_t* seg_key = reinterpret_cast<uint64_t*>(w + p.off_key);
    const ScanArgs sa{logits, ld, finished, static_cast<int32_t>(V), static_cast<int32_t>(n_out), p.segs, p.per_seg,
                      seg_m, seg_s, seg_key};
    const dim3 grid(p.segs, static_cast<unsigned>(items * beams));
    const lce_status_t sc = with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        LCE_PROFILED(beam_scan_kernel<T><<<grid, SCAN_THREADS, 0, s>>>(sa));
        return LCE_OK;
    });
    if (sc != LCE_OK) return sc;
    const JoinArgs ja{seg_m, seg_s, seg_key, scores, finished, static_cast<int32_t>(beams), static_cast<int32_t>(n_out),
                      p.segs, static_cast<int32_t>(V), pad_token, eos_token, out_scores, out_tokens, out_parents,
                      out_finished};
    LCE_PROFILED(beam_join_kernel<<<static_cast<unsigned>(items), 256, static_cast<size_t>(beams) * n_out * 8, s>>>(ja));
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
