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
//
// Where rows are many the scan issues in 56 of 100 cycles, 26 instructions per
// logit, with a third of the warps: 461 unfinished rows of 50257 fp32 logits
// take 36 us, 2.6 TB/s; what its warps wait for most are the barriers between
// chunks.  The join of 64 items takes 8.6 us.  A call of one item is two
// latencies, 5 to 6 and 6 to 8 us one by one and cold.  The copy of the states
// is bound by memory: 16 states of 32 rows of 3 MB take 361 us.
#include <float.h>

#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int SCAN_THREADS = 256;
constexpr int SCAN_WARPS = SCAN_THREADS / 32;
constexpr int SCAN_CAP = 448;                         // keys the buffer holds beside the list
constexpr int SCAN_MORE = 16;                         // keys beside the list that start a merge
constexpr int SCAN_STAGES = 3;                        // chunks in shared memory
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

// A sum in two floats: the exact error of each addition of the first, by
// Knuth's TwoSum, goes to the second.  FP64 adds run at 1/64 of the rate here.
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
    int n;     // keys in the buffer, or more where they overflowed it
    int kept;  // of them from before the last chunk with candidates
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
#pragma unroll 4
            for (int j = 0; j + 1 < n; j += 2) {
                const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(sh.buf + j);
                r += (k.x > key[q]) + (k.y > key[q]);
            }
            if (n & 1) r += sh.buf[n - 1] > key[q];
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

// A chunk of a row in shared memory: SCAN_THREADS x W words of 32 bits.  Word w
// of a thread is the chunk's word w * SCAN_THREADS + thread: one fp32 logit, or
// two neighbours in 16 bits.  A row that starts `shift` bytes past a 16-byte
// boundary is copied with what lies before it, so the words start at `shift`;
// the places do not depend on it, and equal rows give equal sums.
template <typename T, int W>
struct Chunk {
    static constexpr int PW = 4 / sizeof(T);                 // logits of a word
    static constexpr int PER = W * PW;                       // of a thread
    static constexpr uint32_t TOKENS = SCAN_THREADS * PER;
    static constexpr int BYTES = SCAN_THREADS * W * 4 + 16;  // of a stage
    const char* base;  // the stage, past the shift
    uint32_t first, V;

    __device__ __forceinline__ uint32_t token(int e) const {
        return first + ((e / PW) * SCAN_THREADS + threadIdx.x) * PW + e % PW;
    }
    // Logit e of the thread; its token is below V.
    __device__ __forceinline__ float at(int e) const { return to_f32(*reinterpret_cast<const T*>(base + (token(e) - first) * sizeof(T))); }
    __device__ __forceinline__ uint32_t word(int w) const {
        const char* p = base + (w * SCAN_THREADS + threadIdx.x) * 4;
        if (sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(base) & 2)) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p - 2);
            return __funnelshift_r(q[0], q[1], 16);
        }
        return *reinterpret_cast<const uint32_t*>(p);
    }
    // The thread's logits as pairs; -inf past the row's end.
    __device__ __forceinline__ void read(F2 (&x)[PER / 2]) const {
        const bool tail = first + TOKENS > V;
#pragma unroll
        for (int p = 0; p < PER / 2; ++p) {
            if constexpr (sizeof(T) == 4) {
                x[p] = f2(__uint_as_float(word(2 * p)), __uint_as_float(word(2 * p + 1)));
            } else {
                const uint32_t w = word(p);
                T v[2];
                __builtin_memcpy(v, &w, 4);
                x[p] = pair_of(v);
            }
            if (tail) x[p] = f2(token(2 * p) < V ? lo(x[p]) : -INFINITY, token(2 * p + 1) < V ? hi(x[p]) : -INFINITY);
        }
    }
    // Starts the copies of the chunk that begins at token `from` into a stage.
    // Only whole 16-byte units inside the row are copied as such.
    static __device__ __forceinline__ void copy(char* stage, const T* row, uint32_t from, uint32_t V) {
        const char* begin = reinterpret_cast<const char*>(row);
        const char* end = begin + static_cast<size_t>(V) * sizeof(T);
        const char* src = begin + static_cast<size_t>(from) * sizeof(T);
        src -= reinterpret_cast<uintptr_t>(src) & 15u;
        if (src >= begin && src + BYTES <= end) {  // inside the row
            const char* p = src + threadIdx.x * 16;
            char* to = stage + threadIdx.x * 16;
#pragma unroll
            for (int u = 0; u < BYTES / 16 / SCAN_THREADS; ++u)
                copy_async<16>(to + u * SCAN_THREADS * 16, p + u * SCAN_THREADS * 16);
            if (threadIdx.x == 0) copy_async<16>(stage + BYTES - 16, src + BYTES - 16);
            return;
        }
#pragma unroll
        for (int u = 0; u < (BYTES / 16 + SCAN_THREADS - 1) / SCAN_THREADS; ++u) {
            const int at = u * SCAN_THREADS + threadIdx.x;
            const char* p = src + at * 16;
            if (at >= BYTES / 16 || p >= end) continue;
            if (p >= begin && p + 16 <= end) {
                copy_async<16>(stage + at * 16, p);
            } else {
#pragma unroll
                for (int j = 0; j < 16; j += sizeof(T))
                    if (p + j >= begin && p + j < end)
                        *reinterpret_cast<T*>(stage + at * 16 + j) = *reinterpret_cast<const T*>(p + j);
            }
        }
    }
};

// The sum of e^(x - m).
template <int PAIRS>
__device__ __forceinline__ float sum_exp(const F2 (&x)[PAIRS], float m) {
    F2 s0 = f2(0.f), s1 = f2(0.f);
    const F2 m2 = f2(-m), l2 = f2(LOG2E);
#pragma unroll
    for (int p = 0; p < PAIRS; p += 2) {
        const F2 a = mul2(add2(x[p], m2), l2), b = mul2(add2(x[p + 1], m2), l2);
        s0 = add2(s0, f2(fast_exp2(lo(a)), fast_exp2(hi(a))));
        s1 = add2(s1, f2(fast_exp2(lo(b)), fast_exp2(hi(b))));
    }
    s0 = add2(s0, s1);
    const float s = lo(s0) + hi(s0);
    if (s < INFINITY) return s;
    float c = 0.f;  // a NaN or an infinity among them
#pragma unroll
    for (int p = 0; p < PAIRS; ++p)
        c += fast_exp2((clean(lo(x[p])) - m) * LOG2E) + fast_exp2((clean(hi(x[p])) - m) * LOG2E);
    return c;
}

// The M best of the thread's chunk by rounds of a block-wide maximum, appended
// to the buffer: for chunks whose candidates overflow it.
template <typename T, int W>
__device__ void best_by_rounds(ScanShared& sh, const Chunk<T, W>& c, int M, int n) {
    uint64_t below = ~0ull;
    for (int r = 0; r < M; ++r) {
        uint64_t best = 0;
        for (int e = 0; e < c.PER; ++e) {
            const uint32_t t = c.token(e);
            const uint64_t k = t < c.V ? logit_key(c.at(e), t) : 0;
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

// A part of a row.  Chunks are copied two ahead; a chunk's candidates go to the
// buffer as they are found, and are looked at when the next chunk is there
// (while the chunk they came from still is: if they overflowed, it is gone
// through again).  A chunk costs a barrier, two with candidates in the one
// before it.
template <typename T, int W>
__global__ void __launch_bounds__(SCAN_THREADS, 4) beam_scan_kernel(ScanArgs a) {
    using C = Chunk<T, W>;
    extern __shared__ __align__(16) char ring[];  // [SCAN_STAGES, BYTES]
    __shared__ ScanShared sh;
    launch_dependents();
    const int64_t row = blockIdx.y;
    const int seg = blockIdx.x;
    if (a.finished && a.finished[row]) return;  // the join does not read its parts
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) & 15u);
    const uint32_t V = static_cast<uint32_t>(a.V);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = static_cast<int64_t>(seg) * a.per_seg;
    int64_t left = (V + C::TOKENS - 1) / C::TOKENS - c0;
    const int chunks = static_cast<int>(left < a.per_seg ? left : a.per_seg);
    auto begin_copy = [&](int c) {
        if (c < chunks) C::copy(ring + (c % SCAN_STAGES) * C::BYTES, z, static_cast<uint32_t>((c0 + c) * C::TOKENS), V);
        copy_async_commit();
    };
    auto chunk = [&](int c) {
        return C{ring + (c % SCAN_STAGES) * C::BYTES + shift, static_cast<uint32_t>((c0 + c) * C::TOKENS), V};
    };
    int n = 0;         // keys in the buffer (all threads agree)
    uint64_t tau = 0;  // the M-th best so far, 0 while there are fewer
    float m = -INFINITY;
    Sum2 s{0.f, 0.f};
    if (threadIdx.x == 0) sh.n = sh.kept = 0;
#pragma unroll
    for (int k = 0; k < SCAN_STAGES - 1; ++k) begin_copy(k);
    bool pushed = false;
    for (int c = 0; c <= chunks; ++c) {  // the last turn only looks at the last chunk's candidates
        copy_async_wait<SCAN_STAGES - 2>();
        if (__syncthreads_or(pushed)) {
            n = sh.n;
            if (n > MAX_M + SCAN_CAP) {
                n = keep_best(sh, sh.kept, a.M);
                best_by_rounds<T, W>(sh, chunk(c - 1), a.M, n);
                n = keep_best(sh, n + a.M, a.M);
            } else if (n > a.M + SCAN_MORE || tau == 0) {
                n = keep_best(sh, n, a.M);
            }
            if (n == a.M) tau = sh.buf[n - 1] > tau ? sh.buf[n - 1] : tau;
            if (threadIdx.x == 0) sh.kept = n;
            __syncthreads();
        }
        if (c == chunks) break;
        begin_copy(c + SCAN_STAGES - 1);
        const C k = chunk(c);
        F2 x[C::PER / 2];
        k.read(x);
        float raw = lo(x[0]);
#pragma unroll
        for (int p = 0; p < C::PER / 2; ++p) raw = fmaxf(raw, fmaxf(lo(x[p]), hi(x[p])));
        const float mx = clean(raw), m2 = fmaxf(m, mx);
        if (m2 > -INFINITY) {
            if (m2 > m) s.scale(fast_exp2((m - m2) * LOG2E));  // of nothing at first
            s.add(sum_exp(x, m2));
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
                for (int e = C::PER - 1; e >= 0; --e) at = (e & 1 ? hi(x[e / 2]) : lo(x[e / 2])) >= raw ? e : at;
            const uint32_t t = k.token(at);
            uint64_t below = t < V ? logit_key(mx, t) : 0, rth = 0;
            for (int i = 0; i < (a.M + SCAN_WARPS - 1) / SCAN_WARPS; ++i) {
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
        pushed = logit_key(mx, 0) > limit;
        if (pushed) {
            // what is not below the least candidate: a NaN stays, for its key to decide as -inf
            const float least = key_logit(limit + 1);
            uint32_t which = 0;
#pragma unroll
            for (int e = 0; e < C::PER; ++e)
                which |= static_cast<uint32_t>(!((e & 1 ? hi(x[e / 2]) : lo(x[e / 2])) < least)) << e;
            if (limit == 0) which = static_cast<uint32_t>((1ull << C::PER) - 1);
            for (; which; which &= which - 1) {
                const int e = __ffs(which) - 1;
                const uint32_t t = k.token(e);
                const uint64_t key = t < V ? logit_key(k.at(e), t) : 0;
                if (key > limit) {
                    const int place = atomicAdd(&sh.n, 1);
                    if (place < MAX_M + SCAN_CAP) sh.buf[place] = key;
                }
            }
        }
    }
    if (n > a.M) n = keep_best(sh, n, a.M);
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
// lists; then all scores are computed, and the beams are merged: by counting
// where a thread can take each candidate, else by the first warp, a lane
// holding the beams l and l + 32.  A merge takes the largest head M times.
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
        // (a finished beam's parts were not written; what is read there is not used)
        uint64_t* list = a.segs > 1 ? lists + warp * a.segs * a.M : keys + k * a.M;
        const uint64_t* from = a.seg_key + row * a.segs * a.M;
        for (int i = lane; i < a.segs * a.M; i += 32) list[i] = from[i];
        const bool have = lane < a.segs;
        const float m = have ? a.seg_m[row * a.segs + lane] : -INFINITY;
        const float2 ms = have ? a.seg_s[row * a.segs + lane] : make_float2(0.f, 0.f);
        const bool over = a.finished && a.finished[row];
        if (lane == 0) {
            ended[k] = over;
            top[k] = 0.f;
            sums[k] = make_float2(1.f, 0.f);
        }
        if (over) continue;
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
        if (a.segs == 1) continue;  // the part's list is the beam's
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
    const int all = a.K * a.M;
    for (int i = threadIdx.x; i < all; i += 32 * JOIN_WARPS) {
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
    // candidate i of the item as its result r
    auto write = [&](int i, int r) {
        const int k = i / a.M;
        const int64_t token = ended[k] ? a.pad : static_cast<int64_t>(key_token(keys[i])), o = b * a.M + r;
        a.out_scores[o] = static_cast<float>(from_ordered(score[i]));
        a.out_tokens[o] = token;
        a.out_parents[o] = k;
        if (a.out_finished) a.out_finished[o] = ended[k] || (a.eos >= 0 && token == a.eos);
    };
    if (all <= 32 * JOIN_WARPS) {
        // a thread per candidate: its place is the number of better ones, among equals those before it
        const int i = threadIdx.x;
        if (i < all && score[i]) {
            const uint64_t mine = score[i];
            int r = 0;
#pragma unroll 8
            for (int j = 0; j < all; ++j) r += score[j] > mine || (score[j] == mine && j < i);
            if (r < a.M) write(i, r);
        }
        return;
    }
    if (warp != 0) return;
    int at0 = lane * a.M, at1 = (lane + 32) * a.M;
    const int stop0 = at0 + a.M, stop1 = at1 + a.M;
    uint64_t k0 = lane < a.K ? score[at0] : 0, k1 = lane + 32 < a.K ? score[at1] : 0;
    int mine[2] = {0, 0};  // results `lane` and `lane + 32`
    for (int r = 0; r < a.M; ++r) {
        const uint64_t best = warp_max(k1 > k0 ? k1 : k0);
        // the lowest beam among equals: the lanes' first beams before their second ones
        const unsigned has0 = __ballot_sync(0xFFFFFFFFu, k0 == best), has1 = __ballot_sync(0xFFFFFFFFu, k1 == best);
        const int winner = __ffs(has0 ? has0 : has1) - 1;
        const int at = __shfl_sync(0xFFFFFFFFu, has0 ? at0 : at1, winner);
        if (lane == (r & 31)) mine[r >> 5] = at;
        if (lane == winner) {
            if (has0)
                k0 = ++at0 < stop0 ? score[at0] : 0;
            else
                k1 = ++at1 < stop1 ? score[at1] : 0;
        }
    }
    if (lane < a.M) write(mine[0], lane);
    if (lane + 32 < a.M) write(mine[1], lane + 32);
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
    bool small;  // chunks of 4 KB, not 16 KB
    int32_t segs, per_seg;
    size_t off_m, off_key, total;
};

// A row's chunks and how they are shared out: one round of blocks where there
// are rows for it.  With few rows, chunks of 4 KB spread the work over four
// times the blocks (one request of four bf16 beams over 32768 tokens: 64
// blocks, not 16).
BeamPlan beam_plan(int64_t rows, int64_t V, int64_t M, int dtype) {
    BeamPlan p;
    const int64_t per_kb = 1024 / static_cast<int64_t>(dtype_bytes(dtype));
    p.small = rows * ((V + 16 * per_kb - 1) / (16 * per_kb)) < SCAN_BLOCKS / 4;
    const int64_t chunk = (p.small ? 4 : 16) * per_kb, chunks = (V + chunk - 1) / chunk;
    int64_t segs = rows < SCAN_BLOCKS ? SCAN_BLOCKS / rows : 1;
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

template <typename T, int W>
lce_status_t beam_scan(const ScanArgs& a, int64_t rows, cudaStream_t s) {
    constexpr int smem = SCAN_STAGES * Chunk<T, W>::BYTES;
    if (smem > 40 * 1024 && cudaFuncSetAttribute(beam_scan_kernel<T, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 smem) != cudaSuccess)
        return LCE_ERR_CUDA;
    const dim3 grid(a.segs, static_cast<unsigned>(rows));
    LCE_PROFILED(beam_scan_kernel<T, W><<<grid, SCAN_THREADS, smem, s>>>(a));
    return LCE_OK;
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status_t lce_beam_workspace_size(int64_t items, int64_t beams, int64_t V, int64_t n_out, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = beam_sizes(items, beams, V, n_out);
    if (st == LCE_OK) {  // of either type
        const size_t a = beam_plan(items * beams, V, n_out, LCE_BF16).total, b = beam_plan(items * beams, V, n_out, LCE_F32).total;
        *bytes = a > b ? a : b;
    }
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
    const BeamPlan p = beam_plan(items * beams, V, n_out, dtype);
    if (ws_bytes < p.total) return LCE_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(ws);
    float2* seg_s = reinterpret_cast<float2*>(w + 1024);
    float* seg_m = reinterpret_cast<float*>(w + p.off_m);
    uint64_t* seg_key = reinterpret_cast<uint64_t*>(w + p.off_key);
    const ScanArgs sa{logits, ld, finished, static_cast<int32_t>(V), static_cast<int32_t>(n_out), p.segs, p.per_seg,
                      seg_m, seg_s, seg_key};
    const lce_status_t sc = with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        return p.small ? beam_scan<T, 4>(sa, items * beams, s) : beam_scan<T, 16>(sa, items * beams, s);
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
    int n = 0;
    uint64_t pieces = 0;
    auto flush = [&]() -> lce_status_t {
        if (n) LCE_PROFILED(beam_move_kernel<<<static_cast<unsigned>(pieces), MOVE_THREADS, 0, s>>>(a));
        n = 0;
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
        if (n == MOVE_STATES || pieces + more > INT32_MAX) {
            const lce_status_t st = flush();
            if (st != LCE_OK) return st;
        }
        pieces += more;
        a.st[n] = m;
        a.end[n++] = static_cast<uint32_t>(pieces);
    }
    return flush();
}

}  // extern "C"
