// Embedding lookup with scaling, and its gradient.
//
//   y_i = c W[t_i],   dW[v] = c sum_{i: t_i = v} dy_i
//
// Both are bound by the bytes of the rows.  The gradient adds the rows of a
// token in the order in which they come: the tokens are sorted (lce_sort.cuh),
// so no float is added by an atomic and equal calls give equal bits.  Sums are
// FP32, scaled and rounded once.
#include "lce_sort.cuh"

namespace lce {
namespace {

constexpr int64_t EMB_MAX_H = LCE_NORM_MAX_H;
constexpr int EMB_DIGIT_BITS = 10;

template <typename T>
struct EmbFwd {
    const void* tokens;
    bool idx64;
    const T* w;
    int64_t ldw, N, V;
    int64_t padding;
    float scale;
    T* y;
    int64_t ldy;
    unsigned* status;  // nullable
    int32_t H;
    Deal deal;         // of the rows' vectors
};

__device__ __forceinline__ int64_t token_at(const void* tokens, bool idx64, int64_t i) {
    return idx64 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// Wide rows: a warp per U vectors of each lane of a token's row, so that the
// token is looked up once for them.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) emb_fwd_wide(EmbFwd<T> a) {
    using V = Vec<T, VEC>;
    wait_for_primary();
    const int n = a.H / VEC, parts = (n + 32 * U - 1) / (32 * U), lane = threadIdx.x & 31;
    const int64_t item = blockIdx.x * 8ll + (threadIdx.x >> 5), i = item / parts;
    if (i >= a.N) return;
    const int64_t v = token_at(a.tokens, a.idx64, i);
    const bool in = v >= 0 && v < a.V;
    const float fill = v == a.padding ? 0.f : __int_as_float(0x7fffffff);
    const int k0 = static_cast<int>(item % parts) * 32 * U + lane;
    if (!in && v != a.padding && a.status && k0 == 0) atomicOr(a.status, STATUS_INDEX);
    const V* w = reinterpret_cast<const V*>(a.w + (in ? v : 0) * a.ldw);
    V* y = reinterpret_cast<V*>(a.y + i * a.ldy);
    V x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (in && k0 + 32 * u < n) x[u] = w[k0 + 32 * u];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (k0 + 32 * u >= n) break;
        if (!in)
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u].set(e, fill);
        else if (a.scale != 1.f)
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u].set(e, x[u].f(e) * a.scale);
        y[k0 + 32 * u] = x[u];
    }
}

// Narrow rows, dealt out by the vector.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) emb_fwd_narrow(EmbFwd<T> a) {
    using V = Vec<T, VEC>;
    wait_for_primary();
    const Dealt<U> mine(a.deal, blockIdx.x);
    V x[U];
    uint32_t at[U];
    int64_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = mine.get(a.deal, u, at + u);
        v[u] = i < a.N ? token_at(a.tokens, a.idx64, i) : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (v[u] >= 0 && v[u] < a.V) x[u] = reinterpret_cast<const V*>(a.w + v[u] * a.ldw)[at[u]];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = mine.get(a.deal, u, at + u);
        if (i >= a.N) break;
        if (v[u] < 0 || v[u] >= a.V) {
            const bool padding = v[u] == a.padding;
            if (!padding && a.status && at[u] == 0) atomicOr(a.status, STATUS_INDEX);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u].set(e, padding ? 0.f : __int_as_float(0x7fffffff));
        } else if (a.scale != 1.f) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u].set(e, x[u].f(e) * a.scale);
        }
        reinterpret_cast<V*>(a.y + i * a.ldy)[at[u]] = x[u];
    }
}

// ---------------------------------------------------------------- the gradient

// The workspace.
struct EmbSpace {
    WsHeader* hdr;
    int32_t* n_spans;        // how many runs were cut at chunks' borders
    int4* spans;             // [chunks]: the first and one past the last chunk of one, and its token
    uint8_t* named;          // [V]: 1 for rows that a token names
    int32_t *bad, *hist, *keys[2], *rows[2];
    float* parts;            // [chunks, 2, H]
};

// A share of the gradient's rows to be cleared.
struct Clear {
    uint8_t* at;
    int64_t rows, bytes;  // of a row
    int64_t stride;       // bytes from row to row
    int part, of;         // the shares of all rows that its first kernel takes, the next one the next
};

__device__ __forceinline__ void clear_bytes(uint8_t* p, int64_t n) {  // by a block; p and n even
    const int64_t head = -reinterpret_cast<intptr_t>(p) & 15, lead = head < n ? head : n;
    const int64_t mid = (n - lead) / 16;
    for (int64_t i = threadIdx.x; i < lead / 2; i += SORT_THREADS) reinterpret_cast<uint16_t*>(p)[i] = 0;
    uint4* q = reinterpret_cast<uint4*>(p + lead);
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < mid; i += SORT_THREADS) q[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = lead + mid * 16 + 2 * threadIdx.x; i < n; i += 2 * SORT_THREADS) *reinterpret_cast<uint16_t*>(p + i) = 0;
}

// Piece by piece, side by side with the other blocks: all of them together
// write one window that moves on (311 MB by 152 blocks: 53 us; a stretch of
// its own to each block 60).
__device__ __forceinline__ void clear_share(const Clear& c, int kernel, int64_t block, int64_t of) {
    const int64_t first = c.rows * (c.part + kernel) / c.of, rows = c.rows * (c.part + kernel + 1) / c.of - first;
    if (c.stride == c.bytes) {
        constexpr int64_t PIECE = 64 * SORT_THREADS;
        uint8_t* p = c.at + first * c.bytes;
        const int64_t n = rows * c.bytes;
        for (int64_t i = block * PIECE; i < n; i += of * PIECE) clear_bytes(p + i, n - i < PIECE ? n - i : PIECE);
    } else {
        for (int64_t r = block; r < rows; r += of) clear_bytes(c.at + (first + r) * c.stride, c.bytes);
    }
}

struct SortItem {
    int32_t digit, key, row;
};

// The first digit: tokens as they come.  V stands for the ones to leave out.
struct FirstDigit {
    static constexpr bool SEGMENTS = false;
    using Item = SortItem;
    const void* tokens;
    bool idx64;
    int32_t V, mask;
    int64_t padding;
    int32_t *keys, *rows;
    unsigned* stat;
    int32_t* n_spans;
    uint8_t* named;  // nullable
    int32_t sorting;  // blocks that sort
    Clear clear;
    __device__ __forceinline__ void beside(int kernel, int64_t block, int64_t of) const { clear_share(clear, kernel, block, of); }
    __device__ __forceinline__ void begin() const {
        if (blockIdx.x == 0 && threadIdx.x == 0) *n_spans = 0;
        if (named)
            for (int64_t v = static_cast<int64_t>(blockIdx.x) * SORT_THREADS + threadIdx.x; v * 16 < V;
                 v += static_cast<int64_t>(sorting) * SORT_THREADS)
                reinterpret_cast<uint4*>(named)[v] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ Item load(int64_t i, bool* bad) const {
        const int64_t v = token_at(tokens, idx64, i);
        const bool in = v >= 0 && v < V && v != padding;
        *bad |= !in && v != padding;
        const int32_t key = in ? static_cast<int32_t>(v) : V;
        return {key & mask, key, static_cast<int32_t>(i)};
    }
    __device__ __forceinline__ void put(const Item& x, int32_t at) const {
        keys[at] = x.key;
        rows[at] = x.row;
    }
    __device__ __forceinline__ void status(int any) const { *stat = any ? STATUS_INDEX : 0u; }
};

// A later digit.
struct NextDigit {
    static constexpr bool SEGMENTS = false;
    using Item = SortItem;
    const int32_t *from_keys, *from_rows;
    int32_t shift, mask;
    int32_t *keys, *rows;
    Clear clear;
    __device__ __forceinline__ void beside(int kernel, int64_t block, int64_t of) const { clear_share(clear, kernel, block, of); }
    __device__ __forceinline__ void begin() const {}
    __device__ __forceinline__ Item load(int64_t i, bool*) const {
        const int32_t key = from_keys[i];
        return {key >> shift & mask, key, from_rows[i]};
    }
    __device__ __forceinline__ void put(const Item& x, int32_t at) const {
        keys[at] = x.key;
        rows[at] = x.row;
    }
    __device__ __forceinline__ void status(int) const {}
};

constexpr int EMB_CHUNK = 32;       // sorted tokens of a warp
constexpr int EMB_AHEAD = 8;        // rows on their way
constexpr int EMB_ANY_WORDS = 132;  // of a row's slab on any boundary: 128 and the next

template <typename T>
struct EmbBwd {
    const T* dy;
    int64_t ldd, N, V;
    float scale;
    const int32_t *keys, *rows;  // sorted
    uint8_t* named;        // nullable: the others need not be cleared
    int32_t* n_spans;
    int4* spans;
    float* parts;
    void* dw;
    int64_t lddw, chunks;
    bool add, few;
    int32_t H, slabs;
    int32_t split;    // warps to a chunk and slab
    int32_t joining;  // blocks of the last kernel that add pieces up
    int32_t clear_rows;  // vocabulary rows of a warp of the others
};

// A lane's share of a row's slab: ITEMS vectors, 32 vectors apart, as pairs of FP32 sums.
template <typename W, int VEC, int ITEMS>
__device__ __forceinline__ void emb_store(const F2 (&s)[VEC * ITEMS / 2], W* row, int k0, int n, float scale, bool add) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (k0 + 32 * i >= n) break;
        Vec<W, VEC>* out = reinterpret_cast<Vec<W, VEC>*>(row) + k0 + 32 * i;
        Vec<W, VEC> o{};
        if (add) o = *out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float v = (i * VEC + e) & 1 ? hi(s[(i * VEC + e) / 2]) : lo(s[(i * VEC + e) / 2]);
            o.set(e, add ? fmaf(v, scale, o.f(e)) : v * scale);
        }
        *out = o;
    }
}

// The same of a row on any boundary, element by element.
template <typename W, int ITEMS>
__device__ __forceinline__ void emb_store_any(const F2 (&s)[ITEMS], W* row, int k0, int H, float scale, bool add) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 2 * (k0 + 32 * i) + e;
            if (c >= H) break;
            const float v = e ? hi(s[i]) : lo(s[i]);
            row[c] = from_f32<W>(add ? fmaf(v, scale, to_f32(row[c])) : v * scale);
        }
}

// The sums.  A warp takes 32 sorted tokens and a slab of columns, copies their
// rows ahead to shared memory and adds them up until the token changes.  A run
// of equal tokens that reaches into the next chunk belongs to the warp it starts in, as
// long as it has at most 32 rows.  Longer ones are cut at the chunks' borders
// and their pieces go to `parts`: [chunk][0] of a run that comes from the chunk
// before, [chunk][1] of one that starts here; so a token that fills half of the
// batch is spread over as many warps as its rows need.
// ANY: rows of 16-bit elements on any boundary.  They are copied by the words
// that they lie in, and a lane puts its two columns together from one word or
// two neighbours.  A word that reaches past the first or the last row is read by
// its half inside, as nothing says that what lies there may be read (40000 x 1601 bf16 into 32768 rows: 118 us, element by element 351).
template <typename T, typename W, int VEC, int ITEMS, bool ANY>
__global__ void __launch_bounds__(256) emb_sum(EmbBwd<T> a) {
    extern __shared__ __align__(16) uint8_t dyn[];
    using V = Vec<T, VEC>;
    static_assert(!ANY || (VEC == 2 && sizeof(T) == 2));
    constexpr unsigned ALL = 0xFFFFFFFFu;
    constexpr int AHEAD = EMB_AHEAD;
    const int lane = threadIdx.x & 31;
    const int n = a.H / VEC;  // (not with ANY)
    int64_t item = blockIdx.x * 8ll + (threadIdx.x >> 5);
    launch_dependents();
    wait_for_primary();
    if (item >= a.chunks * a.slabs * a.split) return;
    const int sub = static_cast<int>(item % a.split);
    item /= a.split;
    const int64_t c = item / a.slabs;
    const int k0 = static_cast<int>(item % a.slabs) * 32 * ITEMS + lane;
    const int64_t at = c * EMB_CHUNK + lane;
    const int32_t none = static_cast<int32_t>(a.V);  // the key of what is left out, behind all others
    const int32_t key = at < a.N ? a.keys[at] : none, key2 = at + EMB_CHUNK < a.N ? a.keys[at + EMB_CHUNK] : none;
    const int32_t key0 = c > 0 ? a.keys[at - EMB_CHUNK] : -1;  // of the chunk before
    const int32_t row = at < a.N ? a.rows[at] : 0, row2 = at + EMB_CHUNK < a.N ? a.rows[at + EMB_CHUNK] : 0;
    const int items = __popc(__ballot_sync(ALL, key < none));
    if (items == 0) return;
    const int32_t head = __shfl_sync(ALL, key, 0), tail = __shfl_sync(ALL, key, 31);
    // rows of the first run before and in this chunk, and of the last one in this chunk and behind it
    const int head_before = __clz(~__ballot_sync(ALL, key0 == head)), head_here = __ffs(~__ballot_sync(ALL, key == head)) - 1;
    const int tail_here = __clz(~__ballot_sync(ALL, key == tail)), tail_behind = __ffs(~__ballot_sync(ALL, key2 == tail)) - 1;
    auto whole = [](int rows) { return rows < 0 ? 32 : rows; };  // __ffs finds nothing where all 32 are equal
    const bool came = head_before > 0, goes = items == 32 && tail_behind != 0;
    const bool head_long = came && head_before + whole(head_here) > 32, tail_long = goes && tail_here + whole(tail_behind) > 32;
    int begin = came && !head_long ? head_here : 0;                         // the warp before has those
    int end = goes && !tail_long ? 32 + tail_behind : items;
    int32_t next = __shfl_down_sync(ALL, key, 1);
    if (lane == 31) next = -1;                                              // a border, unless the last run goes on
    unsigned last = __ballot_sync(ALL, key != next);
    if (end > 32) last &= 0x7FFFFFFFu;
    if (tail_long && !(head_long && head == tail) && k0 == lane && sub == 0) {  // a long run starts here: where does it end?
        int64_t to = c + 1;
        for (unsigned same = ALL; same == ALL; to += same == ALL ? 32 : __ffs(~same) - 1)
            same = __ballot_sync(ALL, to + lane < a.chunks && a.keys[(to + lane) * EMB_CHUNK] == tail);
        if (lane == 0) a.spans[atomicAdd(a.n_spans, 1)] = make_int4(static_cast<int>(c), static_cast<int>(to), tail, 0);
    }
    if (a.split > 1) {  // the runs that start in this part of the chunk
        const int width = 32 / a.split, lo = sub * width;
        const unsigned starts = (last << 1 | 1u << (begin & 31)) & ALL << (begin & 31) & (items < 32 ? (1u << items) - 1 : ALL);
        const unsigned here = starts >> lo & ((1u << width) - 1), behind = lo + width < 32 ? starts >> (lo + width) : 0u;
        if (!here || begin >= items) return;
        begin = lo + __ffs(here) - 1;
        if (behind) end = lo + width + __ffs(behind) - 1;
    }
    constexpr int PAIRS = VEC * ITEMS / 2;
    F2 s[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) s[p] = f2(0.f);
    const int shift = ANY ? 0 : k0;  // a row's address at this lane's columns: shifted back by the lane that holds the row
    const uintptr_t from = reinterpret_cast<uintptr_t>(reinterpret_cast<const V*>(a.dy + row * a.ldd) + shift);
    const uintptr_t from2 = reinterpret_cast<uintptr_t>(reinterpret_cast<const V*>(a.dy + row2 * a.ldd) + shift);
    auto row_at = [&](int i) {
        const unsigned long long p = __shfl_sync(ALL, static_cast<unsigned long long>(i < 32 ? from : from2), i & 31);
        return reinterpret_cast<const V*>(p) + (ANY ? 0 : lane - (i & 31));
    };
    auto finish = [&](int i) {  // of a run, or of its part in this chunk: i is its last row
        const int32_t v = i < 32 ? __shfl_sync(ALL, key, i) : tail;
        const bool is_head = v == head && head_long, is_tail = v == tail && tail_long;
        if (a.named && k0 == 0) a.named[v] = 1;
        const bool whole_run = !is_head && !is_tail;
        W* out = static_cast<W*>(a.dw) + v * a.lddw;
        float* piece = a.parts + (c * 2 + (is_head ? 0 : 1)) * a.H;
        if constexpr (ANY) {
            if (whole_run)
                emb_store_any<W, ITEMS>(s, out, k0, a.H, a.scale, a.add);
            else
                emb_store_any<float, ITEMS>(s, piece, k0, a.H, 1.f, false);
        } else {
            if (whole_run)
                emb_store<W, VEC, ITEMS>(s, out, k0, n, a.scale, a.add);
            else
                emb_store<float, VEC, ITEMS>(s, piece, k0, n, 1.f, false);
        }
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) s[p] = f2(0.f);
    };
    auto sum_rows = [&](auto next_row) {
        for (int i = begin; i < end;) {
            const unsigned ends = i < 32 ? last >> i : 0u;
            const int stop = ends ? i + __ffs(ends) : end;
            for (; i < stop; ++i) {
                const RowVectors<T, VEC, ITEMS> x = next_row(i);
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) s[p] = add2(s[p], x.pair(p));
            }
            finish(i - 1);
        }
    };
    int slot = 0;
    if constexpr (!ANY) {
        // rows on their way: [AHEAD][ITEMS][threads], each thread its own vectors
        constexpr int SLOT = ITEMS * 256;
        V* ring = reinterpret_cast<V*>(dyn) + threadIdx.x;
        auto copy = [&](int i, int to) {
            if (i < end) {
                const V* p = row_at(i);
#pragma unroll
                for (int k = 0; k < ITEMS; ++k)
                    if (k0 + 32 * k < n) copy_async<sizeof(V)>(ring + to + k * 256, p + 32 * k);
            }
            copy_async_commit();
        };
#pragma unroll
        for (int k = 0; k < AHEAD - 1; ++k) copy(begin + k, k * SLOT);
        sum_rows([&](int i) {
            copy(i + AHEAD - 1, (slot + (AHEAD - 1) * SLOT) & (AHEAD * SLOT - 1));
            copy_async_wait<AHEAD - 1>();
            RowVectors<T, VEC, ITEMS> x;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) x.v[k] = ring[slot + k * 256];
            slot = (slot + SLOT) & (AHEAD * SLOT - 1);
            return x;
        });
    } else {
        // rows on their way: [warps][AHEAD][EMB_ANY_WORDS], a warp's words side by side
        static_assert(32 * ITEMS + 1 <= EMB_ANY_WORDS);
        uint32_t* ring = reinterpret_cast<uint32_t*>(dyn) + (threadIdx.x >> 5) * AHEAD * EMB_ANY_WORDS;
        const unsigned odd = __ballot_sync(ALL, from & 2), odd2 = __ballot_sync(ALL, from2 & 2);  // rows that start in a word's middle
        const uintptr_t first_row = reinterpret_cast<uintptr_t>(a.dy), last_row = reinterpret_cast<uintptr_t>(a.dy + (a.N - 1) * a.ldd);
        const int bytes = 2 * a.H;
        auto copy = [&](int i, int to) {
            if (i < end) {
                const uintptr_t p = reinterpret_cast<uintptr_t>(row_at(i));
                const int words = static_cast<int>((p & 2) + bytes + 3) >> 2;
                const uint32_t* w = reinterpret_cast<const uint32_t*>(p & ~uintptr_t{3});
                uint32_t* out = ring + to * EMB_ANY_WORDS - (k0 - lane);
                const bool before = p == first_row && (p & 2), behind = p == last_row && ((p + bytes) & 2);  // words that reach outside
                auto word = [&](int q) {
                    if (before && q == 0)
                        out[q] = static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(w + q)[1]) << 16;
                    else if (behind && q == words - 1)
                        out[q] = *reinterpret_cast<const uint16_t*>(w + q);
                    else if (q < words)
                        copy_async<4>(out + q, w + q);
                };
#pragma unroll
                for (int k = 0; k < ITEMS; ++k) word(k0 + 32 * k);
                if (lane == 0 && (p & 2)) word(k0 + 32 * ITEMS);
            }
            copy_async_commit();
        };
#pragma unroll
        for (int k = 0; k < AHEAD - 1; ++k) copy(begin + k, k);
        sum_rows([&](int i) {
            copy_async_wait<AHEAD - 2>();
            __syncwarp();  // all lanes' words of this row have come, and the row before has been read
            copy(i + AHEAD - 1, (slot + AHEAD - 1) & (AHEAD - 1));
            const uint32_t* w = ring + slot * EMB_ANY_WORDS + lane;
            const unsigned by = (i < 32 ? odd >> i : odd2 >> (i - 32)) & 1 ? 0x5432 : 0x3210;
            RowVectors<T, VEC, ITEMS> x;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const uint32_t both = __byte_perm(w[32 * k], w[32 * k + 1], by);
                __builtin_memcpy(&x.v[k], &both, 4);
            }
            slot = (slot + 1) & (AHEAD - 1);
            return x;
        });
    }
}

// ---------------------------------------------------------------- few tokens

// Up to EMB_RANK tokens are sorted in one kernel: a token's place is the number of tokens that come before it, and every
// block counts them for 32, a lane each, its warps a share of the tokens.  That is N * N comparisons, and the gradient's
// rows are cleared behind them: 620 tokens of 128 bf16 11.8 us, 17.0 by digits in one block; 5084 of 128 fp16 19.8 and
// 23.8 by digits; 8192 of 512 bf16 27.7 and 27.9, of 1024 into 151936 rows 68.9 and 62.9.
constexpr int EMB_RANK = 6144;

struct RankJob {
    FirstDigit f;
    int32_t n, blocks;  // blocks that count; all of them clear a share
};
__global__ void __launch_bounds__(SORT_THREADS) emb_rank(RankJob job) {
    __shared__ __align__(16) int32_t keys[EMB_RANK];
    __shared__ int32_t before[32];
    const FirstDigit& f = job.f;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = job.n;
    if (!f.clear.rows) launch_dependents();
    wait_for_primary();
    f.begin();
    if (static_cast<int>(blockIdx.x) < job.blocks) {
        bool bad = false;
#pragma unroll 4
        for (int i = t; i < (n + 3) / 4 * 4; i += SORT_THREADS) keys[i] = i < n ? f.load(i, &bad).key : INT32_MAX;
        if (t < 32) before[t] = 0;
        const int any = __syncthreads_or(bad);
        if (t == 0 && blockIdx.x == 0) f.status(any);
        const int own = blockIdx.x * 32, i = own + lane;
        const int32_t key = i < n ? keys[i] : 0;
        const int each = (n + 4 * SORT_WARPS - 1) / (4 * SORT_WARPS) * 4, j0 = warp * each, end = (n + 3) / 4 * 4, j1 = j0 + each < end ? j0 + each : end;
        const int lo = own < j1 ? own : j1, hi = own + 32 < j1 ? own + 32 : j1;
        int32_t count = 0;
        int j = j0;
        auto add = [&](int32_t a, int32_t b, int32_t c, int32_t d) {
            const int4 k = *reinterpret_cast<const int4*>(keys + j);
            count += (k.x < a) + (k.y < b) + (k.z < c) + (k.w < d);
        };
#pragma unroll 4
        for (; j < lo; j += 4) add(key + 1, key + 1, key + 1, key + 1);  // equal ones that stand before come before
        for (; j < hi; j += 4) add(key + (j < i), key + (j + 1 < i), key + (j + 2 < i), key + (j + 3 < i));
#pragma unroll 4
        for (; j < j1; j += 4) add(key, key, key, key);
        atomicAdd(before + lane, count);
        __syncthreads();
        if (t < 32 && i < n) f.put({0, key, i}, before[lane]);
    }
    if (f.clear.rows) clear_share(f.clear, 0, blockIdx.x, gridDim.x);
}

// A block adds up a whole run, where there are up to EMB_FEW tokens: no pieces, so no third kernel.  64 tokens of 256 bf16
// 8.1 us, 10.4 the long way, 256 of 513 fp16 10.1 and 24.1, with one token alone 16.6 and 21.6; but a run waits on one
// block: 512 of 64 bf16 7.9 and 10.9, with one token alone 18.1 and 10.9.
constexpr int EMB_FEW = 256, EMB_FEW_WARPS = 8;

// A block per sorted token and slab: the first of a run adds it up, its rows
// shared out over its warps and joined in a fixed order.
template <typename T, typename W, int VEC, int ITEMS>
__global__ void __launch_bounds__(32 * EMB_FEW_WARPS) emb_sum_few(EmbBwd<T> a) {
    using V = Vec<T, VEC>;
    constexpr int PAIRS = VEC * ITEMS / 2, WARPS = EMB_FEW_WARPS, BATCH = VEC * sizeof(T) == 16 ? 8 / ITEMS : 4;
    __shared__ F2 part[WARPS][PAIRS][32];
    wait_for_primary();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = a.H / VEC, N = static_cast<int>(a.N);
    const int i = static_cast<int>(blockIdx.x / a.slabs), k0 = static_cast<int>(blockIdx.x % a.slabs) * 32 * ITEMS + lane;
    const int32_t v = a.keys[i];
    if (v >= a.V || (i > 0 && a.keys[i - 1] == v)) return;
    int end = i + 1;
    for (unsigned same = 0xFFFFFFFFu; same == 0xFFFFFFFFu; end += same == 0xFFFFFFFFu ? 32 : __ffs(~same) - 1)
        same = __ballot_sync(0xFFFFFFFFu, end + lane < N && a.keys[end + lane] == v);
    if (warp && end - i == 1) return;
    F2 s[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) s[p] = f2(0.f);
    for (int r = i + warp; r < end; r += WARPS * BATCH) {
        RowVectors<T, VEC, ITEMS> x[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const bool in = r + WARPS * b < end;
            const V* from = reinterpret_cast<const V*>(a.dy + static_cast<int64_t>(in ? a.rows[r + WARPS * b] : 0) * a.ldd) + k0;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                x[b].v[k] = V{};
                if (in && k0 + 32 * k < n) load_now(x[b].v[k], from + 32 * k);
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) s[p] = add2(s[p], x[b].pair(p));
    }
    if (end - i > 1) {
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) part[warp][p][lane] = s[p];
        __syncthreads();
        if (warp) return;
        for (int w = 1; w < WARPS; ++w)
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) s[p] = add2(s[p], part[w][p][lane]);
    }
    emb_store<W, VEC, ITEMS>(s, static_cast<W*>(a.dw) + v * a.lddw, k0, n, a.scale, a.add);
}

// ---------------------------------------------------------------- the end

// What is left after the sums.  The first `joining` blocks: the runs that reach
// past a chunk, a slab of columns of one per block, its pieces shared out over
// eight warps and added in a fixed order.  The others: the vocabulary rows that
// no token names are cleared, while those wait for their pieces.
template <typename W, int VEC, int ITEMS, int CLEAR_VEC>
__global__ void __launch_bounds__(256) emb_finish(EmbBwd<float> a) {
    constexpr int PAIRS = VEC * ITEMS / 2;
    __shared__ F2 s[8][PAIRS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_primary();
    if (static_cast<int>(blockIdx.x) >= a.joining) {
        const int64_t v0 = ((static_cast<int64_t>(blockIdx.x) - a.joining) * 8 + warp) * a.clear_rows;
        const unsigned named = __ballot_sync(0xFFFFFFFFu, lane >= a.clear_rows || v0 + lane >= a.V || a.named[v0 + lane]);
        for (int j = 0; j < a.clear_rows; ++j) {
            if (named >> j & 1) continue;
            using Z = Vec<W, CLEAR_VEC>;
            Z* out = reinterpret_cast<Z*>(static_cast<W*>(a.dw) + (v0 + j) * a.lddw);
#pragma unroll 4
            for (int k = lane; k < a.H / CLEAR_VEC; k += 32) out[k] = Z{};
        }
        return;
    }
    const int n = a.H / VEC;
    const int64_t items = static_cast<int64_t>(*a.n_spans) * a.slabs;
    for (int64_t item = blockIdx.x; item < items; item += a.joining) {
        const int4 span = a.spans[item / a.slabs];
        const int k0 = static_cast<int>(item % a.slabs) * 32 * ITEMS + lane;
        const int64_t c0 = span.x, end = span.y, v = span.z;
        F2 sum[PAIRS];
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) sum[p] = f2(0.f);
        auto load = [&](RowVectors<float, VEC, ITEMS>& x, int64_t part) {  // -1: none
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                x.v[i] = Vec<float, VEC>{};
                if (part >= 0 && k0 + 32 * i < n) load_now(x.v[i], reinterpret_cast<const Vec<float, VEC>*>(a.parts + part * a.H) + k0 + 32 * i);
            }
        };
        if (warp == 0) {
            RowVectors<float, VEC, ITEMS> x;
            load(x, c0 * 2 + 1);
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) sum[p] = x.pair(p);
        }
        for (int64_t c = c0 + 1 + warp; c < end; c += 64) {  // eight loads on their way
            RowVectors<float, VEC, ITEMS> x[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) load(x[b], c + 8 * b < end ? (c + 8 * b) * 2 : -1);
#pragma unroll
            for (int b = 0; b < 8; ++b)
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) sum[p] = add2(sum[p], x[b].pair(p));
        }
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) s[warp][p][lane] = sum[p];
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < 8; ++w)
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) sum[p] = add2(sum[p], s[w][p][lane]);
            emb_store<W, VEC, ITEMS>(sum, static_cast<W*>(a.dw) + v * a.lddw, k0, n, a.scale, a.add);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host

lce_status_t emb_sizes(int64_t N, int64_t V, int64_t H) {
    if (N < 0 || V <= 0 || H <= 0) return LCE_ERR_INVALID_ARG;
    if (N > INT32_MAX || V >= INT32_MAX || H > EMB_MAX_H) return LCE_ERR_UNSUPPORTED;
    return LCE_OK;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Bits of the keys 0 .. V, in digits of at most EMB_DIGIT_BITS.
struct Digits {
    int passes, bits;
};
Digits digits_of(int64_t V) {
    int bits = 1;
    while ((V >> bits) != 0) ++bits;
    const int passes = (bits + EMB_DIGIT_BITS - 1) / EMB_DIGIT_BITS;
    return {passes, (bits + passes - 1) / passes};
}

size_t emb_space(int64_t N, int64_t V, int64_t H, EmbSpace* e, void* ws) {
    const Digits d = digits_of(V);
    const int64_t chunks = (N + EMB_CHUNK - 1) / EMB_CHUNK;
    const size_t blocks = static_cast<size_t>(sort_blocks(N)), items = align256(static_cast<size_t>(N) * 4);
    size_t at = 1024;
    auto take = [&](size_t bytes) {
        uint8_t* p = static_cast<uint8_t*>(ws) + at;
        at += align256(bytes);
        return p;
    };
    EmbSpace here{};
    EmbSpace& f = e ? *e : here;
    f.hdr = static_cast<WsHeader*>(ws);
    f.bad = reinterpret_cast<int32_t*>(take(blocks * 4));
    f.hist = reinterpret_cast<int32_t*>(take(blocks * 4 << d.bits));
    f.n_spans = reinterpret_cast<int32_t*>(take(4));
    f.spans = reinterpret_cast<int4*>(take(static_cast<size_t>(chunks) * 16));
    f.named = take(static_cast<size_t>(V));
    for (int k = 0; k < 2; ++k) {
        f.keys[k] = reinterpret_cast<int32_t*>(take(items));
        f.rows[k] = reinterpret_cast<int32_t*>(take(items));
    }
    f.parts = reinterpret_cast<float*>(take(chunks > 1 ? static_cast<size_t>(chunks) * 2 * H * 4 : 0));
    return at;
}

// Whether all of the gradient's rows are cleared while the tokens are sorted, on
// the SMs that the sort leaves idle, although some are written again: where the
// sort by digits has few blocks and more rows than tokens lie behind it, or where
// the clearing behind the one kernel that ranks few tokens is short.  Else the rows
// that no token names are cleared at the end, by many short blocks.  Early and
// late: 16384 tokens, 151936 rows of 1024 bf16 70.5 and 75.4 us; 31070 and 50257
// of 1472 63.7 and 74.4; 40183 and 5534 of 2176 80.2 and 76.9; 131072 and 151936
// of 1024 175 and 155; and ranked 4000 and 8000 of 1024 16.7 and 22.2, 3000 and
// 8000 of 4096 27.1 and 26.4, 4096 and 151936 of 1024 61.7 and 56.4.
constexpr int64_t EMB_CLEAR_TOKENS = 65536;
constexpr int64_t EMB_CLEAR_BYTES = 512ll << 20, EMB_CLEAR_BYTES_RANKED = 32ll << 20;
bool emb_early(int64_t N, int64_t V, int64_t bytes) {
    if (N == 0) return true;  // no kernel comes after the one that ranks
    if (N <= EMB_RANK) return bytes <= EMB_CLEAR_BYTES_RANKED;
    return N <= EMB_CLEAR_TOKENS && N <= V && bytes <= EMB_CLEAR_BYTES;
}

// The sorted tokens: their place in e.keys and e.rows.
lce_status_t emb_sort(int64_t N, int64_t V, const void* tokens, bool idx64, int64_t padding, bool name, Clear clear,
                      const EmbSpace& e, int* where, cudaStream_t s) {
    if (N <= EMB_RANK) {
        const int32_t blocks = N > 32 ? static_cast<int32_t>((N + 31) / 32) : 1;
        const int32_t all = blocks < SORT_BLOCKS && clear.rows ? static_cast<int32_t>(SORT_BLOCKS) : blocks;
        const RankJob job{{tokens, idx64, static_cast<int32_t>(V), 0, padding, e.keys[0], e.rows[0], &e.hdr->status, e.n_spans,
                           name ? e.named : nullptr, all, clear},
                          static_cast<int32_t>(N), blocks};
        *where = 0;
        LCE_PROFILED(launch_after(emb_rank, dim3(static_cast<unsigned>(all)), SORT_THREADS, 0, s, job));
        return LCE_OK;
    }
    const Digits d = digits_of(V);
    SortShape shape{};
    shape.n = N;
    shape.bins = 1 << d.bits;
    shape.blocks = static_cast<int32_t>(sort_blocks(N));
    shape.per = (N + shape.blocks - 1) / shape.blocks;
    shape.hist = e.hist;
    shape.bad = e.bad;
    if (clear.rows) shape.extra = static_cast<int32_t>(SORT_BLOCKS) - shape.blocks;
    *where = (d.passes - 1) & 1;
    FirstDigit first{tokens, idx64, static_cast<int32_t>(V), shape.bins - 1, padding, e.keys[0], e.rows[0], &e.hdr->status,
                           e.n_spans, name ? e.named : nullptr, shape.blocks, clear};
    auto next = [&](int p) {
        const int from = (p - 1) & 1, to = p & 1;
        return NextDigit{e.keys[from], e.rows[from], p * d.bits, shape.bins - 1, e.keys[to], e.rows[to], clear};
    };
    clear.of = 2 * d.passes;  // a share for each kernel
    first.clear = clear;
    lce_status_t st = sort_by(first, shape, s);
    shape.bad = nullptr;
    for (int p = 1; p < d.passes && st == LCE_OK; ++p) {
        clear.part = 2 * p;
        st = sort_by(next(p), shape, s);
    }
    return st;
}

// The widest vectors in which rows `ld` elements apart from p can be read.
template <typename T>
int vector_of(const void* p, int64_t ld, int64_t H) {
    constexpr int V = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
    if (H % V == 0 && ld % V == 0 && aligned_to(p, 16)) return V;
    return H % V4 == 0 && ld % V4 == 0 && aligned_to(p, 4) ? V4 : 1;
}

// Rows of at least 64 vectors take a warp (16384 tokens of 1024 bf16: 8.9 us,
// 10.4 dealt out; 131072 of 64 fp16: 20.7 and 6.5); several vectors a lane where
// that still gives every SM its warps, one for a decode step.
template <typename T, int VEC>
lce_status_t emb_lookup(EmbFwd<T> a, cudaStream_t s) {
    constexpr int U = VEC * sizeof(T) == 16 ? 4 : 8;
    const int64_t n = a.H / VEC;
    if (n >= 64) {
        const int64_t wide = a.N * ((n + 32 * U - 1) / (32 * U));
        const bool enough = wide >= 152 * 32;
        const int64_t blocks = ((enough ? wide : a.N * ((n + 31) / 32)) + 7) / 8;
        if (blocks > INT32_MAX) return LCE_ERR_UNSUPPORTED;
        if (enough)
            LCE_PROFILED(launch_after(emb_fwd_wide<T, VEC, U>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a));
        else
            LCE_PROFILED(launch_after(emb_fwd_wide<T, VEC, 1>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a));
        return LCE_OK;
    }
    const int64_t vectors = a.N * n;
    const bool enough = vectors >= 152 * 4 * 256 * 4;
    const int64_t share = 256 * (enough ? 4 : 1), blocks = (vectors + share - 1) / share;
    if (blocks > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    a.deal = deal_of(n);
    if (enough)
        LCE_PROFILED(launch_after(emb_fwd_narrow<T, VEC, 4>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a));
    else
        LCE_PROFILED(launch_after(emb_fwd_narrow<T, VEC, 1>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a));
    return LCE_OK;
}

int32_t emb_slabs(int64_t vectors, int items) { return static_cast<int32_t>((vectors + 32 * items - 1) / (32 * items)); }

template <typename T, typename W, int VEC>
lce_status_t emb_sums(EmbBwd<T> a, cudaStream_t s) {
    if (a.few) {
        constexpr int ITEMS = 8 / VEC;
        a.slabs = emb_slabs(a.H / VEC, ITEMS);
        const int64_t blocks = a.N * a.slabs;
        if (blocks == 0) return LCE_OK;
        LCE_PROFILED(launch_after(emb_sum_few<T, W, VEC, ITEMS>, dim3(static_cast<unsigned>(blocks)), 32 * EMB_FEW_WARPS, 0, s, a));
        return LCE_OK;
    }
    constexpr bool ANY = VEC * sizeof(T) < 4;
    constexpr int SVEC = ANY ? 2 : VEC, ITEMS = 8 / SVEC;
    a.slabs = emb_slabs(ANY ? (a.H + 1) / 2 : a.H / VEC, ITEMS);
    // a chunk's runs over four warps where there are few chunks (620 tokens of 128 bf16: 12.0 us, not 18.4; 90000 of 64: 51.2
    // and 65.4)
    if (a.chunks * a.slabs < 152 * 32) a.split = 4;
    const int64_t blocks = (a.chunks * a.slabs * a.split + 7) / 8;
    if (blocks == 0) return LCE_OK;  // no tokens: all rows have been cleared (emb_early), or the sums stay as they are
    if (blocks > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    constexpr size_t smem = static_cast<size_t>(EMB_AHEAD) * (ANY ? 8 * EMB_ANY_WORDS * 4 : ITEMS * 256 * VEC * sizeof(T));
    static std::atomic<uint64_t> sums{0}, finishes{0};
    // 16-byte vectors of FP32 pieces where dw's rows have vectors at all, and few columns to a block: there are few long runs
    constexpr int JVEC = VEC % 4 == 0 ? 4 : VEC, JITEMS = JVEC == 4 ? 1 : 4 / JVEC;
    auto finish = emb_finish<W, JVEC, JITEMS, VEC>;
    if (!allow_smem(&sums, emb_sum<T, W, SVEC, ITEMS, ANY>, static_cast<int>(smem)) || !allow_smem(&finishes, finish, 0)) return LCE_ERR_CUDA;
    LCE_PROFILED(launch_after(emb_sum<T, W, SVEC, ITEMS, ANY>, dim3(static_cast<unsigned>(blocks)), 256, smem, s, a));
    EmbBwd<float> j{};
    j.V = a.V;
    j.scale = a.scale;
    j.named = a.named;
    j.n_spans = a.n_spans;
    j.spans = a.spans;
    j.parts = a.parts;
    j.dw = a.dw;
    j.lddw = a.lddw;
    j.chunks = a.chunks;
    j.add = a.add;
    j.H = a.H;
    j.slabs = emb_slabs(a.H / JVEC, JITEMS);
    // about 8 KB to a warp: many short blocks write faster than few long ones (131072 tokens, rows of 4096 bf16: 389 us
    // with one row to a warp, 401 with eight)
    const int64_t some = 8192 / (a.H * static_cast<int64_t>(sizeof(W)));
    j.clear_rows = static_cast<int32_t>(some < 1 ? 1 : some < 8 ? some : 8);
    const int64_t most = (a.chunks - 1) * j.slabs, clearing = a.named ? (a.V + 8 * j.clear_rows - 1) / (8 * j.clear_rows) : 0;
    if (most + clearing > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    j.joining = static_cast<int32_t>(most < 1216 ? most : 1216);
    if (j.joining + clearing == 0) return LCE_OK;
    LCE_PROFILED(launch_after(finish, dim3(static_cast<unsigned>(j.joining + clearing)), 256, 0, s, j));
    return LCE_OK;
}

template <typename T, typename W>
lce_status_t emb_gradient(const EmbBwd<T>& a, cudaStream_t s) {
    const int in = vector_of<T>(a.dy, a.ldd, a.H), out = vector_of<W>(a.dw, a.lddw, a.H);
    constexpr int V = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
    if (in == V && out == vec16<W>()) return emb_sums<T, W, V>(a, s);
    if (V4 > 1 && in >= V4 && a.lddw % V4 == 0 && aligned_to(a.dw, V4 * sizeof(W))) return emb_sums<T, W, V4>(a, s);
    return emb_sums<T, W, 1>(a, s);
}

bool index_ok(const void* p, int bytes) { return (bytes == 4 || bytes == 8) && p && aligned_to(p, bytes); }

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status_t lce_embedding_forward(int64_t N, int64_t V, int64_t H, int dtype, const void* tokens, int index_bytes,
                                   const void* weight, int64_t ldw, float scale, int64_t padding_token, void* y,
                                   int64_t ldy, void* status, lce_stream_t stream) {
    const lce_status_t st = emb_sizes(N, V, H);
    if (st != LCE_OK) return st;
    if (!dtype_known(dtype) || ldw < H || ldy < H || !aligned_to(status, 4)) return LCE_ERR_INVALID_ARG;
    if (N == 0) return LCE_OK;
    const size_t es = dtype_bytes(dtype);
    if (!index_ok(tokens, index_bytes) || !weight || !aligned_to(weight, es) || !y || !aligned_to(y, es))
        return LCE_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        const EmbFwd<T> a{tokens, index_bytes == 8, static_cast<const T*>(weight), ldw, N, V, padding_token, scale,
                          static_cast<T*>(y), ldy, static_cast<unsigned*>(status), static_cast<int32_t>(H), {}};
        constexpr int V16 = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
        const int from = vector_of<T>(weight, ldw, H), to = vector_of<T>(y, ldy, H), vec = from < to ? from : to;
        if (vec == V16) return emb_lookup<T, V16>(a, s);
        return V4 > 1 && vec == V4 ? emb_lookup<T, V4>(a, s) : emb_lookup<T, 1>(a, s);
    });
}

lce_status_t lce_embedding_workspace_size(int64_t N, int64_t V, int64_t H, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = emb_sizes(N, V, H);
    if (st == LCE_OK) *bytes = emb_space(N, V, H, nullptr, nullptr);
    return st;
}

lce_status_t lce_embedding_backward(int64_t N, int64_t V, int64_t H, int dtype, int gtype, const void* tokens,
                                    int index_bytes, const void* grad_y, int64_t ldg, float scale,
                                    int64_t padding_token, void* grad_weight, int64_t ldgw, void* ws, size_t ws_bytes,
                                    lce_stream_t stream, uint32_t flags) {
    const lce_status_t st = emb_sizes(N, V, H);
    if (st != LCE_OK) return st;
    const bool add = (flags & LCE_ACCUMULATE) != 0;
    if (!dtype_known(dtype) || !dtype_known(gtype) || ldg < H || ldgw < H || (flags & ~LCE_ACCUMULATE)) return LCE_ERR_INVALID_ARG;
    if ((gtype != dtype && gtype != LCE_F32) || (add && gtype != LCE_F32)) return LCE_ERR_UNSUPPORTED;
    if (!grad_weight || !aligned_to(grad_weight, dtype_bytes(gtype)) || !ws || !aligned_to(ws, 256)) return LCE_ERR_INVALID_ARG;
    if (N && (!index_ok(tokens, index_bytes) || !grad_y || !aligned_to(grad_y, dtype_bytes(dtype)))) return LCE_ERR_INVALID_ARG;
    EmbSpace e;
    if (ws_bytes < emb_space(N, V, H, &e, ws)) return LCE_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int where = 0;
    const int64_t size = static_cast<int64_t>(dtype_bytes(gtype));
    const bool few = N <= EMB_FEW && (add || V * H * size <= EMB_CLEAR_BYTES);
    const bool early = !add && (few || emb_early(N, V, V * H * size)), late = !add && !early;
    const Clear clear{static_cast<uint8_t*>(grad_weight), early ? V : 0, H * size, ldgw * size, 0, 1};
    const lce_status_t sorted = emb_sort(N, V, tokens, index_bytes == 8, padding_token, late, clear, e, &where, s);
    if (sorted != LCE_OK) return sorted;
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        const EmbBwd<T> a{static_cast<const T*>(grad_y), ldg, N, V, scale, e.keys[where], e.rows[where],
                          late ? e.named : nullptr, e.n_spans, e.spans,
                          e.parts, grad_weight, ldgw, (N + EMB_CHUNK - 1) / EMB_CHUNK, add, few, static_cast<int32_t>(H), 0, 1, 0, 0};
        return gtype == LCE_F32 ? emb_gradient<T, float>(a, s) : emb_gradient<T, T>(a, s);
    });
}

}  // extern "C"
