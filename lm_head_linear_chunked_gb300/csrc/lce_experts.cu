// Rows sorted by expert, and back.
//
// T tokens name k experts each (a slot is (t, j), its number t k + j).  The
// plan sorts the slots by expert, in the order of their numbers: expert e's
// rows are offsets[e] .. offsets[e] + counts[e], each segment starting on a
// multiple of `align`.
//
//   dispatch  xs[pos_tj] = x_t, 0 in rows that no slot takes;  dx_t = sum_j dxs[pos_tj]
//   combine   y_t = sum_j w_tj ys[pos_tj];  dys[pos_tj] = w_tj dy_t,  dw_tj = <dy_t, ys[pos_tj]>
//
// All four passes go by tokens, so a token's row is read or written once and
// its slots' rows are each touched once: they are bound by those bytes.  Sums
// over slots and columns are FP32, in an order fixed by the sizes.
#include <type_traits>

#include "lce_sort.cuh"

namespace lce {
namespace {

struct PlanArgs {
    static constexpr bool SEGMENTS = true;
    struct Item {
        int32_t digit, slot;  // the expert, and the slot's number
    };
    const void* experts;
    bool idx64;
    const uint8_t* mask;   // nullable; one byte per token
    int32_t E, k, align;
    int32_t *positions, *slots;
    int64_t *counts, *offsets;
    int32_t R;
    unsigned* stat;
    __device__ __forceinline__ void begin() const {}
    __device__ __forceinline__ void beside(int, int64_t, int64_t) const {}
    __device__ __forceinline__ Item load(int64_t i, bool* bad) const {
        const int32_t slot = static_cast<int32_t>(i);
        const int64_t e = idx64 ? static_cast<const int64_t*>(experts)[i] : static_cast<const int32_t*>(experts)[i];
        if (mask && !mask[slot / k]) return {E, slot};
        if (e >= 0 && e < E) return {static_cast<int32_t>(e), slot};
        if (e != -1) *bad = true;
        return {E, slot};
    }
    __device__ __forceinline__ void put(const Item& x, int32_t at) const {
        positions[x.slot] = x.digit < E ? at : -1;
        if (x.digit < E) slots[at] = x.slot;
    }
    __device__ __forceinline__ void segment(int32_t e, int32_t count, int32_t start) const {
        offsets[e] = start;
        if (e == E) return;  // the end of the last one
        counts[e] = count;
        const int32_t end = start + (count + align - 1) / align * align;
        for (int32_t r = start + count; r < end; ++r) slots[r] = -1;
    }
    __device__ __forceinline__ void ends(int32_t end) const {
        for (int64_t r = end + static_cast<int64_t>(blockIdx.x) * SORT_THREADS + threadIdx.x; r < R;
             r += static_cast<int64_t>(gridDim.x) * SORT_THREADS)
            slots[r] = -1;
    }
    __device__ __forceinline__ void status(int any) const { *stat = any ? STATUS_INDEX : 0u; }
};

struct MoveArgs {
    const int32_t *positions, *slots;
    const void* token_rows;  // x, dy, or the output
    const void* slot_rows;
    const void* weights;     // nullable: 1
    bool w32;
    void *token_out, *slot_out, *weights_out;  // each nullable
    int64_t ldt, lds, ldto, ldso;
    int64_t T, R;
    int32_t k, H;
    int32_t share;           // warps to a token (combine's gradients): 1, 2, 4 or 8
    int32_t clearing;        // blocks that clear rows
    Deal deal;               // of the tokens' vectors
};

// The rows of up to 32 slots of a token, one to a lane; -1 for none (a position
// outside the rows, as of a plan made for others, counts as none).
__device__ __forceinline__ int64_t lane_row(const MoveArgs& a, int64_t t, int j0) {
    const int j = j0 + (threadIdx.x & 31);
    const int64_t p = j < a.k ? a.positions[t * a.k + j] : -1;
    return p < a.R ? p : -1;
}
template <typename T>
__device__ __forceinline__ float lane_weight(const MoveArgs& a, int64_t t, int j0) {
    const int j = j0 + (threadIdx.x & 31);
    return a.weights && j < a.k ? load_w<T>(a.weights, a.w32, t * a.k + j) : 1.f;
}

// EXPERT_CLEAR sorted rows of a warp: those that no slot takes are zero.
constexpr int EXPERT_CLEAR = 8;
template <typename T, int VEC>
__device__ __forceinline__ void clear_rows(const MoveArgs& a, int64_t r0) {
    using V = Vec<T, VEC>;
    const int lane = threadIdx.x & 31;
    unsigned todo = __ballot_sync(0xFFFFFFFFu, lane < EXPERT_CLEAR && r0 + lane < a.R && a.slots[r0 + lane] < 0);
    for (; todo; todo &= todo - 1) {
        V* out = reinterpret_cast<V*>(static_cast<T*>(a.slot_out) + (r0 + __ffs(todo) - 1) * a.ldso);
#pragma unroll 4
        for (int i = lane; i < a.H / VEC; i += 32) out[i] = V{};
    }
}

// dispatch: a warp per token and U vectors of each lane, read once and written
// to all the token's rows.  The first blocks clear rows.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) expert_spread(MoveArgs a) {
    using V = Vec<T, VEC>;
    wait_for_primary();
    const int lane = threadIdx.x & 31, n = a.H / VEC, parts = (n + 32 * U - 1) / (32 * U);
    if (static_cast<int>(blockIdx.x) < a.clearing) return clear_rows<T, VEC>(a, (blockIdx.x * 8ll + (threadIdx.x >> 5)) * EXPERT_CLEAR);
    const uint32_t item = (blockIdx.x - a.clearing) * 8u + (threadIdx.x >> 5);
    if (item >= static_cast<uint32_t>(a.T) * parts) return;
    const int64_t t = item / parts;
    const int k0 = static_cast<int>(item % parts) * 32 * U + lane;
    const V* x = reinterpret_cast<const V*>(static_cast<const T*>(a.token_rows) + t * a.ldt);
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (k0 + 32 * u < n) v[u] = x[k0 + 32 * u];
    for (int j0 = 0; j0 < a.k; j0 += 32) {
        const int64_t p = lane_row(a, t, j0);
        for (unsigned todo = __ballot_sync(0xFFFFFFFFu, p >= 0); todo; todo &= todo - 1) {
            V* out = reinterpret_cast<V*>(static_cast<T*>(a.slot_out) + __shfl_sync(0xFFFFFFFFu, p, __ffs(todo) - 1) * a.ldso);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + 32 * u < n) out[k0 + 32 * u] = v[u];
        }
    }
}

// combine, and dispatch's gradient (without weights): a warp per token and U
// vectors of each lane, with the vectors of BATCH slots on their way.
template <typename T, int VEC, int U, int BATCH>
__global__ void __launch_bounds__(256) expert_join(MoveArgs a) {
    using Row = RowVectors<T, VEC, U>;
    using V = Vec<T, VEC>;
    wait_for_primary();
    const int lane = threadIdx.x & 31, n = a.H / VEC, parts = (n + 32 * U - 1) / (32 * U);
    const uint32_t item = blockIdx.x * 8u + (threadIdx.x >> 5);
    if (item >= static_cast<uint32_t>(a.T) * parts) return;
    const int64_t t = item / parts;
    const int k0 = static_cast<int>(item % parts) * 32 * U + lane;
    F2 s[Row::PAIRS];
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) s[p] = f2(0.f);
    for (int j0 = 0; j0 < a.k; j0 += 32) {
        const int64_t row = lane_row(a, t, j0);
        const float weight = lane_weight<T>(a, t, j0);
        unsigned todo = __ballot_sync(0xFFFFFFFFu, row >= 0);
        while (todo) {
            Row x[BATCH];
            float w[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int j = todo ? __ffs(todo) - 1 : 0;
                const V* from = reinterpret_cast<const V*>(static_cast<const T*>(a.slot_rows) + __shfl_sync(0xFFFFFFFFu, row, j) * a.lds);
                w[b] = __shfl_sync(0xFFFFFFFFu, weight, j);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[b].v[u] = V{};
                    if (todo && k0 + 32 * u < n) load_now(x[b].v[u], from + k0 + 32 * u);
                }
                if (!todo) w[b] = 0.f;
                todo &= todo - 1;
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int p = 0; p < Row::PAIRS; ++p) s[p] = fma2(f2(w[b]), x[b].pair(p), s[p]);
        }
    }
    Row o;
    V* y = reinterpret_cast<V*>(static_cast<T*>(a.token_out) + t * a.ldto);
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) o.set(p, s[p]);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (k0 + 32 * u < n) y[k0 + 32 * u] = o.v[u];
}

// The row of a slot; -1 for none.
__device__ __forceinline__ int64_t slot_row(const MoveArgs& a, int64_t slot) {
    const int64_t p = a.positions[slot];
    return p < a.R ? p : -1;
}

// dispatch of narrow rows, dealt out by the vector: it is read once and written to all its rows.  The
// first blocks clear rows.
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(256) expert_spread_narrow(MoveArgs a) {
    using V = Vec<T, VEC>;
    wait_for_primary();
    if (static_cast<int>(blockIdx.x) < a.clearing) return clear_rows<T, VEC>(a, (blockIdx.x * 8ll + (threadIdx.x >> 5)) * EXPERT_CLEAR);
    const Dealt<U> mine(a.deal, blockIdx.x - a.clearing);
    V v[U];
    uint32_t at[U];
    int64_t t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        t[u] = mine.get(a.deal, u, at + u);
        if (t[u] < a.T) v[u] = reinterpret_cast<const V*>(static_cast<const T*>(a.token_rows) + t[u] * a.ldt)[at[u]];
    }
    for (int j = 0; j < a.k; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t p = t[u] < a.T ? slot_row(a, t[u] * a.k + j) : -1;
            if (p >= 0) reinterpret_cast<V*>(static_cast<T*>(a.slot_out) + p * a.ldso)[at[u]] = v[u];
        }
}

// combine of narrow rows, dealt out by the vector.
template <typename T, int VEC, int U, int BATCH>
__global__ void __launch_bounds__(256) expert_join_narrow(MoveArgs a) {
    using Row = RowVectors<T, VEC, U>;
    using V = Vec<T, VEC>;
    wait_for_primary();
    const Dealt<U> mine(a.deal, blockIdx.x);
    uint32_t at[U];
    int64_t t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] = mine.get(a.deal, u, at + u);
    F2 s[Row::PAIRS];
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) s[p] = f2(0.f);
    for (int j0 = 0; j0 < a.k; j0 += BATCH) {
        Row x[BATCH];
        float w[BATCH][U];
        int64_t row[BATCH][U];
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = j0 + b < a.k && t[u] < a.T;
                row[b][u] = in ? slot_row(a, t[u] * a.k + j0 + b) : -1;
                w[b][u] = in && a.weights && row[b][u] >= 0 ? load_w<T>(a.weights, a.w32, t[u] * a.k + j0 + b) : 1.f;
            }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[b].v[u] = V{};
                if (row[b][u] >= 0) load_now(x[b].v[u], reinterpret_cast<const V*>(static_cast<const T*>(a.slot_rows) + row[b][u] * a.lds) + at[u]);
            }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int p = 0; p < Row::PAIRS; ++p)
                s[p] = fma2(VEC == 1 ? f2(w[b][2 * p % U], w[b][(2 * p + 1) % U]) : f2(w[b][2 * p / VEC]), x[b].pair(p), s[p]);
    }
    Row o;
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) o.set(p, s[p]);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (t[u] < a.T) reinterpret_cast<V*>(static_cast<T*>(a.token_out) + t[u] * a.ldto)[at[u]] = o.v[u];
}

// combine's gradients: LANES lanes of a warp per token for narrow rows, else
// `share` warps of a block, each every share-th stretch of U vectors of each
// lane; BATCH slots at a time.  The sums over a row are put together lane by
// lane, then warp by warp.  The first blocks clear rows.
template <typename T, int VEC, int U, int BATCH, int LANES>
__global__ void __launch_bounds__(256) expert_join_bwd(MoveArgs a) {
    using Row = RowVectors<T, VEC, U>;
    using V = Vec<T, VEC>;
    static_assert(BATCH <= LANES);
    constexpr unsigned ALL = 0xFFFFFFFFu;
    __shared__ float part[8][BATCH];
    wait_for_primary();
    const int lane = threadIdx.x & (LANES - 1), warp = threadIdx.x >> 5, n = a.H / VEC;
    if (static_cast<int>(blockIdx.x) < a.clearing) return clear_rows<T, VEC>(a, (blockIdx.x * 8ll + warp) * EXPERT_CLEAR);
    const int64_t block = static_cast<int64_t>(blockIdx.x) - a.clearing;
    const int64_t t = LANES < 32 ? block * (256 / LANES) + threadIdx.x / LANES : block * (8 / a.share) + warp / a.share;
    const bool here = t < a.T, lead = LANES < 32 || warp % a.share == 0;
    const int first = (LANES < 32 ? 0 : warp % a.share * 32 * U) + lane, step = LANES < 32 ? LANES * U : a.share * 32 * U;
    const V* dy = reinterpret_cast<const V*>(static_cast<const T*>(a.token_rows) + t * a.ldt);
    for (int j0 = 0; j0 < a.k; j0 += BATCH) {
        const bool mine_in = here && lane < BATCH && j0 + lane < a.k;
        const int64_t row = mine_in ? slot_row(a, t * a.k + j0 + lane) : -1;
        const float weight = mine_in && a.weights ? load_w<T>(a.weights, a.w32, t * a.k + j0 + lane) : 1.f;
        const V* from[BATCH];
        V* to[BATCH];
        F2 w[BATCH], dot[BATCH];
        bool any = false;
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int64_t r = __shfl_sync(ALL, row, b, LANES);
            from[b] = r >= 0 && a.weights_out ? reinterpret_cast<const V*>(static_cast<const T*>(a.slot_rows) + r * a.lds) : nullptr;
            to[b] = r >= 0 && a.slot_out ? reinterpret_cast<V*>(static_cast<T*>(a.slot_out) + r * a.ldso) : nullptr;
            w[b] = f2(__shfl_sync(ALL, weight, b, LANES));
            dot[b] = f2(0.f);
            any |= r >= 0;
        }
        if (any)
            for (int k0 = first; k0 < n; k0 += step) {
                Row d, y[BATCH];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    d.v[u] = V{};
                    if (k0 + LANES * u < n) d.v[u] = dy[k0 + LANES * u];
                }
#pragma unroll
                for (int b = 0; b < BATCH; ++b)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        y[b].v[u] = V{};
                        if (from[b] && k0 + LANES * u < n) load_now(y[b].v[u], from[b] + k0 + LANES * u);
                    }
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
#pragma unroll
                    for (int p = 0; p < Row::PAIRS; ++p) dot[b] = fma2(d.pair(p), y[b].pair(p), dot[b]);
                    if (!to[b]) continue;
                    Row o;
#pragma unroll
                    for (int p = 0; p < Row::PAIRS; ++p) o.set(p, mul2(w[b], d.pair(p)));
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (k0 + LANES * u < n) to[b][k0 + LANES * u] = o.v[u];
                }
            }
        if (!a.weights_out) continue;
        float mine = 0.f;  // lane b: the batch's slot b
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            float v = from[b] ? lo(dot[b]) + hi(dot[b]) : 0.f;  // without a row not 0 dy: dy may be infinite or NaN
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
            if (lane == b) mine = v;
        }
        if (LANES == 32 && a.share > 1) {
            __syncthreads();
            if (lane < BATCH) part[warp][lane] = mine;
            __syncthreads();
            if (lead && lane < BATCH)
                for (int s = 1; s < a.share; ++s) mine += part[warp + s][lane];
        }
        if (mine_in && lead) {
            const int64_t slot = t * a.k + j0 + lane;
            if (a.w32)
                static_cast<float*>(a.weights_out)[slot] = mine;
            else
                static_cast<T*>(a.weights_out)[slot] = from_f32<T>(mine);
        }
    }
}

// ---------------------------------------------------------------- host

lce_status_t plan_sizes(int64_t T, int64_t k, int64_t E, int64_t align, int64_t* rows) {
    if (T < 0 || k <= 0 || E <= 0 || align <= 0) return LCE_ERR_INVALID_ARG;
    if (E > LCE_BALANCE_MAX_E || k > E || align > LCE_EXPERT_MAX_ALIGN || T > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    const int64_t most = (T * k + E * (align - 1) + align - 1) / align * align;
    if (most > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    if (rows) *rows = most;
    return LCE_OK;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t plan_space(int64_t T, int64_t k, int64_t E, SortShape* shape, void* ws) {
    const int64_t n = T * k, blocks = sort_blocks(n);
    const size_t hist = 1024 + align256(static_cast<size_t>(blocks) * 4);
    if (shape) {
        uint8_t* w = static_cast<uint8_t*>(ws);
        shape->n = n;
        shape->blocks = static_cast<int32_t>(blocks);
        shape->per = (n + blocks - 1) / blocks;
        shape->bins = static_cast<int32_t>(E + 1);
        shape->bad = reinterpret_cast<int32_t*>(w + 1024);
        shape->hist = reinterpret_cast<int32_t*>(w + hist);
    }
    return hist + static_cast<size_t>(blocks) * (E + 1) * 4;
}

struct MoveIn {
    int64_t T, k, H, R;
    int dtype, wtype;
    const int32_t* positions;
};

lce_status_t move_args(const MoveIn& in, MoveArgs* a) {
    if (in.T < 0 || in.k <= 0 || in.H <= 0 || in.R < 0 || !dtype_known(in.dtype) || !dtype_known(in.wtype)) return LCE_ERR_INVALID_ARG;
    if (in.wtype != in.dtype && in.wtype != LCE_F32) return LCE_ERR_UNSUPPORTED;
    if (in.k > LCE_BALANCE_MAX_E || in.H > LCE_NORM_MAX_H || in.T > INT32_MAX || in.R > INT32_MAX || in.T * in.k > INT32_MAX)
        return LCE_ERR_UNSUPPORTED;
    if (in.T && (!in.positions || !aligned_to(in.positions, 4))) return LCE_ERR_INVALID_ARG;
    *a = MoveArgs{};
    a->positions = in.positions;
    a->T = in.T;
    a->R = in.R;
    a->k = static_cast<int32_t>(in.k);
    a->H = static_cast<int32_t>(in.H);
    a->w32 = in.wtype == LCE_F32;
    return LCE_OK;
}

bool rows_ok(const void* p, int64_t n, int64_t ld, int64_t H, int dtype) {
    return ld >= H && (n == 0 || (p && aligned_to(p, dtype_bytes(dtype))));
}

// Whether rows can be read and written in vectors of `vec` elements, `bytes` bytes.
bool in_vectors(const MoveArgs& a, int vec, int bytes) {
    return a.H % vec == 0 && a.ldt % vec == 0 && a.lds % vec == 0 && a.ldto % vec == 0 && a.ldso % vec == 0 &&
           aligned_to(a.token_rows, bytes) && aligned_to(a.slot_rows, bytes) && aligned_to(a.token_out, bytes) &&
           aligned_to(a.slot_out, bytes);
}

enum class Move { SPREAD, JOIN, JOIN_BWD };

// Vectors of a lane: as many as 16 bytes hold of single elements, and with
// 16-byte vectors `wide` of them where that still gives every SM its warps.
template <typename T, int VEC>
lce_status_t move_as(MoveArgs a, Move what, cudaStream_t s) {
    // (16384 tokens of 8 slots, 2048 bf16: combine with two vectors and eight slots at a time 4% faster than with one and
    // eight or four and four; single elements with four slots, not eight: 4099 x 1601 fp16 in training 95 us, not 138;
    // their gradients with four elements a lane 23 us, with two 28, with eight 26.  Rows on any boundary put together in
    // registers from two aligned vectors: dispatch 15 us, not 12, combine 32, not 14)
    constexpr bool V16 = VEC * sizeof(T) == 16;
    constexpr int NARROW = VEC == 1 ? 8 : V16 ? 1 : 4, WIDE = V16 ? 4 : NARROW, BWD = VEC == 1 ? 4 : V16 ? 1 : 2, JOIN = V16 ? 2 : NARROW;
    constexpr int BATCH = V16 ? 8 : 4;
    const int64_t n = a.H / VEC, vectors = a.T * n;
    auto parts = [&](int u) { return (n + 32 * u - 1) / (32 * u); };
    // rows of less than half a warp of 16-byte vectors are dealt out by the vector (65536 tokens of 4 slots, 64 bf16:
    // dispatch 10.3 us, combine 14.5; a warp to a token 16.5 and 40.6), in combine of less than a warp (20000 tokens of 4
    // slots, 192: 6.9 and 9.1), with one or two slots than two (60000 of one, 192: 9.0 and 15.2; 40000 of 2, 512: 27.3 and
    // 25.8).  The gradients take parts of a warp, up to a warp's width with one or two slots (60000 of one, 192: 18.3 us,
    // a warp 27.3; 20000 of 4, 192: 18.0 and 17.2)
    const bool narrow = V16 && (n <= 16 || (what == Move::JOIN && (n < 32 || (n < 64 && a.k <= 2))));
    const bool wide = !narrow && what == Move::SPREAD && a.T * parts(WIDE) >= 152 * 32, halves = n > 16 && n <= 32 && a.k <= 2;
    const int lanes = !V16 || (n > 16 && !halves) ? 32 : n > 8 ? 16 : 8;
    int64_t work = 0;  // blocks
    if (what == Move::JOIN_BWD) {
        a.share = 1;
        while (a.share < 8 && a.share < parts(BWD) && a.T * a.share < 152 * 32) a.share *= 2;
        const int64_t tokens = lanes < 32 ? 256 / lanes : 8 / a.share;
        work = (a.T + tokens - 1) / tokens;
    } else if (narrow) {
        work = (vectors + 256 * JOIN - 1) / (256 * JOIN);
        a.deal = deal_of(n);
    } else {
        work = (a.T * parts(what == Move::JOIN ? JOIN : wide ? WIDE : NARROW) + 7) / 8;
        if (work * 8 > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    }
    const int64_t clearing = what != Move::JOIN && a.slot_out ? (a.R + 8 * EXPERT_CLEAR - 1) / (8 * EXPERT_CLEAR) : 0;
    const int64_t blocks = work + clearing;
    if (blocks == 0) return LCE_OK;
    if (blocks > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    a.clearing = static_cast<int32_t>(clearing);
    const unsigned grid = static_cast<unsigned>(blocks);
    // no more slots at a time than a token has (16384 tokens of one, 2048 bf16: combine 28.6 us, with eight 38.8, its
    // gradients 35.6 and, with four, 41.9)
    auto by_slots = [&](auto launch) -> lce_status_t {
        if (a.k <= 2) return launch(std::integral_constant<int, 2>{});
        if constexpr (BATCH > 4)
            if (a.k > 4) return launch(std::integral_constant<int, BATCH>{});
        return launch(std::integral_constant<int, 4>{});
    };
    if (what == Move::JOIN_BWD) {
        return by_slots([&](auto batch) -> lce_status_t {
            constexpr int B = decltype(batch)::value;
            if constexpr (V16) {
                constexpr int FEW = B < 4 ? B : 4;
                if constexpr (B == 2)
                    if (halves) {
                        LCE_PROFILED(launch_after(expert_join_bwd<T, VEC, 2, B, 16>, dim3(grid), 256, 0, s, a));
                        return LCE_OK;
                    }
                if (lanes < 32) {
                    if (lanes == 16)
                        LCE_PROFILED(launch_after(expert_join_bwd<T, VEC, BWD, FEW, 16>, dim3(grid), 256, 0, s, a));
                    else
                        LCE_PROFILED(launch_after(expert_join_bwd<T, VEC, BWD, FEW, 8>, dim3(grid), 256, 0, s, a));
                    return LCE_OK;
                }
            }
            LCE_PROFILED(launch_after(expert_join_bwd<T, VEC, BWD, B, 32>, dim3(grid), 256, 0, s, a));
            return LCE_OK;
        });
    } else if (what == Move::JOIN) {
        return by_slots([&](auto batch) -> lce_status_t {
            constexpr int B = decltype(batch)::value;
            if constexpr (V16) {
                if (narrow) {
                    LCE_PROFILED(launch_after(expert_join_narrow<T, VEC, JOIN, B>, dim3(grid), 256, 0, s, a));
                    return LCE_OK;
                }
            }
            LCE_PROFILED(launch_after(expert_join<T, VEC, JOIN, B>, dim3(grid), 256, 0, s, a));
            return LCE_OK;
        });
    } else {
        if constexpr (V16) {
            if (narrow) {
                LCE_PROFILED(launch_after(expert_spread_narrow<T, VEC, JOIN>, dim3(grid), 256, 0, s, a));
                return LCE_OK;
            }
        }
        if (wide)
            LCE_PROFILED(launch_after(expert_spread<T, VEC, WIDE>, dim3(grid), 256, 0, s, a));
        else
            LCE_PROFILED(launch_after(expert_spread<T, VEC, NARROW>, dim3(grid), 256, 0, s, a));
    }
    return LCE_OK;
}

lce_status_t move(const MoveArgs& a, int dtype, Move what, lce_stream_t stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        constexpr int V = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
        if (in_vectors(a, V, 16)) return move_as<T, V>(a, what, s);
        return V4 > 1 && in_vectors(a, V4, 4) ? move_as<T, V4>(a, what, s) : move_as<T, 1>(a, what, s);
    });
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status_t lce_expert_rows(int64_t T, int64_t k, int64_t E, int64_t align, int64_t* rows) {
    if (!rows) return LCE_ERR_INVALID_ARG;
    return plan_sizes(T, k, E, align, rows);
}

lce_status_t lce_expert_plan_workspace_size(int64_t T, int64_t k, int64_t E, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = plan_sizes(T, k, E, 1, nullptr);
    if (st == LCE_OK) *bytes = plan_space(T, k, E, nullptr, nullptr);
    return st;
}

lce_status_t lce_expert_plan(int64_t T, int64_t k, int64_t E, int64_t align, const void* experts, int index_bytes,
                             const uint8_t* mask, int32_t* positions, int32_t* slots, int64_t* counts,
                             int64_t* offsets, void* ws, size_t ws_bytes, lce_stream_t stream) {
    int64_t rows = 0;
    const lce_status_t st = plan_sizes(T, k, E, align, &rows);
    if (st != LCE_OK) return st;
    if (index_bytes != 4 && index_bytes != 8) return LCE_ERR_INVALID_ARG;
    if (T && (!experts || !aligned_to(experts, index_bytes) || !positions || !aligned_to(positions, 4))) return LCE_ERR_INVALID_ARG;
    if ((rows && !slots) || !aligned_to(slots, 4) || !counts || !aligned_to(counts, 8) || !offsets || !aligned_to(offsets, 8))
        return LCE_ERR_INVALID_ARG;
    if (!ws || !aligned_to(ws, 256)) return LCE_ERR_INVALID_ARG;
    SortShape shape{};
    if (ws_bytes < plan_space(T, k, E, &shape, ws)) return LCE_ERR_WORKSPACE;
    const PlanArgs a{experts, index_bytes == 8, mask, static_cast<int32_t>(E), static_cast<int32_t>(k), static_cast<int32_t>(align),
                     positions, slots, counts, offsets, static_cast<int32_t>(rows), &static_cast<WsHeader*>(ws)->status};
    return sort_by(a, shape, reinterpret_cast<cudaStream_t>(stream));
}

lce_status_t lce_expert_dispatch(int64_t T, int64_t k, int64_t H, int64_t R, int dtype, const void* x, int64_t ldx,
                                 const int32_t* positions, const int32_t* slots, void* rows, int64_t ldr,
                                 lce_stream_t stream) {
    MoveArgs a;
    const lce_status_t st = move_args({T, k, H, R, dtype, dtype, positions}, &a);
    if (st != LCE_OK) return st;
    if (!rows_ok(x, T, ldx, H, dtype) || !rows_ok(rows, R, ldr, H, dtype) || (R && (!slots || !aligned_to(slots, 4))))
        return LCE_ERR_INVALID_ARG;
    a.slots = slots;
    a.token_rows = x;
    a.ldt = ldx;
    a.slot_out = rows;
    a.ldso = ldr;
    return move(a, dtype, Move::SPREAD, stream);
}

lce_status_t lce_expert_dispatch_backward(int64_t T, int64_t k, int64_t H, int64_t R, int dtype, const void* grad_rows,
                                          int64_t ldr, const int32_t* positions, void* grad_x, int64_t ldx,
                                          lce_stream_t stream) {
    return lce_expert_combine(T, k, H, R, dtype, dtype, grad_rows, ldr, nullptr, positions, grad_x, ldx, stream);
}

lce_status_t lce_expert_combine(int64_t T, int64_t k, int64_t H, int64_t R, int dtype, int wtype, const void* rows,
                                int64_t ldr, const void* weights, const int32_t* positions, void* y, int64_t ldy,
                                lce_stream_t stream) {
    MoveArgs a;
    const lce_status_t st = move_args({T, k, H, R, dtype, wtype, positions}, &a);
    if (st != LCE_OK) return st;
    if (!rows_ok(y, T, ldy, H, dtype) || !rows_ok(rows, R, ldr, H, dtype) || !aligned_to(weights, dtype_bytes(wtype)))
        return LCE_ERR_INVALID_ARG;
    a.slot_rows = rows;
    a.lds = ldr;
    a.weights = weights;
    a.token_out = y;
    a.ldto = ldy;
    return move(a, dtype, Move::JOIN, stream);
}

lce_status_t lce_expert_combine_backward(int64_t T, int64_t k, int64_t H, int64_t R, int dtype, int wtype,
                                         const void* grad_y, int64_t ldg, const void* rows, int64_t ldr,
                                         const void* weights, const int32_t* positions, const int32_t* slots,
                                         void* grad_rows, int64_t ldgr, void* grad_weights, lce_stream_t stream) {
    MoveArgs a;
    const lce_status_t st = move_args({T, k, H, R, dtype, wtype, positions}, &a);
    if (st != LCE_OK) return st;
    if (!rows_ok(grad_y, T, ldg, H, dtype) || (grad_weights && !rows_ok(rows, R, ldr, H, dtype)) ||
        !aligned_to(weights, dtype_bytes(wtype)) || !aligned_to(grad_weights, dtype_bytes(wtype)))
        return LCE_ERR_INVALID_ARG;
    if (grad_rows && (!rows_ok(grad_rows, R, ldgr, H, dtype) || (R && (!slots || !aligned_to(slots, 4))))) return LCE_ERR_INVALID_ARG;
    if (!grad_rows && !grad_weights) return LCE_OK;
    a.slots = slots;
    a.token_rows = grad_y;
    a.ldt = ldg;
    a.slot_rows = grad_weights ? rows : nullptr;
    a.lds = grad_weights ? ldr : ldg;
    a.weights = weights;
    a.slot_out = grad_rows;
    a.ldso = grad_rows ? ldgr : ldg;
    a.weights_out = grad_weights;
    return move(a, dtype, Move::JOIN_BWD, stream);
}

}  // extern "C"
