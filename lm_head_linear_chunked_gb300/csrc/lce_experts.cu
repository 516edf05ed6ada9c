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
};

__device__ __forceinline__ int64_t row_of(const MoveArgs& a, int64_t slot) {
    const int64_t p = a.positions[slot];
    return p < a.R ? p : -1;  // a plan of other rows
}

template <typename T>
__device__ __forceinline__ float weight_of(const MoveArgs& a, int64_t slot) {
    return a.weights ? load_w<T>(a.weights, a.w32, slot) : 1.f;
}

// Block T + r: row r of the sorted ones is zero where no slot takes it.
template <typename T, int VEC>
__device__ __forceinline__ void zero_row(const MoveArgs& a, int64_t r) {
    if (a.slots[r] >= 0) return;
    Vec<T, VEC>* out = reinterpret_cast<Vec<T, VEC>*>(static_cast<T*>(a.slot_out) + r * a.ldso);
    for (int i = threadIdx.x; i < a.H / VEC; i += blockDim.x) out[i] = Vec<T, VEC>{};
}

// dispatch: a block per token.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) expert_spread(MoveArgs a) {
    const int64_t t = blockIdx.x;
    if (t >= a.T) return zero_row<T, VEC>(a, t - a.T);
    using V = Vec<T, VEC>;
    const V* x = reinterpret_cast<const V*>(static_cast<const T*>(a.token_rows) + t * a.ldt);
    for (int i = threadIdx.x; i < a.H / VEC; i += blockDim.x) {
        const V v = x[i];
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = row_of(a, t * a.k + j);
            if (p >= 0) reinterpret_cast<V*>(static_cast<T*>(a.slot_out) + p * a.ldso)[i] = v;
        }
    }
}

// combine, and dispatch's gradient (without weights): a block per token.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) expert_join(MoveArgs a) {
    const int64_t t = blockIdx.x;
    using V = Vec<T, VEC>;
    V* y = reinterpret_cast<V*>(static_cast<T*>(a.token_out) + t * a.ldto);
    for (int i = threadIdx.x; i < a.H / VEC; i += blockDim.x) {
        float s[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int64_t p = row_of(a, t * a.k + j);
            if (p < 0) continue;
            const float w = weight_of<T>(a, t * a.k + j);
            const V v = reinterpret_cast<const V*>(static_cast<const T*>(a.slot_rows) + p * a.lds)[i];
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] = fmaf(w, v.f(e), s[e]);
        }
        V o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.set(e, s[e]);
        y[i] = o;
    }
}

// combine's gradients: a block per token, a slot after the other.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) expert_join_bwd(MoveArgs a) {
    __shared__ float part[8];
    const int64_t t = blockIdx.x;
    if (t >= a.T) return zero_row<T, VEC>(a, t - a.T);
    using V = Vec<T, VEC>;
    const V* dy = reinterpret_cast<const V*>(static_cast<const T*>(a.token_rows) + t * a.ldt);
    for (int j = 0; j < a.k; ++j) {
        const int64_t slot = t * a.k + j, p = row_of(a, slot);
        float s = 0.f;
        if (p >= 0) {
            const float w = weight_of<T>(a, slot);
            const V* y = reinterpret_cast<const V*>(static_cast<const T*>(a.slot_rows) + p * a.lds);
            V* out = a.slot_out ? reinterpret_cast<V*>(static_cast<T*>(a.slot_out) + p * a.ldso) : nullptr;
            for (int i = threadIdx.x; i < a.H / VEC; i += blockDim.x) {
                const V d = dy[i];
                V o;
                if (a.weights_out) {
                    const V v = y[i];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) s = fmaf(d.f(e), v.f(e), s);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) o.set(e, w * d.f(e));
                if (out) out[i] = o;
            }
        }
        if (!a.weights_out) continue;
        s = warp_sum(s);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            s = 0.f;
            for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += part[w];
            if (a.w32)
                static_cast<float*>(a.weights_out)[slot] = s;
            else
                static_cast<T*>(a.weights_out)[slot] = from_f32<T>(s);
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

// Whether rows can be read and written in vectors of 16 bytes.
template <typename T>
bool wide(const MoveArgs& a) {
    constexpr int V = vec16<T>();
    return a.H % V == 0 && a.ldt % V == 0 && a.lds % V == 0 && a.ldto % V == 0 && a.ldso % V == 0 && aligned_to(a.token_rows, 16) &&
           aligned_to(a.slot_rows, 16) && aligned_to(a.token_out, 16) && aligned_to(a.slot_out, 16);
}

enum class Move { SPREAD, JOIN, JOIN_BWD };

template <typename T, int VEC>
lce_status_t move_as(const MoveArgs& a, Move what, cudaStream_t s) {
    const int64_t blocks = a.T + (what != Move::JOIN && a.slot_out ? a.R : 0);
    if (blocks == 0) return LCE_OK;
    if (blocks > INT32_MAX) return LCE_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (what == Move::SPREAD)
        LCE_PROFILED(expert_spread<T, VEC><<<grid, 256, 0, s>>>(a));
    else if (what == Move::JOIN)
        LCE_PROFILED(expert_join<T, VEC><<<grid, 256, 0, s>>>(a));
    else
        LCE_PROFILED(expert_join_bwd<T, VEC><<<grid, 256, 0, s>>>(a));
    return LCE_OK;
}

lce_status_t move(const MoveArgs& a, int dtype, Move what, lce_stream_t stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        return wide<T>(a) ? move_as<T, vec16<T>()>(a, what, s) : move_as<T, 1>(a, what, s);
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
    return sort_by(a, shape, true, reinterpret_cast<cudaStream_t>(stream));
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
