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
};

__device__ __forceinline__ int64_t token_at(const void* tokens, bool idx64, int64_t i) {
    return idx64 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// A block per token.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) emb_fwd(EmbFwd<T> a) {
    using V = Vec<T, VEC>;
    const int64_t i = blockIdx.x;
    const int64_t v = token_at(a.tokens, a.idx64, i);
    const bool in = v >= 0 && v < a.V;
    const float fill = v == a.padding ? 0.f : __int_as_float(0x7fffffff);
    if (!in && v != a.padding && a.status && threadIdx.x == 0) atomicOr(a.status, STATUS_INDEX);
    const V* w = reinterpret_cast<const V*>(a.w + (in ? v : 0) * a.ldw);
    V* y = reinterpret_cast<V*>(a.y + i * a.ldy);
    for (int k = threadIdx.x; k < a.H / VEC; k += blockDim.x) {
        V x{};
        if (in) x = w[k];
#pragma unroll
        for (int e = 0; e < VEC; ++e) x.set(e, in ? x.f(e) * a.scale : fill);
        y[k] = x;
    }
}

// ---------------------------------------------------------------- the gradient

// The workspace.
struct EmbSpace {
    WsHeader* hdr;
    int32_t *bad, *hist, *keys[2], *rows[2];
};

// The first digit: tokens as they come.  V stands for the ones to leave out.
struct FirstDigit {
    static constexpr bool SEGMENTS = false;
    const void* tokens;
    bool idx64;
    int32_t V, mask;
    int64_t padding;
    int32_t *keys, *rows;
    unsigned* stat;
    __device__ __forceinline__ int32_t key(int64_t i, bool* bad) const {
        const int64_t v = token_at(tokens, idx64, i);
        if (v == padding) return V;
        if (v >= 0 && v < V) return static_cast<int32_t>(v);
        *bad = true;
        return V;
    }
    __device__ __forceinline__ int32_t digit(int64_t i, bool* bad) const { return key(i, bad) & mask; }
    __device__ __forceinline__ void put(int64_t i, int32_t, int32_t at) const {
        bool bad;
        keys[at] = key(i, &bad);
        rows[at] = static_cast<int32_t>(i);
    }
    __device__ __forceinline__ void status(int any) const { *stat = any ? STATUS_INDEX : 0u; }
};

// A later digit.
struct NextDigit {
    static constexpr bool SEGMENTS = false;
    const int32_t *from_keys, *from_rows;
    int32_t shift, mask;
    int32_t *keys, *rows;
    __device__ __forceinline__ int32_t digit(int64_t i, bool*) const { return from_keys[i] >> shift & mask; }
    __device__ __forceinline__ void put(int64_t i, int32_t, int32_t at) const {
        keys[at] = from_keys[i];
        rows[at] = from_rows[i];
    }
    __device__ __forceinline__ void status(int) const {}
};

template <typename T>
struct EmbBwd {
    const T* dy;
    int64_t ldd, N, V;
    float scale;
    const int32_t *keys, *rows;  // sorted
    void* dw;
    int64_t lddw;
    bool add;
    int32_t H;
};

// A block per vocabulary row: its place among the sorted tokens, then its rows.
template <typename T, typename W>
__global__ void __launch_bounds__(256) emb_bwd_row(EmbBwd<T> a) {
    const int64_t v = blockIdx.x;
    wait_for_primary();
    int64_t lo = 0, hi = a.N;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.keys[mid] < v)
            lo = mid + 1;
        else
            hi = mid;
    }
    W* dw = static_cast<W*>(a.dw) + v * a.lddw;
    if (a.add && (lo == a.N || a.keys[lo] != v)) return;
    for (int h = threadIdx.x; h < a.H; h += blockDim.x) {
        float s = 0.f;
        for (int64_t i = lo; i < a.N && a.keys[i] == v; ++i) s += to_f32(a.dy[a.rows[i] * a.ldd + h]);
        s *= a.scale;
        if (a.add) s += to_f32(dw[h]);
        dw[h] = from_f32<W>(s);
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

size_t emb_space(int64_t N, int64_t V, EmbSpace* e, void* ws) {
    const Digits d = digits_of(V);
    const size_t blocks = static_cast<size_t>(sort_blocks(N)), items = align256(static_cast<size_t>(N) * 4);
    const size_t hist = 1024 + align256(blocks * 4);
    const size_t keys = hist + align256(blocks * 4 << d.bits);
    if (e) {
        uint8_t* w = static_cast<uint8_t*>(ws);
        e->hdr = reinterpret_cast<WsHeader*>(w);
        e->bad = reinterpret_cast<int32_t*>(w + 1024);
        e->hist = reinterpret_cast<int32_t*>(w + hist);
        for (int k = 0; k < 2; ++k) {
            e->keys[k] = reinterpret_cast<int32_t*>(w + keys + 2 * k * items);
            e->rows[k] = reinterpret_cast<int32_t*>(w + keys + (2 * k + 1) * items);
        }
    }
    return keys + 4 * items;
}

// The sorted tokens: their place in e->keys and e->rows.
lce_status_t emb_sort(int64_t N, int64_t V, const void* tokens, bool idx64, int64_t padding, const EmbSpace& e, int* where,
                      cudaStream_t s) {
    const Digits d = digits_of(V);
    SortShape shape{};
    shape.n = N;
    shape.bins = 1 << d.bits;
    shape.blocks = static_cast<int32_t>(sort_blocks(N));
    shape.per = (N + shape.blocks - 1) / shape.blocks;
    shape.hist = e.hist;
    shape.bad = e.bad;
    const FirstDigit first{tokens, idx64, static_cast<int32_t>(V), shape.bins - 1, padding, e.keys[0], e.rows[0], &e.hdr->status};
    lce_status_t st = sort_by(first, shape, true, s);
    shape.bad = nullptr;
    for (int p = 1; p < d.passes && st == LCE_OK; ++p) {
        const int from = (p - 1) & 1, to = p & 1;
        st = sort_by(NextDigit{e.keys[from], e.rows[from], p * d.bits, shape.bins - 1, e.keys[to], e.rows[to]}, shape, false, s);
    }
    *where = (d.passes - 1) & 1;
    return st;
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
        constexpr int VEC = vec16<T>();
        const EmbFwd<T> a{tokens, index_bytes == 8, static_cast<const T*>(weight), ldw, N, V, padding_token, scale,
                          static_cast<T*>(y), ldy, static_cast<unsigned*>(status), static_cast<int32_t>(H)};
        const unsigned blocks = static_cast<unsigned>(N);
        if (H % VEC == 0 && ldw % VEC == 0 && ldy % VEC == 0 && aligned_to(weight, 16) && aligned_to(y, 16))
            LCE_PROFILED(emb_fwd<T, VEC><<<blocks, 256, 0, s>>>(a));
        else
            LCE_PROFILED(emb_fwd<T, 1><<<blocks, 256, 0, s>>>(a));
        return LCE_OK;
    });
}

lce_status_t lce_embedding_workspace_size(int64_t N, int64_t V, int64_t H, size_t* bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    const lce_status_t st = emb_sizes(N, V, H);
    if (st == LCE_OK) *bytes = emb_space(N, V, nullptr, nullptr);
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
    if (ws_bytes < emb_space(N, V, &e, ws)) return LCE_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int where = 0;
    const lce_status_t sorted = emb_sort(N, V, tokens, index_bytes == 8, padding_token, e, &where, s);
    if (sorted != LCE_OK) return sorted;
    return with_dtype(dtype, [&](auto t) -> lce_status_t {
        using T = decltype(t);
        const EmbBwd<T> a{static_cast<const T*>(grad_y), ldg, N, V, scale, e.keys[where], e.rows[where], grad_weight, ldgw,
                          add, static_cast<int32_t>(H)};
        const dim3 blocks(static_cast<unsigned>(V));
        if (gtype == LCE_F32)
            LCE_PROFILED(launch_after(emb_bwd_row<T, float>, blocks, 256, 0, s, a));
        else
            LCE_PROFILED(launch_after(emb_bwd_row<T, T>, blocks, 256, 0, s, a));
        return LCE_OK;
    });
}

}  // extern "C"
