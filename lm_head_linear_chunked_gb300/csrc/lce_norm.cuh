// Layer norm of the rows that the head reads, forward and backward.
//
//   mean = sum_h x / H,  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - mean_h(g) - xh mean_h(g xh))
//   dw = sum_r dy xh,  db = sum_r dy
//
// All sums are FP32; the variance is summed from the centred values, so an
// offset of the row costs no digits.
#pragma once

#include <atomic>

#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {

// Parts of the weight gradient's sum over the rows: at most four blocks on each of 152 SMs.
constexpr int64_t NORM_PARTS = 608;
constexpr int NORM_BWD_STAGES = 3;
// Dynamic shared memory of a block; the widest ring takes 192 KB of it.
constexpr int NORM_SMEM_MAX = 224 * 1024;

// What a launch needs, by the element type (one translation unit each).
struct NormCall {
    const void *x, *dy, *w, *b;
    int64_t ldx, ldd, ldy;
    bool w32;
    float eps;
    void* y;
    float *mean_out, *rstd_out;
    const float *mean, *rstd;
    void *dw, *db;
    float* parts;       // [2, NORM_PARTS, H]
    int64_t rows;
    int32_t H;
    cudaStream_t s;
};
lce_status_t norm_forward_bf16(const NormCall& c);
lce_status_t norm_forward_f16(const NormCall& c);
lce_status_t norm_forward_f32(const NormCall& c);
lce_status_t norm_backward_bf16(const NormCall& c);
lce_status_t norm_backward_f16(const NormCall& c);
lce_status_t norm_backward_f32(const NormCall& c);

namespace {

// One value for the whole block: the sum of v over its threads, added in a
// fixed order.  `part` holds 32 floats and may be reused after the next
// barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5, l = threadIdx.x & 31;
    return warp_sum(l < warps ? part[l] : 0.f);
}

template <typename T>
struct NormFwd {
    const T* x;
    int64_t ldx;
    const void *w, *b;  // each nullable; fp32 with w32, else T
    bool w32;
    float eps;
    T* y;
    int64_t ldy;
    float *mean, *rstd;  // nullable
    int64_t rows;
    int32_t H;
};

template <typename T>
__device__ __forceinline__ float load_w(const void* w, bool w32, int64_t i) {
    return w32 ? static_cast<const float*>(w)[i] : to_f32(static_cast<const T*>(w)[i]);
}

// How a row is shared out.  Vector i of a thread is the row's vector
// i * TPR + t, with TPR threads to a row: the lanes of a warp, or all threads
// of a block.  The row stays in registers between the sums and the output, as
// pairs of FP32 values.
template <typename T, int VEC, int ITEMS>
struct RowRegs : RowVectors<T, VEC, ITEMS> {
    using Base = RowVectors<T, VEC, ITEMS>;
    using Base::v;
    static constexpr int PAIRS = Base::PAIRS;
    __device__ __forceinline__ void load(const T* row, int t, int tpr, int n) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            v[i] = Vec<T, VEC>{};
            if (i * tpr + t < n) v[i] = reinterpret_cast<const Vec<T, VEC>*>(row)[i * tpr + t];
        }
    }
    __device__ __forceinline__ void store(T* row, int t, int tpr, int n) const {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (i * tpr + t < n) reinterpret_cast<Vec<T, VEC>*>(row)[i * tpr + t] = v[i];
    }
    // x in the halves of pair p that lie inside the row, 0 in the others.
    static __device__ __forceinline__ F2 inside(int p, F2 x, int t, int tpr, int n) {
        const int a = VEC == 1 ? 2 * p : 2 * p / VEC, b = VEC == 1 ? 2 * p + 1 : 2 * p / VEC;
        return f2(a * tpr + t < n ? lo(x) : 0.f, b * tpr + t < n ? hi(x) : 0.f);
    }
};

// Narrow rows: a warp per row, four rows to a block, the row in registers.
// Nothing waits for another warp, and the many blocks keep the memory busy.
template <typename T, typename W, int VEC, int ITEMS>
__global__ void __launch_bounds__(128) norm_fwd_warp(NormFwd<T> a) {
    using Row = RowRegs<T, VEC, ITEMS>;
    const int t = threadIdx.x & 31;
    const int64_t r = blockIdx.x * 4ll + (threadIdx.x >> 5);
    if (r >= a.rows) return;
    const int n = a.H / VEC;
    const float inv = 1.f / static_cast<float>(a.H);
    Row x;
    x.load(a.x + r * a.ldx, t, 32, n);
    F2 d[Row::PAIRS], s = f2(0.f);
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) {
        d[p] = x.pair(p);
        s = add2(s, d[p]);
    }
    const float mean = warp_sum(lo(s) + hi(s)) * inv;
    F2 q = f2(0.f);
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) {
        d[p] = Row::inside(p, add2(d[p], f2(-mean)), t, 32, n);
        q = fma2(d[p], d[p], q);
    }
    const float rstd = rsqrtf(warp_sum(lo(q) + hi(q)) * inv + a.eps);
    RowRegs<W, VEC, ITEMS> w, b;
    if (a.w) w.load(static_cast<const W*>(a.w), t, 32, n);
    if (a.b) b.load(static_cast<const W*>(a.b), t, 32, n);
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) {
        F2 v = mul2(d[p], f2(rstd));
        if (a.w) v = mul2(v, w.pair(p));
        if (a.b) v = add2(v, b.pair(p));
        x.set(p, v);
    }
    x.store(a.y + r * a.ldy, t, 32, n);
    if (t == 0 && a.mean) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
    }
}

// Wide rows, many of them: a block takes R rows at a time and copies the
// next ones ahead, each thread its own vectors, so that only the sums over a
// row wait for the other warps, once per R rows: each warp centres its share
// of a row on the share's own mean, and the shares' means and squares are
// put together as  M2 = sum_w M2_w + sum_w n_w (mean_w - mean)^2  (Chan, Golub
// and LeVeque's joining of variances).
template <typename T, typename W, int VEC, int ITEMS, int R, int STAGES, int MAX_WARPS, int BLOCKS>
__global__ void __launch_bounds__(32 * MAX_WARPS, BLOCKS) norm_fwd_rows(NormFwd<T> a) {
    constexpr bool RING = sizeof(Vec<T, VEC>) >= 4;  // single 16-bit elements wait in registers
    using Row = RowRegs<T, VEC, ITEMS>;
    using V = Vec<T, VEC>;
    __shared__ float2 part[2][R][MAX_WARPS];
    extern __shared__ __align__(16) uint8_t dyn[];
    const int t = threadIdx.x, threads = blockDim.x, warp = t >> 5, warps = threads >> 5, lane = t & 31;
    const int n = a.H / VEC;
    const float inv = 1.f / static_cast<float>(a.H);
    V* ring = reinterpret_cast<V*>(dyn);  // [STAGES][R][ITEMS][threads]
    const int64_t groups = (a.rows + R - 1) / R;
    auto copy_group = [&](int64_t g, int stage) {
        if constexpr (RING) {
            if (g < groups)
#pragma unroll
                for (int k = 0; k < R; ++k)
                    if (g * R + k < a.rows) {
                        const V* x = reinterpret_cast<const V*>(a.x + (g * R + k) * a.ldx);
#pragma unroll
                        for (int i = 0; i < ITEMS; ++i)
                            if (i * threads + t < n)
                                copy_async<sizeof(V)>(ring + ((stage * R + k) * ITEMS + i) * threads + t,
                                                      x + i * threads + t);
                    }
            copy_async_commit();
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) copy_group(blockIdx.x + static_cast<int64_t>(k) * gridDim.x, k);
    RowRegs<W, VEC, ITEMS> w, b;
    if (a.w) w.load(static_cast<const W*>(a.w), t, threads, n);
    if (a.b) b.load(static_cast<const W*>(a.b), t, threads, n);
    // elements of a row in the share of a warp; each lane joins one warp's, all
    // MAX_WARPS of them in every group of as many lanes
    auto share_of = [&](int c) {
        int k = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int left = n - i * threads - c * 32;
            k += left >= 32 ? 32 : (left > 0 ? left : 0);
        }
        return static_cast<float>(k * VEC);
    };
    const float mine = share_of(warp), inv_mine = mine > 0.f ? 1.f / mine : 0.f;
    const int other = lane & (MAX_WARPS - 1);
    const float weight = other < warps ? share_of(other) * inv : 0.f;
    const bool whole = ITEMS * threads == n;
    int stage = 0, flip = 0;
    Row next;
    if constexpr (!RING) next.load(a.x + blockIdx.x * a.ldx, t, threads, n);
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        int ahead = stage + STAGES - 1;
        if (ahead >= STAGES) ahead -= STAGES;
        copy_group(g + static_cast<int64_t>(STAGES - 1) * gridDim.x, ahead);
        if constexpr (RING) copy_async_wait<STAGES - 1>();
        F2 d[R][Row::PAIRS];
        float m[R], q[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            Row x;
            if constexpr (RING) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    x.v[i] = V{};
                    if (i * threads + t < n) x.v[i] = ring[((stage * R + k) * ITEMS + i) * threads + t];
                }
            } else {
                static_assert(RING || R == 1, "the next row waits in registers");
                x = next;
                if (g + gridDim.x < groups) next.load(a.x + (g + gridDim.x) * a.ldx, t, threads, n);
            }
            F2 s[2] = {f2(0.f), f2(0.f)};
#pragma unroll
            for (int p = 0; p < Row::PAIRS; ++p) {
                d[k][p] = x.pair(p);
                s[p & 1] = add2(s[p & 1], d[k][p]);
            }
            s[0] = add2(s[0], s[1]);
            m[k] = lo(s[0]) + hi(s[0]);
        }
        if (++stage == STAGES) stage = 0;
#pragma unroll
        for (int k = 0; k < R; ++k) m[k] = warp_sum(m[k]) * inv_mine;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            F2 s[2] = {f2(0.f), f2(0.f)};
            const F2 m2 = f2(-m[k]);
#pragma unroll
            for (int p = 0; p < Row::PAIRS; ++p) {
                d[k][p] = add2(d[k][p], m2);
                if (!whole) d[k][p] = Row::inside(p, d[k][p], t, threads, n);
                s[p & 1] = fma2(d[k][p], d[k][p], s[p & 1]);
            }
            s[0] = add2(s[0], s[1]);
            q[k] = lo(s[0]) + hi(s[0]);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            q[k] = warp_sum(q[k]);
            if (lane == 0) part[flip][k][warp] = make_float2(m[k], q[k]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = g * R + k;
            if (r >= a.rows) break;
            const float2 v = other < warps ? part[flip][k][other] : make_float2(0.f, 0.f);
            float mean = weight * v.x;
#pragma unroll
            for (int o = MAX_WARPS / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(0xFFFFFFFFu, mean, o);
            float var = fmaf(weight * (v.x - mean), v.x - mean, v.y * inv);
#pragma unroll
            for (int o = MAX_WARPS / 2; o > 0; o >>= 1) var += __shfl_xor_sync(0xFFFFFFFFu, var, o);
            const float rstd = rsqrtf(var + a.eps);
            const F2 shift = f2(m[k] - mean), r2 = f2(rstd);
            Row o;
#pragma unroll
            for (int p = 0; p < Row::PAIRS; ++p) {
                F2 v = mul2(add2(d[k][p], shift), r2);
                if (a.w) v = mul2(v, w.pair(p));
                if (a.b) v = add2(v, b.pair(p));
                o.set(p, v);
            }
            o.store(a.y + r * a.ldy, t, threads, n);
            if (t == 0 && a.mean) {
                a.mean[r] = mean;
                a.rstd[r] = rstd;
            }
        }
        flip ^= 1;
    }
}

// A block per row, any width: the row is read three times (mean, variance,
// output), the later times from L1 or L2.
template <typename T>
__global__ void __launch_bounds__(512) norm_fwd_any(NormFwd<T> a) {
    __shared__ float part[2][32];
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) s += to_f32(x[i]);
    const float mean = block_sum(s, part[0]) / static_cast<float>(a.H);
    float q = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float d = to_f32(x[i]) - mean;
        q += d * d;
    }
    const float rstd = 1.f / sqrtf(block_sum(q, part[1]) / static_cast<float>(a.H) + a.eps);
    T* y = a.y + r * a.ldy;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        float v = (to_f32(x[i]) - mean) * rstd;
        if (a.w) v *= load_w<T>(a.w, a.w32, i);
        if (a.b) v += load_w<T>(a.b, a.w32, i);
        y[i] = from_f32<T>(v);
    }
    if (threadIdx.x == 0 && a.mean) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
    }
}

template <typename T>
struct NormBwd {
    const T *dy, *x;
    int64_t ldd, ldx;
    const void* w;
    bool w32;
    const float *mean, *rstd;
    T* dx;  // nullable
    int64_t lddx;
    float* part_w;  // [parts, H], nullable
    float* part_b;
    int64_t rows, rows_per_part;
    int32_t H;
};

// dx of a block's row, any width.
template <typename T>
__global__ void __launch_bounds__(512) norm_dx_any(NormBwd<T> a) {
    __shared__ float part[2][32];
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    const T* dy = a.dy + r * a.ldd;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s = 0.f, q = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f);
        s += g;
        q += g * (to_f32(x[i]) - mean) * rstd;
    }
    s = block_sum(s, part[0]) / static_cast<float>(a.H);
    q = block_sum(q, part[1]) / static_cast<float>(a.H);
    T* dx = a.dx + r * a.lddx;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f);
        dx[i] = from_f32<T>(rstd * (g - s - (to_f32(x[i]) - mean) * rstd * q));
    }
}

// Column sums of a block of rows: 32 columns per block, 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_any(NormBwd<T> a) {
    __shared__ float sw[8][33], sb[8][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    const int64_t r0 = blockIdx.y * a.rows_per_part;
    const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
    float w = 0.f, b = 0.f;
    if (col < a.H)
        for (int64_t r = r0 + k; r < r1; r += 8) {
            const float d = to_f32(a.dy[r * a.ldd + col]);
            w += d * (to_f32(a.x[r * a.ldx + col]) - a.mean[r]) * a.rstd[r];
            b += d;
        }
    sw[k][c] = w;
    sb[k][c] = b;
    __syncthreads();
    if (k == 0 && col < a.H) {
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            w += sw[j][c];
            b += sb[j][c];
        }
        if (a.part_w) a.part_w[static_cast<int64_t>(blockIdx.y) * a.H + col] = w;
        if (a.part_b) a.part_b[static_cast<int64_t>(blockIdx.y) * a.H + col] = b;
    }
}

// dx and the column sums of the block's rows in one pass: each block takes
// the rows blockIdx.x, + gridDim.x, ... (with WARP each of its warps) and keeps
// the sums of its threads' columns in registers.  Rows are copied ahead, each
// thread its own vectors, to a ring of STAGES rows in shared memory: no
// barrier is needed for the data, only for the two sums over a row.
// KEEP: xh and g stay in registers between the sums and dx; without it they
// are computed again from the ring, for the widest rows.
template <typename T, typename W, int VEC, int ITEMS, bool WARP, bool KEEP>
__global__ void __launch_bounds__(WARP ? 128 : 512) norm_bwd_rows(NormBwd<T> a) {
    constexpr int STAGES = NORM_BWD_STAGES;
    __shared__ float2 part[2][16];
    extern __shared__ __align__(16) uint8_t dyn[];  // the ring, then (WARP) the sums of the columns
    using Row = RowRegs<T, VEC, ITEMS>;
    using V = Vec<T, VEC>;
    launch_dependents();
    constexpr bool RING = sizeof(V) >= 4;  // single 16-bit elements wait in registers
    static_assert(KEEP || RING, "the rows are read again from the ring");
    const int tpr = WARP ? 32 : blockDim.x;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    const int n = a.H / VEC;
    const int64_t step = WARP ? gridDim.x * 4ll : gridDim.x;
    const float inv = 1.f / static_cast<float>(a.H);
    V* ring = reinterpret_cast<V*>(dyn);  // [STAGES][2][ITEMS][threads]
    const int64_t r0 = WARP ? blockIdx.x * 4ll + warp : blockIdx.x;
    auto copy_row = [&](int64_t r, int stage) {
        if constexpr (RING) {
            if (r < a.rows) {
                const V* x = reinterpret_cast<const V*>(a.x + r * a.ldx);
                const V* d = reinterpret_cast<const V*>(a.dy + r * a.ldd);
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (i * tpr + t < n) {
                        copy_async<sizeof(V)>(ring + ((stage * 2) * ITEMS + i) * blockDim.x + threadIdx.x, x + i * tpr + t);
                        copy_async<sizeof(V)>(ring + ((stage * 2 + 1) * ITEMS + i) * blockDim.x + threadIdx.x, d + i * tpr + t);
                    }
            }
            copy_async_commit();
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) copy_row(r0 + k * step, k);
    RowRegs<W, VEC, ITEMS> w;
    if (a.w) w.load(static_cast<const W*>(a.w), t, tpr, n);
    F2 sw[Row::PAIRS], sb[Row::PAIRS];
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) sw[p] = sb[p] = f2(0.f);
    int flip = 0, stage = 0;
    float mean_next = 0.f, rstd_next = 0.f;
    if (r0 < a.rows) {
        mean_next = a.mean[r0];
        rstd_next = a.rstd[r0];
    }
    Row x_next, d_next;  // without a ring, the next row waits in registers
    if constexpr (!RING)
        if (r0 < a.rows) {
            x_next.load(a.x + r0 * a.ldx, t, tpr, n);
            d_next.load(a.dy + r0 * a.ldd, t, tpr, n);
        }
    for (int64_t r = r0; r < a.rows; r += step) {
        const float mean = mean_next, rstd = rstd_next;
        if (r + step < a.rows) {
            mean_next = a.mean[r + step];
            rstd_next = a.rstd[r + step];
        }
        Row x, d;
        auto from_ring = [&]() {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                x.v[i] = d.v[i] = V{};
                if (i * tpr + t < n) {
                    x.v[i] = ring[((stage * 2) * ITEMS + i) * blockDim.x + threadIdx.x];
                    d.v[i] = ring[((stage * 2 + 1) * ITEMS + i) * blockDim.x + threadIdx.x];
                }
            }
        };
        if constexpr (RING) {
            int ahead = stage + STAGES - 1;
            if (ahead >= STAGES) ahead -= STAGES;
            copy_row(r + (STAGES - 1) * step, ahead);
            copy_async_wait<STAGES - 1>();
            from_ring();
        } else {
            x = x_next;
            d = d_next;
            if (r + step < a.rows) {
                x_next.load(a.x + (r + step) * a.ldx, t, tpr, n);
                d_next.load(a.dy + (r + step) * a.ldd, t, tpr, n);
            }
        }
        // outside the row dy = 0, so nothing is added
        F2 s2 = f2(0.f), q2 = f2(0.f), kx[KEEP ? Row::PAIRS : 1], kg[KEEP ? Row::PAIRS : 1];
#pragma unroll
        for (int p = 0; p < Row::PAIRS; ++p) {
            const F2 dy = d.pair(p);
            const F2 xh = mul2(add2(x.pair(p), f2(-mean)), f2(rstd));
            const F2 g = a.w ? mul2(dy, w.pair(p)) : dy;
            s2 = add2(s2, g);
            q2 = fma2(g, xh, q2);
            sb[p] = add2(sb[p], dy);
            sw[p] = fma2(dy, xh, sw[p]);
            if constexpr (KEEP) {
                kx[p] = xh;
                kg[p] = g;
            }
        }
        if (a.dx) {
            float s = warp_sum(lo(s2) + hi(s2)), q = warp_sum(lo(q2) + hi(q2));
            if (!WARP) {
                if (lane == 0) part[flip][warp] = make_float2(s, q);
                __syncthreads();
                s = q = 0.f;
                for (int k = 0; k < warps; ++k) {
                    s += part[flip][k].x;
                    q += part[flip][k].y;
                }
                flip ^= 1;
            }
            const F2 ms = f2(-s * inv), mq = f2(-q * inv);
            if constexpr (!KEEP) from_ring();
#pragma unroll
            for (int p = 0; p < Row::PAIRS; ++p) {
                F2 xh, g;
                if constexpr (KEEP) {
                    xh = kx[p];
                    g = kg[p];
                } else {
                    xh = mul2(add2(x.pair(p), f2(-mean)), f2(rstd));
                    g = a.w ? mul2(d.pair(p), w.pair(p)) : d.pair(p);
                }
                x.set(p, mul2(f2(rstd), fma2(xh, mq, add2(g, ms))));
            }
            x.store(a.dx + r * a.lddx, t, tpr, n);
        }
        if (++stage == STAGES) stage = 0;
    }
    if (!a.part_w) return;
    float* pw = a.part_w + static_cast<int64_t>(blockIdx.x) * a.H;
    float* pb = a.part_b + static_cast<int64_t>(blockIdx.x) * a.H;
    auto column = [&](int e) { return VEC == 1 ? e * tpr + t : ((e / VEC) * tpr + t) * VEC + e % VEC; };
    if (WARP) {  // the warps' sums, one warp after the other
        float* cols = reinterpret_cast<float*>(dyn + (RING ? STAGES * 2 * ITEMS * 128 * sizeof(V) : 0));
        for (int k = 0; k < 4; ++k) {
            if (warp == k)
#pragma unroll
                for (int e = 0; e < 2 * Row::PAIRS; ++e) {
                    const int c = column(e);
                    if (c >= a.H) continue;
                    cols[c] = (k ? cols[c] : 0.f) + (e & 1 ? hi(sw[e / 2]) : lo(sw[e / 2]));
                    cols[a.H + c] = (k ? cols[a.H + c] : 0.f) + (e & 1 ? hi(sb[e / 2]) : lo(sb[e / 2]));
                }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.H; c += 128) {
            pw[c] = cols[c];
            pb[c] = cols[a.H + c];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 2 * Row::PAIRS; ++e) {
            const int c = column(e);
            if (c >= a.H) continue;
            pw[c] = e & 1 ? hi(sw[e / 2]) : lo(sw[e / 2]);
            pb[c] = e & 1 ? hi(sb[e / 2]) : lo(sb[e / 2]);
        }
    }
}

// Adds the parts' column sums in a fixed order: 32 columns per block, 32
// threads a column with up to eight parts of each in flight.
struct JoinArgs {
    const float *part_w, *part_b;
    int32_t parts, H;
    void *dw, *db;  // each nullable
};
template <typename W>
__global__ void __launch_bounds__(1024) norm_dw_join(JoinArgs a) {
    __shared__ float s[32][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    const float* p = blockIdx.y ? a.part_b : a.part_w;
    W* out = static_cast<W*>(blockIdx.y ? a.db : a.dw);
    if (!out) return;
    wait_for_primary();
    float v = 0.f;
    if (col < a.H)
#pragma unroll 8
        for (int j = k; j < a.parts; j += 32) v += p[static_cast<int64_t>(j) * a.H + col];
    s[k][c] = v;
    __syncthreads();
    v = warp_sum(s[c][k]);  // column k of this block
    if (c == 0 && blockIdx.x * 32 + k < a.H) out[blockIdx.x * 32 + k] = from_f32<W>(v);
}

// Blocks of `kernel` that stay on the current device at once, after raising
// its shared memory limit; asked once per kernel, device and launch shape.
struct Resident {
    std::atomic<int64_t> known[16];
};
template <typename K>
int resident_blocks(Resident* memo, K kernel, int threads, size_t smem) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int64_t tag = (static_cast<int64_t>(threads) << 40) | (static_cast<int64_t>(smem) << 16);
    std::atomic<int64_t>* slot = dev < 16 ? &memo->known[dev] : nullptr;
    if (slot) {
        const int64_t v = slot->load(std::memory_order_relaxed);
        if ((v & ~0xFFFFll) == tag && (v & 0xFFFF)) return static_cast<int>(v & 0xFFFF);
    }
    int per = 0, sms = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_SMEM_MAX) != cudaSuccess ||
        smem > NORM_SMEM_MAX)
        return 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    const int n = per * sms;
    if (slot && n > 0 && n < 0x10000) slot->store(tag | n, std::memory_order_relaxed);
    return n;
}

int threads_for(int vectors, int items) { return (((vectors + items - 1) / items) + 31) / 32 * 32; }

template <typename T, typename W, int VEC, int ITEMS, int R, int STAGES, int MAX_WARPS, int BLOCKS>
lce_status_t fwd_rows(const NormFwd<T>& a, cudaStream_t s) {
    static Resident memo;
    auto kernel = norm_fwd_rows<T, W, VEC, ITEMS, R, STAGES, MAX_WARPS, BLOCKS>;
    const int threads = threads_for(a.H / VEC, ITEMS);
    const size_t smem = sizeof(Vec<T, VEC>) >= 4 ? static_cast<size_t>(STAGES) * R * ITEMS * threads * sizeof(Vec<T, VEC>) : 0;
    const int64_t most = resident_blocks(&memo, kernel, threads, smem), groups = (a.rows + R - 1) / R;
    if (most <= 0) return LCE_ERR_CUDA;
    LCE_PROFILED(kernel<<<static_cast<unsigned>(groups < most ? groups : most), threads, smem, s>>>(a));
    return LCE_OK;
}

// The forward's form by the row's width in vectors (16 bytes where rows start
// on 16-byte boundaries; else 4 bytes; else one element), measured on 2^29
// bf16 elements against the copy rate:
//  - up to 64 vectors (512 bf16): a warp per row, 6.1 TB/s at 512;
//  - up to 128: the same with the next rows copied ahead and weight and bias
//    kept, 6.1 TB/s at 1024 (a block of two warps: 4.7).  16384 rows of it with
//    fp32 weights take 13 us, against 18 where each warp ends with its row;
//  - up to 2048: a block per row, four vectors a thread, 6.4 TB/s at 4096 (a
//    warp per row: 5.7, two vectors: 5.3);
//  - where a quarter of such a block would be idle, two rows of two vectors a
//    thread: 5.9 TB/s at 2560 against 4.9;
//  - narrower vectors: eight a thread, or sixteen single elements; 2.6 TB/s at
//    1601 fp16, where the warps (29% of them) issue in 58 of 100 cycles and
//    wait for shared memory and shuffles.  16-byte vectors counted from each
//    row's own start reached 2.4: a row's two ends cost the warp that has them
//    more than the vectors save;
//  - wider rows: the row is read again.
template <typename T, typename W>
lce_status_t norm_forward(const NormCall& c) {
    const NormFwd<T> a{static_cast<const T*>(c.x), c.ldx, c.w, c.b, c.w32, c.eps, static_cast<T*>(c.y), c.ldy,
                       c.mean_out, c.rstd_out, c.rows, c.H};
    cudaStream_t s = c.s;
    constexpr int V = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
    auto fits = [&](int vec) {  // rows of x and y, weight and bias can be read in vectors of `vec`
        const size_t b = vec * sizeof(T), wb = vec * sizeof(W) < 16 ? vec * sizeof(W) : 16;
        return c.H % vec == 0 && c.ldx % vec == 0 && c.ldy % vec == 0 && aligned_to(c.x, b) && aligned_to(c.y, b) &&
               aligned_to(c.w, wb) && aligned_to(c.b, wb);
    };
    if (fits(V) && c.H / V <= 2048) {
        const int n = c.H / V;
        const unsigned blocks = static_cast<unsigned>((c.rows + 3) / 4);
        if (n <= 32) {
            LCE_PROFILED(norm_fwd_warp<T, W, V, 1><<<blocks, 128, 0, s>>>(a));
        } else if (n <= 64) {
            LCE_PROFILED(norm_fwd_warp<T, W, V, 2><<<blocks, 128, 0, s>>>(a));
        } else if (n <= 128) {
            return fwd_rows<T, W, V, 4, 1, 3, 1, 12>(a, s);
        } else if (n <= 512 && 4 * threads_for(n, 4) > n + n / 8) {
            return fwd_rows<T, W, V, 2, 2, 2, 8, 2>(a, s);
        } else if (n <= 512) {
            return fwd_rows<T, W, V, 4, 1, 3, 4, 4>(a, s);
        } else if (n <= 1024) {
            return fwd_rows<T, W, V, 4, 1, 3, 8, 2>(a, s);
        } else {
            return fwd_rows<T, W, V, 4, 1, 3, 16, 1>(a, s);
        }
        return LCE_OK;
    }
    if (V4 > 1 && fits(V4) && c.H / V4 <= 4096) return fwd_rows<T, W, V4, 8, 1, 3, 16, 1>(a, s);
    if (c.H <= 4096) return fwd_rows<T, W, 1, 8, 1, 3, 16, 1>(a, s);
    if (c.H <= 8192) return fwd_rows<T, W, 1, 16, 1, 3, 16, 1>(a, s);
    LCE_PROFILED(norm_fwd_any<T><<<static_cast<unsigned>(c.rows), 512, 0, s>>>(a));
    return LCE_OK;
}

template <typename T, typename W, int VEC, int ITEMS, bool WARP, bool KEEP>
lce_status_t bwd_rows(const NormBwd<T>& a, int* parts, cudaStream_t s) {
    static Resident memo;
    auto kernel = norm_bwd_rows<T, W, VEC, ITEMS, WARP, KEEP>;
    const int threads = WARP ? 128 : threads_for(a.H / VEC, ITEMS);
    const size_t vec = sizeof(Vec<T, VEC>), ring = vec >= 4 ? NORM_BWD_STAGES * 2 * ITEMS * threads * vec : 0;
    const size_t smem = ring + (WARP ? 2 * static_cast<size_t>(a.H) * 4 : 0);
    int64_t blocks = resident_blocks(&memo, kernel, threads, smem);
    if (blocks <= 0) return LCE_ERR_CUDA;
    const int64_t work = WARP ? (a.rows + 3) / 4 : a.rows;
    if (blocks > work) blocks = work;
    if (blocks > NORM_PARTS) blocks = NORM_PARTS;
    *parts = static_cast<int>(blocks);
    LCE_PROFILED(kernel<<<static_cast<unsigned>(blocks), threads, smem, s>>>(a));
    return LCE_OK;
}

// The backward's form, by the same widths (2^29 bf16 elements):
//  - up to 128 vectors: a warp per row, 6.4 TB/s at 1024, 6.8 at 512.  Blocks
//    of two warps reach 6.7 at 1024, but leave four times the parts to add;
//  - up to 1024: a block per row, two vectors a thread, 6.6 TB/s at 4096 (one
//    vector: 4.3, as the sums over a row then cost as much as the row);
//  - up to 2048: four vectors a thread, read twice from the ring;
//  - narrower vectors: eight a thread, or sixteen single elements (3.0 TB/s at
//    1601 fp16);
//  - wider rows: dx, reading the row again, and the column sums by themselves.
template <typename T, typename W>
lce_status_t norm_backward(const NormCall& c) {
    NormBwd<T> a{static_cast<const T*>(c.dy), static_cast<const T*>(c.x), c.ldd, c.ldx, c.w, c.w32, c.mean, c.rstd,
                 static_cast<T*>(c.y), c.ldy, nullptr, nullptr, c.rows, 0, c.H};
    cudaStream_t s = c.s;
    const bool sums = c.dw || c.db;
    if (sums) {
        a.part_w = c.parts;
        a.part_b = c.parts + (c.rows < NORM_PARTS ? c.rows : NORM_PARTS) * c.H;
    }
    constexpr int V = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
    auto fits = [&](int vec) {
        const size_t b = vec * sizeof(T), wb = vec * sizeof(W) < 16 ? vec * sizeof(W) : 16;
        return c.H % vec == 0 && c.ldx % vec == 0 && c.ldd % vec == 0 && c.ldy % vec == 0 && aligned_to(c.x, b) &&
               aligned_to(c.dy, b) && aligned_to(c.y, b) && aligned_to(c.w, wb);
    };
    int parts = 0;
    lce_status_t st = LCE_OK;
    if (fits(V) && c.H / V <= 2048) {
        const int n = c.H / V;
        st = n <= 32     ? bwd_rows<T, W, V, 1, true, true>(a, &parts, s)
             : n <= 64   ? bwd_rows<T, W, V, 2, true, true>(a, &parts, s)
             : n <= 128  ? bwd_rows<T, W, V, 4, true, true>(a, &parts, s)
             : n <= 1024 ? bwd_rows<T, W, V, 2, false, true>(a, &parts, s)
                         : bwd_rows<T, W, V, 4, false, false>(a, &parts, s);
    } else if (V4 > 1 && fits(V4) && c.H / V4 <= 4096) {
        st = bwd_rows<T, W, V4, 8, false, true>(a, &parts, s);
    } else if (c.H <= 4096) {
        st = bwd_rows<T, W, 1, 8, false, true>(a, &parts, s);
    } else if (c.H <= 8192) {
        st = bwd_rows<T, W, 1, 16, false, true>(a, &parts, s);
    } else {
        if (c.y) LCE_PROFILED(norm_dx_any<T><<<static_cast<unsigned>(c.rows), 512, 0, s>>>(a));
        if (sums) {
            a.rows_per_part = (c.rows + NORM_PARTS - 1) / NORM_PARTS;
            if (a.rows_per_part < 32) a.rows_per_part = 32;
            parts = static_cast<int>((c.rows + a.rows_per_part - 1) / a.rows_per_part);
            LCE_PROFILED(norm_dw_any<T><<<dim3((c.H + 31) / 32, parts), 256, 0, s>>>(a));
        }
    }
    if (st != LCE_OK || !sums) return st;
    LCE_PROFILED(launch_after(norm_dw_join<W>, dim3((c.H + 31) / 32, 2), 1024, 0, s,
                              JoinArgs{a.part_w, a.part_b, parts, c.H, c.dw, c.db}));
    return LCE_OK;
}

}  // namespace
}  // namespace lce
