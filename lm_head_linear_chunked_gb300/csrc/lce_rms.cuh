// RMS norm with the residual's addition, forward (in the rows' type or in 8
// bits with scales) and backward.
//
//   s = x + r, rounded to the rows' type;  rstd = 1 / sqrt(sum_h s^2 / H + eps)
//   y = s rstd w
//   8 bits: a = max |y| of a group of columns, scale = max(a, 2^-100) / 448,
//     q = e4m3(y (1 / scale))
//   xh = s rstd,  g = dy w,  dx = rstd (g - xh mean_h(g xh)) + ds
//   dw = sum_r dy xh
//
// The sum is rounded before it is normed: the rounded one is what the next
// block adds to and what the backward reads, so all three see the same s.
// y is multiplied by the scale's rounded reciprocal, not divided: two roundings
// of 2^-24 before the one to 8 bits (2^-4), so another value only where y / scale
// lies that close to the middle of two (32768 x 4096 bf16 to 8 bits 153 us, with
// a division for each element 193).
// All sums are FP32.
#pragma once

#include <type_traits>

#include "lce_internal.cuh"
#include "lce_rows.cuh"

namespace lce {

constexpr int RMS_BWD_STAGES = 3;
constexpr float E4M3_MAX = 448.f;
constexpr float RMS_LEAST_AMAX = 0x1p-100f;  // keeps 1 / scale finite where a group is zero

// What a launch needs, by the element type (one translation unit each).
struct RmsCall {
    const void *x, *r, *w, *dy, *ds;
    int64_t ldx, ldr, ldd, ldds, lds, ldy;
    bool w32;
    float eps;
    void *sum, *y;       // y: the output, or dx
    uint8_t* q;
    int64_t ldq;
    float* scales;
    int32_t group;       // columns to a scale (H: one for the row)
    float* rstd_out;
    const float* rstd;
    void* dw;
    float* parts;        // [NORM_PARTS, H]
    int64_t rows;
    int32_t H;
    cudaStream_t s;
};
lce_status_t rms_forward_bf16(const RmsCall& c);
lce_status_t rms_forward_f16(const RmsCall& c);
lce_status_t rms_forward_f32(const RmsCall& c);
lce_status_t rms_backward_bf16(const RmsCall& c);
lce_status_t rms_backward_f16(const RmsCall& c);
lce_status_t rms_backward_f32(const RmsCall& c);

namespace {

// The larger of two, NaN if one is: a row that holds one shows it in its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Two values as e4m3, rounded to nearest even, the first in the low byte.
__device__ __forceinline__ uint16_t to_e4m3x2(float first, float second) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(second), "f"(first));
    return r;
}

__device__ __forceinline__ float group_scale(float amax) { return max_nan(amax, RMS_LEAST_AMAX) / E4M3_MAX; }

template <typename T>
struct RmsFwd {
    const T *x, *r;  // r nullable
    int64_t ldx, ldr;
    const void* w;   // nullable; fp32 with w32, else T
    bool w32;
    float eps;
    T* sum;          // written where r is given
    int64_t lds;
    T* y;            // or q and scales
    int64_t ldy;
    uint8_t* q;
    int64_t ldq;
    float* scales;   // [rows, groups]
    int32_t group, groups;
    float* rstd;     // nullable
    int64_t rows;
    int32_t H;
};

// Where item i of a thread lies in a row of vectors of VEC elements: whole
// groups of LCE_FP8_GROUP columns to a warp (or a half), so that their largest
// magnitude needs shuffles only.
template <int VEC>
__device__ __forceinline__ int rms_at(int i, int warp, int warps, int lane) {
    constexpr int S = VEC >= 4 ? 1 : LCE_FP8_GROUP / 32 / VEC;  // vectors of a lane in a group
    return ((i / S * warps + warp) * S + i % S) * 32 + lane;
}

// The sum (largest) over each LANES neighbouring lanes of a warp.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max_nan(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// The forward: a block (for narrow rows a warp, or LANES of its lanes) takes R rows at a time and
// copies the next ones ahead, each thread its own vectors, so that only the
// sums over a row wait for the other warps.  The row stays in registers
// between its sum and the output.
template <typename T, typename W, int VEC, int ITEMS, int R, int STAGES, int MAX_WARPS, int BLOCKS, bool QUANT, int LANES>
__global__ void __launch_bounds__(32 * MAX_WARPS, BLOCKS) rms_fwd_rows(RmsFwd<T> a) {
    constexpr int PER = R * 32 / LANES;  // rows of a block at a time
    static_assert(LANES == 32 || (R == 1 && MAX_WARPS == 1 && ITEMS == 1 && VEC >= 4 && LANES * VEC <= LCE_FP8_GROUP));
    constexpr bool RING = sizeof(Vec<T, VEC>) >= 4;  // single 16-bit elements wait in registers
    static_assert(RING || R == 1, "the next row waits in registers");
    using Row = RowRegs<T, VEC, ITEMS>;
    using V = Vec<T, VEC>;
    constexpr int PAIRS = Row::PAIRS;
    __shared__ float part[2][R][MAX_WARPS], most[2][R][MAX_WARPS];
    extern __shared__ __align__(16) uint8_t dyn[];
    wait_for_primary();
    const int t = threadIdx.x, threads = blockDim.x, warp = t >> 5, warps = threads >> 5, lane = t & (LANES - 1);
    const int sub = LANES < 32 ? t / LANES : 0;  // the row of a warp that takes several
    const int n = a.H / VEC;
    const float inv = 1.f / static_cast<float>(a.H);
    V* ring = reinterpret_cast<V*>(dyn);  // [STAGES][R][x, r][ITEMS][threads]
    const int mats = a.r ? 2 : 1;
    const int64_t groups = (a.rows + PER - 1) / PER;
    auto slot = [&](int stage, int k, int m, int i) { return ring + (((stage * R + k) * mats + m) * ITEMS + i) * threads + t; };
    auto copy_group = [&](int64_t g, int stage) {
        if constexpr (RING) {
            if (g < groups)
#pragma unroll
                for (int k = 0; k < R; ++k)
                    if (g * PER + k + sub < a.rows) {
                        const V* x = reinterpret_cast<const V*>(a.x + (g * PER + k + sub) * a.ldx);
                        const V* r = reinterpret_cast<const V*>(a.r + (g * PER + k + sub) * a.ldr);
#pragma unroll
                        for (int i = 0; i < ITEMS; ++i) {
                            const int at = rms_at<VEC>(i, warp, warps, lane);
                            if (at >= n) continue;
                            copy_async<sizeof(V)>(slot(stage, k, 0, i), x + at);
                            if (a.r) copy_async<sizeof(V)>(slot(stage, k, 1, i), r + at);
                        }
                    }
            copy_async_commit();
        }
    };
    auto load = [&](auto& row, const auto* from) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            using E = std::decay_t<decltype(row.v[0])>;
            const int at = rms_at<VEC>(i, warp, warps, lane);
            row.v[i] = E{};
            if (at < n) row.v[i] = reinterpret_cast<const E*>(from)[at];
        }
    };
    auto store = [&](const Row& row, T* to) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int at = rms_at<VEC>(i, warp, warps, lane);
            if (at < n) reinterpret_cast<V*>(to)[at] = row.v[i];
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) copy_group(blockIdx.x + static_cast<int64_t>(k) * gridDim.x, k);
    RowRegs<W, VEC, ITEMS> w;
    if (a.w) load(w, static_cast<const W*>(a.w));
    int stage = 0, flip = 0;
    Row next, next_r;
    if constexpr (!RING) {
        load(next, a.x + blockIdx.x * a.ldx);
        if (a.r) load(next_r, a.r + blockIdx.x * a.ldr);
    }
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        int ahead = stage + STAGES - 1;
        if (ahead >= STAGES) ahead -= STAGES;
        copy_group(g + static_cast<int64_t>(STAGES - 1) * gridDim.x, ahead);
        if constexpr (RING) copy_async_wait<STAGES - 1>();
        F2 d[R][PAIRS];
        float q[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = g * PER + k + sub;
            Row x, r;
            if constexpr (RING) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    x.v[i] = r.v[i] = V{};
                    if (rms_at<VEC>(i, warp, warps, lane) >= n) continue;
                    x.v[i] = *slot(stage, k, 0, i);
                    if (a.r) r.v[i] = *slot(stage, k, 1, i);
                }
            } else {
                x = next;
                r = next_r;
                if (g + gridDim.x < groups) {
                    load(next, a.x + (g + gridDim.x) * a.ldx);
                    if (a.r) load(next_r, a.r + (g + gridDim.x) * a.ldr);
                }
            }
            if (a.r) {
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) x.set(p, add2(x.pair(p), r.pair(p)));
                if (row < a.rows) store(x, a.sum + row * a.lds);
            }
            F2 s[2] = {f2(0.f), f2(0.f)};
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) {
                d[k][p] = x.pair(p);
                s[p & 1] = fma2(d[k][p], d[k][p], s[p & 1]);
            }
            s[0] = add2(s[0], s[1]);
            q[k] = lo(s[0]) + hi(s[0]);
        }
        if (++stage == STAGES) stage = 0;
#pragma unroll
        for (int k = 0; k < R; ++k) q[k] = lanes_sum<LANES>(q[k]);
        if constexpr (MAX_WARPS > 1) {
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (lane == 0) part[flip][k][warp] = q[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int other = lane & (MAX_WARPS - 1);
                q[k] = other < warps ? part[flip][k][other] : 0.f;
#pragma unroll
                for (int o = MAX_WARPS / 2; o > 0; o >>= 1) q[k] += __shfl_xor_sync(0xFFFFFFFFu, q[k], o);
            }
        }
        float amax[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float rstd = rsqrtf(fmaf(q[k], inv, a.eps));
            const F2 r2 = f2(rstd);
            amax[k] = 0.f;
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) {
                d[k][p] = mul2(d[k][p], r2);
                if (a.w) d[k][p] = mul2(d[k][p], w.pair(p));
                if constexpr (QUANT) amax[k] = max_nan(amax[k], max_nan(fabsf(lo(d[k][p])), fabsf(hi(d[k][p]))));
            }
            const int64_t row = g * PER + k + sub;
            if (warp == 0 && lane == 0 && a.rstd && row < a.rows) a.rstd[row] = rstd;
            if constexpr (!QUANT) {
                if (row >= a.rows) break;
                Row o;
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) o.set(p, d[k][p]);
                store(o, a.y + row * a.ldy);
            }
        }
        if constexpr (QUANT) {
            const bool one = LANES < 32 || a.groups == 1;
            if (one) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    amax[k] = lanes_max_nan<LANES>(amax[k]);
                    if (MAX_WARPS > 1 && lane == 0) most[flip][k][warp] = amax[k];
                }
                if constexpr (MAX_WARPS > 1) {
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < R; ++k) amax[k] = warp_max_nan(lane < warps ? most[flip][k][lane & (MAX_WARPS - 1)] : 0.f);
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t row = g * PER + k + sub;
                if (row >= a.rows) break;
                float scale = group_scale(amax[k]), by = 1.f / scale;
                if (one && warp == 0 && lane == 0) a.scales[row] = scale;
                constexpr int S = VEC >= 4 ? 1 : LCE_FP8_GROUP / 32 / VEC, GROUP = VEC >= 4 ? LCE_FP8_GROUP / VEC : 32;
                constexpr int PER = VEC == 1 ? 1 : VEC / 2;  // pairs of a vector (with single elements half of one)
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    if (LANES == 32 && !one && i % S == 0) {
                        float m = 0.f;
#pragma unroll
                        for (int e = i * VEC; e < (i + S) * VEC; ++e)
                            m = max_nan(m, fabsf(e & 1 ? hi(d[k][e / 2]) : lo(d[k][e / 2])));
#pragma unroll
                        for (int o = GROUP / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                        scale = group_scale(m);
                        by = 1.f / scale;
                        const int at = rms_at<VEC>(i, warp, warps, lane);
                        if ((lane & (GROUP - 1)) == 0 && at < n) a.scales[row * a.groups + at * VEC / LCE_FP8_GROUP] = scale;
                    }
                    const int at = rms_at<VEC>(i, warp, warps, lane);
                    if (at >= n) continue;
                    uint8_t* to = a.q + row * a.ldq + static_cast<int64_t>(at) * VEC;
                    if constexpr (VEC == 1) {
                        *to = static_cast<uint8_t>(to_e4m3x2((i & 1 ? hi(d[k][i / 2]) : lo(d[k][i / 2])) * by, 0.f));
                    } else {
                        Vec<uint16_t, PER> b;
#pragma unroll
                        for (int p = 0; p < PER; ++p) {
                            const F2 v = mul2(d[k][i * PER + p], f2(by));
                            b.v[p] = to_e4m3x2(lo(v), hi(v));
                        }
                        *reinterpret_cast<Vec<uint16_t, PER>*>(to) = b;
                    }
                }
            }
        }
        flip ^= 1;
    }
}

// A block per row, any width: the row is read again for the output (and, in 8
// bits, for the largest magnitude), from L1 or L2.
template <typename T, bool QUANT>
__global__ void __launch_bounds__(512) rms_fwd_any(RmsFwd<T> a) {
    __shared__ float part[2][32];
    wait_for_primary();
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        float v = to_f32(x[i]);
        if (a.r) {
            const T t = from_f32<T>(v + to_f32(a.r[r * a.ldr + i]));
            a.sum[r * a.lds + i] = t;
            v = to_f32(t);
        }
        s = fmaf(v, v, s);
    }
    const float rstd = rsqrtf(block_sum(s, part[0]) / static_cast<float>(a.H) + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    if (a.r) x = a.sum + r * a.lds;
    auto normed = [&](int i) { return to_f32(x[i]) * rstd * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f); };
    if constexpr (!QUANT) {
        for (int i = threadIdx.x; i < a.H; i += blockDim.x) a.y[r * a.ldy + i] = from_f32<T>(normed(i));
    } else if (a.groups == 1) {
        float m = 0.f;
        for (int i = threadIdx.x; i < a.H; i += blockDim.x) m = max_nan(m, fabsf(normed(i)));
        m = warp_max_nan(m);
        if ((threadIdx.x & 31) == 0) part[1][threadIdx.x >> 5] = m;
        __syncthreads();
        m = warp_max_nan((threadIdx.x & 31) < (blockDim.x >> 5) ? part[1][threadIdx.x & 31] : 0.f);
        const float scale = group_scale(m), inv = 1.f / scale;
        if (threadIdx.x == 0) a.scales[r] = scale;
        for (int i = threadIdx.x; i < a.H; i += blockDim.x)
            a.q[r * a.ldq + i] = static_cast<uint8_t>(to_e4m3x2(normed(i) * inv, 0.f));
    } else {
        for (int g = threadIdx.x >> 5; g < a.groups; g += blockDim.x >> 5) {
            const int first = g * a.group + (threadIdx.x & 31);
            const int end = a.H - g * a.group < a.group ? a.H : (g + 1) * a.group;
            float m = 0.f;
            for (int i = first; i < end; i += 32) m = max_nan(m, fabsf(normed(i)));
            m = warp_max_nan(m);
            const float scale = group_scale(m), inv = 1.f / scale;
            if ((threadIdx.x & 31) == 0) a.scales[r * a.groups + g] = scale;
            for (int i = first; i < end; i += 32)
                a.q[r * a.ldq + i] = static_cast<uint8_t>(to_e4m3x2(normed(i) * inv, 0.f));
        }
    }
}

template <typename T>
struct RmsBwd {
    const T *dy, *x, *ds;  // ds nullable
    int64_t ldd, ldx, ldds;
    const void* w;
    bool w32;
    const float* rstd;
    T* dx;                 // nullable
    int64_t lddx;
    float* part_w;         // [parts, H], nullable
    int64_t rows, rows_per_part;
    int32_t H;
};

// dx and the column sums of the block's rows in one pass: each block takes
// the rows blockIdx.x, + gridDim.x, ... (with WARP each of its warps) and keeps
// the sums of its threads' columns in registers.  Rows are copied ahead, each
// thread its own vectors, to a ring in shared memory, so a barrier is needed
// only for the sum over a row.  KEEP: xh and g stay in registers between the
// sum and dx; without it they are computed again from the ring, for the widest
// rows, whose ds has no room in the ring and is read when it is added.
template <typename T, typename W, int VEC, int ITEMS, bool WARP, bool KEEP, int LANES>
__global__ void __launch_bounds__(WARP ? 128 : 512) rms_bwd_rows(RmsBwd<T> a) {
    static_assert(LANES == 32 || (WARP && ITEMS == 1 && VEC > 1));
    constexpr int PER = 32 / LANES;  // rows of a warp at a time
    constexpr int STAGES = RMS_BWD_STAGES;
    __shared__ float part[2][16];
    extern __shared__ __align__(16) uint8_t dyn[];  // the ring, then (WARP) the sums of the columns
    using Row = RowRegs<T, VEC, ITEMS>;
    using V = Vec<T, VEC>;
    constexpr bool RING = sizeof(V) >= 4;  // single 16-bit elements wait in registers
    static_assert(KEEP || RING, "the rows are read again from the ring");
    launch_dependents();
    wait_for_primary();
    const int tpr = WARP ? LANES : blockDim.x;
    const int t = WARP ? threadIdx.x & (LANES - 1) : threadIdx.x;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    const int n = a.H / VEC, mats = KEEP && a.ds ? 3 : 2;
    const int64_t step = WARP ? gridDim.x * 4ll * PER : gridDim.x;
    const float inv = 1.f / static_cast<float>(a.H);
    V* ring = reinterpret_cast<V*>(dyn);  // [STAGES][x, dy, ds][ITEMS][threads]
    const int64_t r0 = WARP ? (blockIdx.x * 4ll + warp) * PER + lane / LANES : blockIdx.x;
    auto slot = [&](int stage, int m, int i) { return ring + ((stage * mats + m) * ITEMS + i) * blockDim.x + threadIdx.x; };
    auto copy_row = [&](int64_t r, int stage) {
        if constexpr (RING) {
            if (r < a.rows) {
                const V* x = reinterpret_cast<const V*>(a.x + r * a.ldx);
                const V* d = reinterpret_cast<const V*>(a.dy + r * a.ldd);
                const V* ds = reinterpret_cast<const V*>(a.ds + r * a.ldds);
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (i * tpr + t < n) {
                        copy_async<sizeof(V)>(slot(stage, 0, i), x + i * tpr + t);
                        copy_async<sizeof(V)>(slot(stage, 1, i), d + i * tpr + t);
                        if (KEEP && a.ds) copy_async<sizeof(V)>(slot(stage, 2, i), ds + i * tpr + t);
                    }
            }
            copy_async_commit();
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) copy_row(r0 + k * step, k);
    RowRegs<W, VEC, ITEMS> w;
    if (a.w) w.load(static_cast<const W*>(a.w), t, tpr, n);
    F2 sw[Row::PAIRS];
#pragma unroll
    for (int p = 0; p < Row::PAIRS; ++p) sw[p] = f2(0.f);
    int flip = 0, stage = 0;
    float rstd_next = r0 < a.rows ? a.rstd[r0] : 0.f;
    Row x_next, d_next, s_next;  // without a ring, the next row waits in registers
    auto load_next = [&](int64_t r) {
        x_next.load(a.x + r * a.ldx, t, tpr, n);
        d_next.load(a.dy + r * a.ldd, t, tpr, n);
        if (a.ds) s_next.load(a.ds + r * a.ldds, t, tpr, n);
    };
    if constexpr (!RING)
        if (r0 < a.rows) load_next(r0);
    // (the lanes of a warp stay together: those without a row have zeros and write nothing)
    for (int64_t r = r0; LANES < 32 ? r - lane / LANES < a.rows : r < a.rows; r += step) {
        const bool in = LANES == 32 || r < a.rows;
        const F2 rstd = f2(rstd_next);
        rstd_next = r + step < a.rows ? a.rstd[r + step] : 0.f;  // 0 without a row: what a NaN would do to the sums
        Row x, d, ds;
        auto from_ring = [&](Row& row, int m) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                row.v[i] = V{};
                if (in && i * tpr + t < n) row.v[i] = *slot(stage, m, i);
            }
        };
        if constexpr (RING) {
            int ahead = stage + STAGES - 1;
            if (ahead >= STAGES) ahead -= STAGES;
            copy_row(r + (STAGES - 1) * step, ahead);
            copy_async_wait<STAGES - 1>();
            from_ring(x, 0);
            from_ring(d, 1);
        } else {
            x = x_next;
            d = d_next;
            ds = s_next;
            if (r + step < a.rows) load_next(r + step);
        }
        // outside the row dy = 0, so nothing is added
        F2 q2 = f2(0.f), kx[KEEP ? Row::PAIRS : 1], kg[KEEP ? Row::PAIRS : 1];
#pragma unroll
        for (int p = 0; p < Row::PAIRS; ++p) {
            const F2 dy = d.pair(p), xh = mul2(x.pair(p), rstd), g = a.w ? mul2(dy, w.pair(p)) : dy;
            q2 = fma2(g, xh, q2);
            sw[p] = fma2(dy, xh, sw[p]);
            if constexpr (KEEP) {
                kx[p] = xh;
                kg[p] = g;
            }
        }
        if (a.dx) {
            float q = lanes_sum<LANES>(lo(q2) + hi(q2));
            if (!WARP) {
                if (lane == 0) part[flip][warp] = q;
                __syncthreads();
                q = 0.f;
                for (int k = 0; k < warps; ++k) q += part[flip][k];
                flip ^= 1;
            }
            const F2 mq = f2(-q * inv);
            if constexpr (!KEEP) {
                from_ring(x, 0);
                from_ring(d, 1);
            }
            if constexpr (!KEEP) {
                if (a.ds) ds.load(a.ds + r * a.ldds, t, tpr, n);
            } else if constexpr (RING) {
                if (a.ds) from_ring(ds, 2);
            }
#pragma unroll
            for (int p = 0; p < Row::PAIRS; ++p) {
                F2 xh, g;
                if constexpr (KEEP) {
                    xh = kx[p];
                    g = kg[p];
                } else {
                    xh = mul2(x.pair(p), rstd);
                    g = a.w ? mul2(d.pair(p), w.pair(p)) : d.pair(p);
                }
                g = fma2(xh, mq, g);
                x.set(p, a.ds ? fma2(rstd, g, ds.pair(p)) : mul2(rstd, g));
            }
            if (in) x.store(a.dx + r * a.lddx, t, tpr, n);
        }
        if (++stage == STAGES) stage = 0;
    }
    if (!a.part_w) return;
    float* pw = a.part_w + static_cast<int64_t>(blockIdx.x) * a.H;
    auto column = [&](int e) { return VEC == 1 ? e * tpr + t : ((e / VEC) * tpr + t) * VEC + e % VEC; };
    if constexpr (LANES < 32)  // of the rows of a warp, pair by pair
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1)
#pragma unroll
            for (int p = 0; p < Row::PAIRS; ++p) sw[p] = add2(sw[p], F2{__shfl_xor_sync(0xFFFFFFFFu, sw[p].u, o)});
    if (WARP) {  // the warps' sums, one warp after the other
        float* cols = reinterpret_cast<float*>(dyn + (RING ? STAGES * mats * ITEMS * 128 * sizeof(V) : 0));
        for (int k = 0; k < 4; ++k) {
            if (warp == k && lane < LANES)
#pragma unroll
                for (int e = 0; e < 2 * Row::PAIRS; ++e) {
                    const int c = column(e);
                    if (c < a.H) cols[c] = (k ? cols[c] : 0.f) + (e & 1 ? hi(sw[e / 2]) : lo(sw[e / 2]));
                }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.H; c += 128) pw[c] = cols[c];
    } else {
#pragma unroll
        for (int e = 0; e < 2 * Row::PAIRS; ++e) {
            const int c = column(e);
            if (c < a.H) pw[c] = e & 1 ? hi(sw[e / 2]) : lo(sw[e / 2]);
        }
    }
}

// dx of a block's row, any width.
template <typename T>
__global__ void __launch_bounds__(512) rms_dx_any(RmsBwd<T> a) {
    __shared__ float part[32];
    wait_for_primary();
    const int64_t r = blockIdx.x;
    const T* x = a.x + r * a.ldx;
    const T* dy = a.dy + r * a.ldd;
    const float rstd = a.rstd[r];
    float q = 0.f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x)
        q += to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f) * (to_f32(x[i]) * rstd);
    q = block_sum(q, part) / static_cast<float>(a.H);
    T* dx = a.dx + r * a.lddx;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = to_f32(dy[i]) * (a.w ? load_w<T>(a.w, a.w32, i) : 1.f);
        float v = rstd * (g - to_f32(x[i]) * rstd * q);
        if (a.ds) v += to_f32(a.ds[r * a.ldds + i]);
        dx[i] = from_f32<T>(v);
    }
}

// Column sums of a block of rows: 32 columns per block, 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) rms_dw_any(RmsBwd<T> a) {
    __shared__ float sw[8][33];
    wait_for_primary();
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    const int64_t r0 = blockIdx.y * a.rows_per_part;
    const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
    float w = 0.f;
    if (col < a.H)
        for (int64_t r = r0 + k; r < r1; r += 8)
            w += to_f32(a.dy[r * a.ldd + col]) * (to_f32(a.x[r * a.ldx + col]) * a.rstd[r]);
    sw[k][c] = w;
    __syncthreads();
    if (k == 0 && col < a.H) {
#pragma unroll
        for (int j = 1; j < 8; ++j) w += sw[j][c];
        a.part_w[static_cast<int64_t>(blockIdx.y) * a.H + col] = w;
    }
}

template <typename T, typename W, int VEC, int ITEMS, int R, int STAGES, int MAX_WARPS, int BLOCKS, bool QUANT, int LANES = 32>
lce_status_t rms_rows(const RmsFwd<T>& a, cudaStream_t s) {
    static Resident memo;
    auto kernel = rms_fwd_rows<T, W, VEC, ITEMS, R, STAGES, MAX_WARPS, BLOCKS, QUANT, LANES>;
    const int threads = LANES < 32 ? 32 : threads_for(a.H / VEC, ITEMS);
    const size_t vec = sizeof(Vec<T, VEC>), smem = vec >= 4 ? (a.r ? 2 : 1) * static_cast<size_t>(STAGES) * R * ITEMS * threads * vec : 0;
    const int64_t per = R * 32 / LANES, most = resident_blocks(&memo, kernel, threads, smem), groups = (a.rows + per - 1) / per;
    if (most <= 0) return LCE_ERR_CUDA;
    LCE_PROFILED(launch_after(kernel, dim3(static_cast<unsigned>(groups < most ? groups : most)), threads, smem, s, a));
    return LCE_OK;
}

// The forward's form by the row's width in vectors: 16 bytes where rows start on
// such boundaries (up to 128 a warp per row with the next rows copied ahead, up
// to 512 a block with four a thread, or two rows of two where a quarter of such
// a block would be idle, up to 2048 wider blocks), else 4 bytes, else one
// element, up to 256 of them a warp per row as well.  A thread has as many as the
// row needs.  Measured with a residual: 32768 x 4096 bf16 to 8 bits 154 us, 0.90
// of the copy rate (two or four stages of the ring 168 and 156, eight warps
// 157), 16384 x 1024 bf16 18.6 us, within the copy rate as its writes stay in L2;
// 71723 x 704 fp16 to 8 bits 62 us with three vectors a thread, 72 with four;
// 88770 x 82 bf16 17.9 us, 38.7 by a block with room for eight 4-byte vectors a thread.
template <typename T, typename W, bool QUANT>
lce_status_t rms_forward_as(const RmsCall& c, const RmsFwd<T>& a) {
    cudaStream_t s = c.s;
    constexpr int V = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
    auto fits = [&](int vec) {  // all rows and the weight can be read and written in vectors of `vec`
        const size_t b = vec * sizeof(T), wb = vec * sizeof(W) < 16 ? vec * sizeof(W) : 16;
        return c.H % vec == 0 && c.ldx % vec == 0 && c.ldr % vec == 0 && c.lds % vec == 0 && c.ldy % vec == 0 && c.ldq % vec == 0 &&
               aligned_to(c.x, b) && aligned_to(c.r, b) && aligned_to(c.sum, b) && aligned_to(c.y, b) && aligned_to(c.q, vec) &&
               aligned_to(c.w, wb);
    };
    if (fits(V) && c.H / V <= 2048) {
        const int n = c.H / V;
        if (n <= 8) return rms_rows<T, W, V, 1, 1, 3, 1, 12, QUANT, 8>(a, s);
        if (n <= 16) return rms_rows<T, W, V, 1, 1, 3, 1, 12, QUANT, 16>(a, s);
        if (n <= 32) return rms_rows<T, W, V, 1, 1, 3, 1, 12, QUANT>(a, s);
        if (n <= 64) return rms_rows<T, W, V, 2, 1, 3, 1, 12, QUANT>(a, s);
        if (n <= 96) return rms_rows<T, W, V, 3, 1, 3, 1, 12, QUANT>(a, s);
        if (n <= 128) return rms_rows<T, W, V, 4, 1, 3, 1, 12, QUANT>(a, s);
        if (n <= 512 && 4 * threads_for(n, 4) > n + n / 8) return rms_rows<T, W, V, 2, 2, 2, 8, 2, QUANT>(a, s);
        if (n <= 512) return rms_rows<T, W, V, 4, 1, 3, 4, 4, QUANT>(a, s);
        if (n <= 1024) return rms_rows<T, W, V, 4, 1, 3, 8, 2, QUANT>(a, s);
        return rms_rows<T, W, V, 4, 1, 3, 16, 1, QUANT>(a, s);
    }
    if (V4 > 1 && fits(V4) && c.H / V4 <= 4096) {
        if (c.H / V4 <= 64) return rms_rows<T, W, V4, 2, 1, 3, 1, 12, QUANT>(a, s);
        if (c.H / V4 <= 128) return rms_rows<T, W, V4, 4, 1, 3, 1, 12, QUANT>(a, s);
        if (c.H / V4 <= 256) return rms_rows<T, W, V4, 8, 1, 3, 1, 12, QUANT>(a, s);
        return rms_rows<T, W, V4, 8, 1, 3, 16, 1, QUANT>(a, s);
    }
    if (c.H <= 128) return rms_rows<T, W, 1, 4, 1, 3, 1, 12, QUANT>(a, s);
    if (c.H <= 256) return rms_rows<T, W, 1, 8, 1, 3, 1, 12, QUANT>(a, s);
    if (c.H <= 4096) return rms_rows<T, W, 1, 8, 1, 3, 16, 1, QUANT>(a, s);
    if (c.H <= 8192) return rms_rows<T, W, 1, 16, 1, 3, 16, 1, QUANT>(a, s);
    LCE_PROFILED(launch_after(rms_fwd_any<T, QUANT>, dim3(static_cast<unsigned>(c.rows)), 512, 0, s, a));
    return LCE_OK;
}

template <typename T, typename W>
lce_status_t rms_forward(const RmsCall& c) {
    const RmsFwd<T> a{static_cast<const T*>(c.x), static_cast<const T*>(c.r), c.ldx, c.ldr, c.w, c.w32, c.eps,
                      static_cast<T*>(c.sum), c.lds, static_cast<T*>(c.y), c.ldy, c.q, c.ldq, c.scales, c.group,
                      (c.H + c.group - 1) / c.group, c.rstd_out, c.rows, c.H};
    return c.q ? rms_forward_as<T, W, true>(c, a) : rms_forward_as<T, W, false>(c, a);
}

// The backward's form by the row's width, as layer norm's (lce_norm.cuh): up to
// 128 16-byte vectors a warp per row, up to 1024 a block with two vectors a
// thread, up to 2048 with four, read twice from the ring; narrower vectors up to
// eight a thread, a warp per row where that covers it (30000 x 250 bf16: 17.7 us
// with four, 25.1 with eight, a block per row 54; 88770 x 82 25.5 with two, 55.5
// with eight), or sixteen single elements; wider rows are read again.
// Measured with the sum's gradient: 16384 x 1024 bf16 27 us (the copy rate
// would be 20), 65536 x 2560 without it 155 us (148).
template <typename T, typename W, int VEC, int ITEMS, bool WARP, bool KEEP, int LANES = 32>
lce_status_t rms_bwd(const RmsBwd<T>& a, int* parts, cudaStream_t s) {
    static Resident memo;
    auto kernel = rms_bwd_rows<T, W, VEC, ITEMS, WARP, KEEP, LANES>;
    const int threads = WARP ? 128 : threads_for(a.H / VEC, ITEMS);
    const size_t vec = sizeof(Vec<T, VEC>), ring = vec >= 4 ? RMS_BWD_STAGES * (KEEP && a.ds ? 3 : 2) * ITEMS * threads * vec : 0;
    const size_t smem = ring + (WARP ? static_cast<size_t>(a.H) * 4 : 0);
    int64_t blocks = resident_blocks(&memo, kernel, threads, smem);
    if (blocks <= 0) return LCE_ERR_CUDA;
    constexpr int PER = WARP ? 4 * 32 / LANES : 1;  // rows of a block at a time
    const int64_t work = (a.rows + PER - 1) / PER;
    if (blocks > work) blocks = work;
    if (blocks > NORM_PARTS) blocks = NORM_PARTS;
    *parts = static_cast<int>(blocks);
    LCE_PROFILED(launch_after(kernel, dim3(static_cast<unsigned>(blocks)), threads, smem, s, a));
    return LCE_OK;
}

template <typename T, typename W>
lce_status_t rms_backward(const RmsCall& c) {
    RmsBwd<T> a{static_cast<const T*>(c.dy), static_cast<const T*>(c.x), static_cast<const T*>(c.ds), c.ldd, c.ldx, c.ldds,
                c.w, c.w32, c.rstd, static_cast<T*>(c.y), c.ldy, c.parts, c.rows, 0, c.H};
    cudaStream_t s = c.s;
    constexpr int V = vec16<T>(), V4 = 4 / static_cast<int>(sizeof(T));
    auto fits = [&](int vec) {
        const size_t b = vec * sizeof(T), wb = vec * sizeof(W) < 16 ? vec * sizeof(W) : 16;
        return c.H % vec == 0 && c.ldx % vec == 0 && c.ldd % vec == 0 && c.ldds % vec == 0 && c.ldy % vec == 0 && aligned_to(c.x, b) &&
               aligned_to(c.dy, b) && aligned_to(c.ds, b) && aligned_to(c.y, b) && aligned_to(c.w, wb);
    };
    int parts = 0;
    lce_status_t st = LCE_OK;
    if (fits(V) && c.H / V <= 2048) {
        const int n = c.H / V;
        st = n <= 8      ? rms_bwd<T, W, V, 1, true, true, 8>(a, &parts, s)
             : n <= 16   ? rms_bwd<T, W, V, 1, true, true, 16>(a, &parts, s)
             : n <= 32   ? rms_bwd<T, W, V, 1, true, true>(a, &parts, s)
             : n <= 64   ? rms_bwd<T, W, V, 2, true, true>(a, &parts, s)
             : n <= 96   ? rms_bwd<T, W, V, 3, true, true>(a, &parts, s)
             : n <= 128  ? rms_bwd<T, W, V, 4, true, true>(a, &parts, s)
             : n <= 1024 ? rms_bwd<T, W, V, 2, false, true>(a, &parts, s)
                         : rms_bwd<T, W, V, 4, false, false>(a, &parts, s);
    } else if (V4 > 1 && fits(V4) && c.H / V4 <= 4096) {
        const int n = c.H / V4;
        st = n <= 64    ? rms_bwd<T, W, V4, 2, true, true>(a, &parts, s)
             : n <= 128 ? rms_bwd<T, W, V4, 4, true, true>(a, &parts, s)
             : n <= 256 ? rms_bwd<T, W, V4, 8, true, true>(a, &parts, s)
                        : rms_bwd<T, W, V4, 8, false, true>(a, &parts, s);
    } else if (c.H <= 4096) {
        st = c.H <= 128   ? rms_bwd<T, W, 1, 4, true, true>(a, &parts, s)
             : c.H <= 256 ? rms_bwd<T, W, 1, 8, true, true>(a, &parts, s)
                          : rms_bwd<T, W, 1, 8, false, true>(a, &parts, s);
    } else if (c.H <= 8192) {
        st = rms_bwd<T, W, 1, 16, false, sizeof(T) == 2>(a, &parts, s);  // (a ring with ds would be 295 KB in fp32)
    } else {
        if (c.y) LCE_PROFILED(launch_after(rms_dx_any<T>, dim3(static_cast<unsigned>(c.rows)), 512, 0, s, a));
        if (c.dw) {
            a.rows_per_part = (c.rows + NORM_PARTS - 1) / NORM_PARTS;
            if (a.rows_per_part < 32) a.rows_per_part = 32;
            parts = static_cast<int>((c.rows + a.rows_per_part - 1) / a.rows_per_part);
            LCE_PROFILED(launch_after(rms_dw_any<T>, dim3((c.H + 31) / 32, parts), 256, 0, s, a));
        }
    }
    if (st != LCE_OK || !c.dw) return st;
    LCE_PROFILED(launch_after(norm_dw_join<W>, dim3((c.H + 31) / 32), 1024, 0, s,
                              JoinArgs{a.part_w, nullptr, parts, c.H, c.dw, nullptr}));
    return LCE_OK;
}

}  // namespace
}  // namespace lce
