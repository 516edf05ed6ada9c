// A stable counting sort by one digit, in two kernels: every block counts the
// digits of its share of the items, then every block adds up what the others
// have counted and puts its items in their places.  The places depend on the
// items alone, so what is summed in the sorted order has equal bits every time.
//
// What the items are is up to a functor F:
//   int32_t digit(int64_t i, bool* bad)   item i's digit in [0, bins)
//   void put(int64_t i, int32_t d, int32_t at)   item i belongs at place `at`
//   static constexpr bool SEGMENTS: whether digits have segments that start on
//     multiples of f.align, the last digit (items to leave out) in none;
//     then also segment(d, count, start), called by one thread per digit, and
//     ends(end), one past the last segment, called by all threads of all blocks
//   void begin()   called by all threads of all blocks of the counting
//   void status(int any)   with shape.bad: whether an item was bad, once
#pragma once

#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {

constexpr int SORT_WARPS = 8;
constexpr int SORT_THREADS = 32 * SORT_WARPS;
constexpr int SORT_BINS_MAX = 1025;  // (SORT_WARPS + 1) counters each fit the 48 KB of a block without asking
constexpr int64_t SORT_ITEMS = 1024; // a block's fewest
constexpr int64_t SORT_BLOCKS = 152;

struct SortShape {
    int64_t n, per;  // items, and items of a block
    int32_t bins, blocks;
    int32_t* hist;   // [blocks, bins]
    int32_t* bad;    // [blocks]: a block has seen an item out of range
};

inline int64_t sort_blocks(int64_t n) {
    const int64_t b = (n + SORT_ITEMS - 1) / SORT_ITEMS;
    return b < 1 ? 1 : (b < SORT_BLOCKS ? b : SORT_BLOCKS);
}
inline size_t sort_smem(int bins) { return static_cast<size_t>(SORT_WARPS + 1) * bins * 4; }

namespace {

template <typename F>
struct SortJob {
    F f;
    SortShape shape;
};

template <typename F>
__global__ void __launch_bounds__(SORT_THREADS) sort_count(SortJob<F> job) {
    const F& f = job.f;
    const SortShape& s = job.shape;
    extern __shared__ int32_t counts[];
    launch_dependents();
    for (int d = threadIdx.x; d < s.bins; d += SORT_THREADS) counts[d] = 0;
    wait_for_primary();
    const int64_t i0 = blockIdx.x * s.per, i1 = i0 + s.per < s.n ? i0 + s.per : s.n;
    bool bad = false;
    f.begin();
    __syncthreads();
    for (int64_t i = i0 + threadIdx.x; i < i1; i += SORT_THREADS) atomicAdd(counts + f.digit(i, &bad), 1);
    const int any = __syncthreads_or(bad);
    for (int d = threadIdx.x; d < s.bins; d += SORT_THREADS) s.hist[static_cast<int64_t>(blockIdx.x) * s.bins + d] = counts[d];
    if (threadIdx.x == 0 && s.bad) s.bad[blockIdx.x] = any;
}

template <typename F>
__global__ void __launch_bounds__(SORT_THREADS) sort_place(SortJob<F> job) {
    const F& f = job.f;
    const SortShape& s = job.shape;
    extern __shared__ int32_t counts[];  // [SORT_WARPS, bins], then [bins]
    __shared__ int32_t sums[SORT_WARPS];
    launch_dependents();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    int32_t* first = counts + SORT_WARPS * s.bins;
    for (int d = t; d < SORT_WARPS * s.bins; d += SORT_THREADS) counts[d] = 0;
    wait_for_primary();
    // each thread a stretch of the digits: their items in all blocks, and in those before this one
    constexpr int MOST = (SORT_BINS_MAX + SORT_THREADS - 1) / SORT_THREADS;
    const int each = (s.bins + SORT_THREADS - 1) / SORT_THREADS;
    int32_t total[MOST], before[MOST], mine = 0;
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        const int d = t * each + j;
        total[j] = before[j] = 0;
        if (j < each && d < s.bins) {
#pragma unroll 16
            for (int b = 0; b < s.blocks; ++b) {
                const int32_t c = s.hist[static_cast<int64_t>(b) * s.bins + d];
                total[j] += c;
                before[j] += b < static_cast<int>(blockIdx.x) ? c : 0;
            }
        }
        if constexpr (F::SEGMENTS) {
            if (d == s.bins - 1) total[j] = 0;  // left out
            mine += (total[j] + f.align - 1) / f.align * f.align;
        } else {
            mine += total[j];
        }
    }
    int32_t upto = mine;  // inclusive scan over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int32_t start = upto - mine;
    for (int w = 0; w < warp; ++w) start += sums[w];
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        const int d = t * each + j;
        if (j >= each || d >= s.bins) break;
        first[d] = start + before[j];
        if constexpr (F::SEGMENTS) {
            if (d % s.blocks == static_cast<int>(blockIdx.x)) f.segment(d, total[j], start);
            start += (total[j] + f.align - 1) / f.align * f.align;
        } else {
            start += total[j];
        }
    }
    // each warp a stretch of the block's items, counted, then put one after the other
    const int64_t i0 = blockIdx.x * s.per, i1 = i0 + s.per < s.n ? i0 + s.per : s.n;
    const int64_t share = (s.per + 32 * SORT_WARPS - 1) / (32 * SORT_WARPS) * 32;
    const int64_t w0 = i0 + warp * share, w1 = w0 + share < i1 ? w0 + share : i1;
    int32_t* own = counts + warp * s.bins;
    bool bad = false;
    for (int64_t i = w0 + lane; i < w1; i += 32) atomicAdd(own + f.digit(i, &bad), 1);
    __syncthreads();
    for (int d = t; d < s.bins; d += SORT_THREADS) {
        int32_t at = first[d];
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            const int32_t c = counts[w * s.bins + d];
            counts[w * s.bins + d] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t base = w0; base < w1; base += 32) {
        const int64_t i = base + lane;
        const bool in = i < w1;
        const unsigned active = __ballot_sync(0xFFFFFFFFu, in);
        if (in) {
            const int32_t d = f.digit(i, &bad);
            const unsigned same = __match_any_sync(active, d);
            const int32_t at = own[d] + __popc(same & ((1u << lane) - 1));
            __syncwarp(active);
            if ((same >> lane) == 1u) own[d] = at + 1;  // the last of them
            f.put(i, d, at);
        }
        __syncwarp();
    }
    if constexpr (F::SEGMENTS) {
        int32_t end = 0;
        for (int w = 0; w < SORT_WARPS; ++w) end += sums[w];
        f.ends(end);
    }
    if (s.bad && blockIdx.x == 0 && t == 0) {
        int any = 0;
        for (int b = 0; b < s.blocks; ++b) any |= s.bad[b];
        f.status(any);
    }
}

// Sorts by one digit; `first`: after all that came before it in the stream,
// else under the kernel before it, whose results it waits for.
template <typename F>
lce_status_t sort_by(const F& f, const SortShape& shape, bool first, cudaStream_t s) {
    const SortJob<F> job{f, shape};
    const unsigned blocks = static_cast<unsigned>(shape.blocks);
    if (first)
        LCE_PROFILED(sort_count<F><<<blocks, SORT_THREADS, static_cast<size_t>(shape.bins) * 4, s>>>(job));
    else
        LCE_PROFILED(launch_after(sort_count<F>, dim3(blocks), SORT_THREADS, static_cast<size_t>(shape.bins) * 4, s, job));
    LCE_PROFILED(launch_after(sort_place<F>, dim3(blocks), SORT_THREADS, sort_smem(shape.bins), s, job));
    return LCE_OK;
}

}  // namespace
}  // namespace lce
