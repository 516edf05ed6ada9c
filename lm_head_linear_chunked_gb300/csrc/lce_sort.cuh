// A stable counting sort by one digit, in two kernels: every block counts the
// digits of its share of the items, then every block adds up what the others
// have counted and puts its items in their places (one block needs the second
// kernel alone).  The places depend on the
// items alone, so what is summed in the sorted order has equal bits every time.
//
// What the items are is up to a functor F:
//   Item load(int64_t i, bool* bad)   item i, whose `digit` lies in [0, bins)
//   void put(const Item& x, int32_t at)   x belongs at place `at`
//   void begin()   called by all threads of all blocks before anything is put
//   static constexpr bool SEGMENTS: whether digits have segments that start on
//     multiples of f.align, the last digit (items to leave out) in none;
//     then also segment(d, count, start), called by one thread per digit, and
//     ends(end), one past the last segment, called by all threads of all blocks
//   void status(int any)   with shape.bad: whether an item was bad, once
//   void beside(int kernel, int64_t block, int64_t of)   called by all threads
//     of the shape's `extra` blocks of each kernel (counting 0, placing 1): work
//     that needs nothing sorted, for the SMs that so few items leave idle; only
//     where both kernels run.  The next kernel is launched when they have ended:
//     earlier, its blocks would crowd onto the first SMs that are free
#pragma once

#include <atomic>

#include "lce_internal.cuh"
#include "lce_vec.cuh"

namespace lce {

// A block is as large as it can be, as every block adds up what all the others
// have counted: 131072 items in 64 blocks of 1024 threads, not 128 of 256.
constexpr int SORT_WARPS = 32;
constexpr int SORT_THREADS = 32 * SORT_WARPS;
constexpr int SORT_BINS_MAX = 1025;
constexpr int64_t SORT_ALONE = 4096;  // items that one block sorts by itself
constexpr int64_t SORT_ITEMS = 2048;  // a block's fewest where there are more
constexpr int64_t SORT_BLOCKS = 152;

struct SortShape {
    int64_t n, per;  // items, and items of a block
    int32_t bins, blocks, extra;
    int32_t* hist;   // [blocks, bins]
    int32_t* bad;    // [blocks]: a block has seen an item out of range
};

inline int64_t sort_blocks(int64_t n) {
    const int64_t b = n <= SORT_ALONE ? 1 : (n + SORT_ITEMS - 1) / SORT_ITEMS;
    return b < SORT_BLOCKS ? b : SORT_BLOCKS;
}
inline size_t sort_smem(int bins) { return static_cast<size_t>(SORT_WARPS) * bins * 4; }

namespace {

template <typename F>
struct SortJob {
    F f;
    SortShape shape;
};

// Calls g(item, whether there is one) for the items i, i + step, ... before end,
// loading several at a time: a block has few, and waits for each load.
template <typename F, typename G>
__device__ __forceinline__ void sort_items(const F& f, int64_t i, int64_t end, int64_t step, bool* bad, G g) {
    constexpr int AHEAD = 4;
    const int64_t lane = threadIdx.x & 31;
    for (; i - lane < end; i += AHEAD * step) {  // the lanes of a warp stay together
        typename F::Item x[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i + k * step < end) x[k] = f.load(i + k * step, bad);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (i - lane + k * step >= end) break;
            g(x[k], i + k * step < end);
        }
    }
}

template <typename F>
__global__ void __launch_bounds__(SORT_THREADS) sort_count(SortJob<F> job) {
    const F& f = job.f;
    const SortShape& s = job.shape;
    extern __shared__ __align__(16) int32_t counts[];
    if (static_cast<int>(blockIdx.x) >= s.blocks) {
        wait_for_primary();
        return f.beside(0, blockIdx.x - s.blocks, s.extra);
    }
    launch_dependents();
    for (int d = threadIdx.x; d < s.bins; d += SORT_THREADS) counts[d] = 0;
    wait_for_primary();
    const int64_t i0 = blockIdx.x * s.per, i1 = i0 + s.per < s.n ? i0 + s.per : s.n;
    bool bad = false;
    f.begin();
    __syncthreads();
    sort_items(f, i0 + threadIdx.x, i1, SORT_THREADS, &bad, [&](const typename F::Item& x, bool in) {
        if (in) atomicAdd(counts + x.digit, 1);
    });
    const int any = __syncthreads_or(bad);
    for (int d = threadIdx.x; d < s.bins; d += SORT_THREADS) s.hist[static_cast<int64_t>(blockIdx.x) * s.bins + d] = counts[d];
    if (threadIdx.x == 0 && s.bad) s.bad[blockIdx.x] = any;
}

// Puts a block's items in their places.
template <typename F>
__device__ __forceinline__ void place_items(const F& f, const SortShape& s) {
    extern __shared__ __align__(16) int32_t counts[];  // [SORT_WARPS, bins]: of each warp's items, then their places
    __shared__ int32_t sums[SORT_WARPS];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    for (int d = t; d < SORT_WARPS * s.bins / 4; d += SORT_THREADS) reinterpret_cast<int4*>(counts)[d] = make_int4(0, 0, 0, 0);
    wait_for_primary();
    const bool alone = s.blocks == 1;  // nothing has been counted before
    bool bad = false;
    if (alone) f.begin();
    __syncthreads();
    // each warp a stretch of the block's items
    const int64_t i0 = blockIdx.x * s.per, i1 = i0 + s.per < s.n ? i0 + s.per : s.n;
    const int64_t share = (s.per + SORT_THREADS - 1) / SORT_THREADS * 32;
    const int64_t w0 = i0 + warp * share, w1 = w0 + share < i1 ? w0 + share : i1;
    int32_t* own = counts + warp * s.bins;
    sort_items(f, w0 + lane, w1, 32, &bad, [&](const typename F::Item& x, bool in) {
        if (in) atomicAdd(own + x.digit, 1);
    });
    // each thread a stretch of the digits: their items in all blocks, and in those before this one
    constexpr int MOST = (SORT_BINS_MAX + SORT_THREADS - 1) / SORT_THREADS;
    const int each = (s.bins + SORT_THREADS - 1) / SORT_THREADS;
    int32_t total[MOST], before[MOST], mine = 0;
    if (alone) bad = __syncthreads_or(bad);
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        const int d = t * each + j;
        total[j] = before[j] = 0;
        if (j < each && d < s.bins) {
            if (alone) {
#pragma unroll
                for (int w = 0; w < SORT_WARPS; ++w) total[j] += counts[w * s.bins + d];
            } else {
                for (int b0 = 0; b0 < s.blocks; b0 += 16) {  // sixteen loads on their way
                    int32_t c[16];
#pragma unroll
                    for (int b = 0; b < 16; ++b) c[b] = b0 + b < s.blocks ? s.hist[static_cast<int64_t>(b0 + b) * s.bins + d] : 0;
#pragma unroll
                    for (int b = 0; b < 16; ++b) {
                        total[j] += c[b];
                        before[j] += b0 + b < static_cast<int>(blockIdx.x) ? c[b] : 0;
                    }
                }
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
    int32_t start = upto - mine + warp_sum(lane < warp ? sums[lane] : 0);
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        const int d = t * each + j;
        if (j >= each || d >= s.bins) break;
        int32_t at = start + before[j], c[SORT_WARPS];
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) c[w] = counts[w * s.bins + d];
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            counts[w * s.bins + d] = at;
            at += c[w];
        }
        if constexpr (F::SEGMENTS) {
            if (d % s.blocks == static_cast<int>(blockIdx.x)) f.segment(d, total[j], start);
            start += (total[j] + f.align - 1) / f.align * f.align;
        } else {
            start += total[j];
        }
    }
    __syncthreads();
    sort_items(f, w0 + lane, w1, 32, &bad, [&](const typename F::Item& x, bool in) {
        const unsigned active = __ballot_sync(0xFFFFFFFFu, in);
        if (in) {
            unsigned same = active;  // the lanes with this digit, bit by bit: a match instruction took longer
#pragma unroll
            for (int b = 0; b < 11; ++b) {
                if (s.bins - 1 >> b == 0) break;
                const unsigned ones = __ballot_sync(active, x.digit >> b & 1);
                same &= x.digit >> b & 1 ? ones : ~ones;
            }
            const int32_t at = own[x.digit] + __popc(same & ((1u << lane) - 1));
            __syncwarp(active);
            if ((same >> lane) == 1u) own[x.digit] = at + 1;  // the last of them
            f.put(x, at);
        }
        __syncwarp();
    });
    if constexpr (F::SEGMENTS) f.ends(warp_sum(lane < SORT_WARPS ? sums[lane] : 0));
    if (s.bad && blockIdx.x == 0) {
        const int any = alone ? bad : __syncthreads_or(t < s.blocks && s.bad[t]);
        if (t == 0) f.status(any);
    }
}

template <typename F>
__global__ void __launch_bounds__(SORT_THREADS) sort_place(SortJob<F> job) {
    if (static_cast<int>(blockIdx.x) >= job.shape.blocks) {
        wait_for_primary();
        return job.f.beside(1, blockIdx.x - job.shape.blocks, job.shape.extra);
    }
    launch_dependents();
    place_items(job.f, job.shape);
}

// Lets a kernel take `bytes` of dynamic shared memory, out of the largest share
// of an SM's: kernels that overlap with the one before them need the same
// division into L1 and shared memory.  Asked once per device.
template <typename K>
bool allow_smem(std::atomic<uint64_t>* known, K kernel, int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (known->load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return false;
    known->fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Sorts by one digit.
template <typename F>
lce_status_t sort_by(const F& f, const SortShape& shape, cudaStream_t s) {
    static std::atomic<uint64_t> counts{0}, places{0};
    if (!allow_smem(&counts, sort_count<F>, SORT_BINS_MAX * 4) ||
        !allow_smem(&places, sort_place<F>, static_cast<int>(sort_smem(SORT_BINS_MAX))))
        return LCE_ERR_CUDA;
    const SortJob<F> job{f, shape};
    const dim3 blocks(static_cast<unsigned>(shape.blocks + shape.extra));
    if (shape.blocks > 1)
        LCE_PROFILED(launch_after(sort_count<F>, blocks, SORT_THREADS, static_cast<size_t>(shape.bins) * 4, s, job));
    LCE_PROFILED(launch_after(sort_place<F>, blocks, SORT_THREADS, sort_smem(shape.bins), s, job));
    return LCE_OK;
}

}  // namespace
}  // namespace lce
