// What the norms' kernels share: how a row lies in a block's registers, sums
// over a block, the joining of column sums, and the number of resident blocks.
#pragma once

#include <atomic>

#include "lce_vec.cuh"

namespace lce {

// Parts of the weight gradient's sum over the rows: at most four blocks on each of 152 SMs.
constexpr int64_t NORM_PARTS = 608;
// Dynamic shared memory of a block; the widest ring takes 192 KB of it.
constexpr int NORM_SMEM_MAX = 224 * 1024;

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

}  // namespace
}  // namespace lce
