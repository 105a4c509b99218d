// gdn_books.cuh -- prefix sums and searches of the page bookkeeping kernels (gdn_kv.cu, gdn_pages.cu): a cluster of CTAs each of
// which scans all sequences for itself.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

struct Pair {
    long long rows, pages;
};

// Exclusive prefix sums of one Pair a thread over the block; *total = the sums of all.
// Every thread of the block calls it; `sums` is shared, 33 entries.
__device__ __forceinline__ Pair block_prefix(Pair v, Pair* sums, Pair* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    Pair x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long r = __shfl_up_sync(0xffffffffu, x.rows, o), g = __shfl_up_sync(0xffffffffu, x.pages, o);
        if (lane >= o) {
            x.rows += r;
            x.pages += g;
        }
    }
    __syncthreads();   // the last use of sums is over
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const Pair s = lane < n_warps ? sums[lane] : Pair{0, 0};
        Pair t = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long r = __shfl_up_sync(0xffffffffu, t.rows, o), g = __shfl_up_sync(0xffffffffu, t.pages, o);
            if (lane >= o) {
                t.rows += r;
                t.pages += g;
            }
        }
        if (lane < n_warps) sums[lane] = Pair{t.rows - s.rows, t.pages - s.pages};
        if (lane == 31) sums[32] = t;
    }
    __syncthreads();
    *total = sums[32];
    return Pair{sums[warp].rows + x.rows - v.rows, sums[warp].pages + x.pages - v.pages};
}

// The last i in 0..n-1 with a[i] <= x (a[0] <= x, a not decreasing).
__device__ __forceinline__ int find(const int* a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}

}  // namespace gdn
