// gdn_chunk.cuh -- what the kernels of gdn_attn_chunk (include/gdn_attn.h) share: the sequences and a worker's share of the
// work (gdn_chunk_plan.h), results, and the join of units that several workers hold parts of.
//
// Mathematics, as in gdn_attn.cuh: over any set of keys a row has m = max s, l = sum 2^(s-m), o = sum 2^(s-m) v with scores in
// base 2 (s log2 e); two sets join as m = max(m1, m2), l = l1 2^(m1-m) + l2 2^(m2-m), o likewise, and o / l is the result
// once.  A row that sees no key has m = -inf, l = 0 and the result 0.
#pragma once

#include "gdn_attn.cuh"
#include "gdn_chunk_plan.h"

namespace gdn {
namespace chunk {

using attn::kLog2e;

constexpr int kMaxWorkers = 512;
// At the start of the workspace: by the worker of a unit's first part, two for each pair of CTAs; behind kMaxWorkers of them by the
// worker of the first of some parts of a unit, two each for whether it is the unit's first one.
constexpr size_t kCounterBytes = 4 * kMaxWorkers * 4;

__device__ __forceinline__ bool rows_ok(const ChunkParams& p, int a, int z) { return a >= 0 && a <= z && z <= p.T; }

// Keys that a sequence can have: what its row of the table names, and few enough that a tile past them still has a number of 31 bits.
__device__ __forceinline__ long long most_keys(const ChunkParams& p) {
    return least(static_cast<long long>(p.max_pages) * p.cache.page_size, INT32_MAX - 4096);
}

__device__ __forceinline__ Rows rows_of(const ChunkParams& p, int b) {
    const int a = p.cu_seqlens[b], z = p.cu_seqlens[b + 1];
    Rows r{a, 0, static_cast<int>(least(most(p.seq_len[b], 0), most_keys(p)))};
    if (rows_ok(p, a, z)) r.n = z - a;
    return r;
}

// What only the device sees of sequence b's arguments.
__device__ __forceinline__ void report_rows(const ChunkParams& p, int b) {
    if (!rows_ok(p, p.cu_seqlens[b], p.cu_seqlens[b + 1]) || p.seq_len[b] > most_keys(p)) atomicOr(p.status + b, kKvBadIndex);
}

// On to the worker's next part (gdn_chunk_plan.h).  A call: it comes once a part in several places of a kernel, and inlined its
// divisions made a kernel of 200 KB, whose warps waited for instructions a third of their time.
static __device__ __noinline__ bool to_next_part(const ChunkParams& p, const Line& ln, const Share& sh, Part& c) {
    return next_part(ln, sh, p.B, p.heads, c, [&](int b) { return rows_of(p, b); });
}

struct PlanSmem {
    long long sums[32], start;   // by warp
    int start_b;
};

// This worker's share and its first part; false if it has none.  All threads of a CTA call it.
__device__ __forceinline__ bool my_share(const ChunkParams& p, const Line& ln, int worker, int workers, int min_share, PlanSmem& sm, Share& sh, Part& c) {
    grid_dependency_wait();   // launched as a programmatic dependent: nothing global is touched before the previous kernel is done
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = static_cast<int>(blockDim.x);
    const int per = (p.B + threads - 1) / threads;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        mine += p.heads * ln.head(rows_of(p, b));
        if (worker == 0 && p.status) report_rows(p, b);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm.sums[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < threads / 32; ++w) {
        if (w < warp) before += sm.sums[w];
        total += sm.sums[w];
    }
    before += incl - mine;
    const int n = total > 0 ? workers_of(total, workers, min_share) : 0;
    if (worker >= n) return false;
    sh = Share::of(total, n, worker);
    if (sh.first >= before && sh.first < before + mine) {   // one thread: its sequences hold the first number
        long long at = before;
        int b = b0;
        for (; b < b1 - 1; ++b) {
            const long long h = p.heads * ln.head(rows_of(p, b));
            if (sh.first < at + h) break;
            at += h;
        }
        sm.start_b = b;
        sm.start = at;
    }
    __syncthreads();
    grid_launch_dependents();
    c.b = sm.start_b;
    c.r = rows_of(p, c.b);
    return first_part(ln, sh, sm.start, c) || to_next_part(p, ln, sh, c);
}

// Rows of a unit, and of row r its token (of the unit) and query head.
__device__ __forceinline__ int tokens_of(const Line& ln, const Part& c) {
    return static_cast<int>(least(ln.tokens, c.r.n - static_cast<long long>(c.i) * ln.tokens));
}

// A row's channels ch..ch+3 of the result, gated.
template <typename Ta, int D, bool add = false>
__device__ __forceinline__ void put(const ChunkParams& p, bool out_bf16, long long t, int h, int ch, float4 y) {
    if (p.gate) {
        const float4 g = StateIO<Ta>::ld(static_cast<const Ta*>(p.gate) + t * p.ldg + static_cast<long long>(h) * D + ch);
        y.x *= gate_of(g.x);
        y.y *= gate_of(g.y);
        y.z *= gate_of(g.z);
        y.w *= gate_of(g.w);
    }
    const long long at = (t * p.Hq + h) * D + ch;
    if (add) {
        const float4 x = out_bf16 ? StateIO<__nv_bfloat16>::ld(static_cast<const __nv_bfloat16*>(p.out) + at)
                                  : StateIO<float>::ld(static_cast<const float*>(p.out) + at);
        y = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    if (out_bf16) StateIO<__nv_bfloat16>::st(static_cast<__nv_bfloat16*>(p.out) + at, y);
    else StateIO<float>::st(static_cast<float*>(p.out) + at, y);
}

// Parts of split units: two places a worker, 2 w for one that goes on from the worker before, 2 w + 1 for one that begins here.
template <int RT, int D>
struct Parts {
    int* counters;
    float* o;      // [2 workers][RT][D], on 32 bytes
    float2* ml;    // [2 workers][RT]
    __device__ __forceinline__ Parts(void* workspace, int workers)
        : counters(static_cast<int*>(workspace)),
          o(reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + kCounterBytes + 31) & ~static_cast<uintptr_t>(31))),
          ml(reinterpret_cast<float2*>(o + static_cast<size_t>(2) * workers * RT * D)) {}
    __device__ __forceinline__ static size_t place(int worker, const Part& c) { return 2 * static_cast<size_t>(worker) + (c.t0 == 0); }
};
template <int RT, int D>
constexpr size_t parts_bytes(int workers) {
    return kCounterBytes + 32 + static_cast<size_t>(2) * workers * RT * (D * 4 + 8);
}

// bf16 cache; *done = false where there is no tensor map of the strides.
cudaError_t launch_tc(const ChunkParams& p, int head_dim, bool out_bf16, int sms, bool* done, cudaStream_t stream);
size_t tc_workspace_bytes(int head_dim, bool out_bf16);

}  // namespace chunk
}  // namespace gdn
