// gdn_norm.cu -- the norms either side of a block with its gate and residual connection
// (include/gdn_norm.h, gdn_norm_residual).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "gdn_norm.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

// Elementwise but for one or two sums over a row, every element read and written once: bound by the memory.  A row
// is held in registers between its passes: with 16-byte accesses (8 channels a thread and chunk) by a CTA, or
// by 1 to 32 lanes of one where it has at most 256 channels (32768 rows of 256, bf16: 18 us against 34 by a CTA a row).
// The fp32 weights come from L1 after the first row of an SM.  Measured: 8192 rows of 5120, fp32 stream, gate and scale
// (587 MB): 98 us, 6.0 TB/s; 64 rows of 2048: 2.7 us, the latency of a launch, its loads and two sums.  Rows off 16 bytes, one element
// a thread at a time: 8192 of 5119 216 us (bf16 206).

__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += s[w];
    return t;
}

constexpr int kAhead = 304;   // rows: two for each of the 152 SMs

// N chunks a thread.  lanes > 0: that many lanes (a power of two <= 32) share a row, several rows a CTA; lanes == 0: a CTA a row.
template <typename Ta, typename Tr, int N>
__global__ void __launch_bounds__(512, N <= 2 ? 2 : 1) norm_residual_kernel(NormParams p, int lanes) {
    __shared__ float sums[16];
    grid_dependency_wait();
    grid_launch_dependents();
    const long long t = lanes ? static_cast<long long>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes : blockIdx.x;
    const int i0 = lanes ? threadIdx.x % lanes : threadIdx.x, step = blockDim.x;
    const int chunks = p.H / 8;
    const bool live = t < p.T;
    auto sum = [&](float v) {
        if (!lanes) return block_sum(v, sums);
        for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    Raw8<Ta> y[N], g[N];
    Raw8<Tr> h[N];
    float g1 = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const int i = i0 + c * step;
        if (live && i < chunks) {
            h[c].load(static_cast<const Tr*>(p.h) + t * p.H + i * 8);
            if (p.y) y[c].load(static_cast<const Ta*>(p.y) + t * p.ldy + i * 8);
            if (p.gate_cols > 1) g[c].load(static_cast<const Ta*>(p.gate) + t * p.ldg + i * 8);
        }
    }
    // A row waits for its sums twice, and the rows that fit an SM meanwhile do not keep the memory busy: the row that a later
    // CTA will take is brought into L2 (8192 x 5120, with a gate of fewer bits: 106.6 -> 95.7 us; 456 rows ahead 96.5, 1000 rows 106).
    if (!lanes && t + kAhead < p.T) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const int i = i0 + c * step;
            if (i < chunks && i % (16 / static_cast<int>(sizeof(Tr))) == 0) prefetch_l2(static_cast<const Tr*>(p.h) + (t + kAhead) * p.H + i * 8);
            if (i < chunks && i % (16 / static_cast<int>(sizeof(Ta))) == 0) {
                if (p.y) prefetch_l2(static_cast<const Ta*>(p.y) + (t + kAhead) * p.ldy + i * 8);
                if (p.gate_cols > 1) prefetch_l2(static_cast<const Ta*>(p.gate) + (t + kAhead) * p.ldg + i * 8);
            }
        }
    }
    if (live && p.gate_cols == 1) g1 = gate_of<sizeof(Tr) == 4>(ld_act(static_cast<const Ta*>(p.gate) + t * p.ldg));
    float r = 1.f;
    if (p.post_w) {
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (live && i0 + c * step < chunks) {
                float u[8];
                y[c].get(u);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
            }
        r = 1.0f / sqrtf(sum(ss) / p.H + p.eps);
    }
    float v[N][8], ss = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const int i = i0 + c * step;
        if (!live || i >= chunks) continue;
        h[c].get(v[c]);
        if (p.y) {
            float u[8], w[8];
            y[c].get(u);
            if (p.post_w) {
                load8(p.post_w + i * 8, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = u[e] * r * w[e];
            }
            if (p.gate_cols == 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= g1;
            } else if (p.gate_cols) {
                g[c].get(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= gate_of<sizeof(Tr) == 4>(w[e]);
            }
            if (p.chan_scale) {
                load8(p.chan_scale + i * 8, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = fmaf(p.alpha, u[e], v[c][e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[c][e], v[c][e], ss);
        if (p.h_out) store8(static_cast<Tr*>(p.h_out) + t * p.H + i * 8, v[c]);
    }
    if (!p.x) return;
    r = 1.0f / sqrtf(sum(ss) / p.H + p.eps);
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const int i = i0 + c * step;
        if (!live || i >= chunks) continue;
        float w[8];
        load8(p.pre_w + i * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = v[c][e] * r * w[e];
        store8(static_cast<Ta*>(p.x) + t * p.H + i * 8, v[c]);
    }
}

// Rows that do not start on 16 bytes: one element a thread at a time, the row in shared memory between the passes.
template <typename Ta, typename Tr>
__global__ void __launch_bounds__(512) norm_residual_any_kernel(const NormParams p) {
    extern __shared__ float row[];
    __shared__ float sums[16];
    grid_dependency_wait();
    grid_launch_dependents();
    const long long t = blockIdx.x;
    const Ta* y = static_cast<const Ta*>(p.y) + t * p.ldy;
    const Ta* gate = static_cast<const Ta*>(p.gate) + t * p.ldg;
    const Tr* h = static_cast<const Tr*>(p.h) + t * p.H;
    float r = 1.f;
    if (p.post_w) {
        float ss = 0.f;
        for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
            const float v = ld_act(y + i);
            ss = fmaf(v, v, ss);
        }
        r = 1.0f / sqrtf(block_sum(ss, sums) / p.H + p.eps);
    }
    float ss = 0.f;
    for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
        float v = ld_act(h + i);
        if (p.y) {
            float u = ld_act(y + i) * r;
            if (p.post_w) u *= p.post_w[i];
            if (p.gate_cols) u *= gate_of<sizeof(Tr) == 4>(ld_act(gate + (p.gate_cols == 1 ? 0 : i)));
            if (p.chan_scale) u *= p.chan_scale[i];
            v = fmaf(p.alpha, u, v);
        }
        row[i] = v;
        ss = fmaf(v, v, ss);
        if (p.h_out) st_out(static_cast<Tr*>(p.h_out) + t * p.H + i, v);
    }
    if (!p.x) return;
    r = 1.0f / sqrtf(block_sum(ss, sums) / p.H + p.eps);
    for (int i = threadIdx.x; i < p.H; i += blockDim.x) st_out(static_cast<Ta*>(p.x) + t * p.H + i, row[i] * r * p.pre_w[i]);
}

template <typename Ta, typename Tr>
cudaError_t norm(const NormParams& p, cudaStream_t stream) {
    const int vec = 16 / static_cast<int>(sizeof(Ta));
    const bool wide = p.H % 8 == 0 && (!p.y || p.ldy % vec == 0) && (p.gate_cols < 2 || p.ldg % vec == 0);
    if (!wide) {
        const int threads = p.H >= 1024 ? 512 : p.H >= 256 ? 128 : 32;
        const int smem = p.H * 4;
        if (smem > 40 * 1024) {   // the limit is the same for every call: another thread's may come before the launch
            const cudaError_t e = cudaFuncSetAttribute(norm_residual_any_kernel<Ta, Tr>, cudaFuncAttributeMaxDynamicSharedMemorySize, GDN_NORM_MAX_H * 4);
            if (e != cudaSuccess) return e;
        }
        return launch_dependent(norm_residual_any_kernel<Ta, Tr>, dim3(p.T), dim3(threads), smem, stream, p);
    }
    const int chunks = p.H / 8;
    if (chunks <= 32) {
        int lanes = 1;
        while (lanes < chunks) lanes *= 2;
        const int rows = 128 / lanes;
        return launch_dependent(norm_residual_kernel<Ta, Tr, 1>, dim3((p.T + rows - 1) / rows), dim3(128), 0, stream, p, lanes);
    }
    const auto a_row = [&](void (*kernel)(NormParams, int), int n) {   // a CTA a row, n chunks a thread
        return launch_dependent(kernel, dim3(p.T), dim3((chunks + 32 * n - 1) / (32 * n) * 32), 0, stream, p, 0);
    };
    // One chunk a thread is quickest to its sums, two keep more loads in flight: one while the call's threads are at most half of
    // what the SMs hold (bf16, 2048 channels: 64 rows 2.7 us against 3.1, 304 rows 3.1 against 3.5, 608 rows 4.8 against 3.9,
    // 8192 rows 33 against 30).  A chunk of fp32 is two loads already: one up to 2048 channels (8192 rows of 1024: 25 us
    // against 28; of 4096: 104 against 89).
    const bool few = static_cast<long long>(p.T) * chunks <= 152 * 512 && chunks <= 512;
    if (few || (sizeof(Ta) == 4 && chunks <= 256)) return a_row(norm_residual_kernel<Ta, Tr, 1>, 1);
    if (chunks <= 1024) return a_row(norm_residual_kernel<Ta, Tr, 2>, 2);
    return a_row(norm_residual_kernel<Ta, Tr, 4>, 4);
}

}  // namespace

cudaError_t launch_norm_residual(const NormParams& p, int act_dtype, int res_dtype, cudaStream_t stream) {
    if (act_dtype == GDN_F32) return norm<float, float>(p, stream);
    return res_dtype == GDN_F32 ? norm<__nv_bfloat16, float>(p, stream) : norm<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace gdn
