// gdn_norm.cu -- the norms either side of a block with its gate and residual connection
// (include/gdn_norm.h, gdn_norm_residual).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_common.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += s[w];
    return t;
}

// One CTA per row, the row in shared memory between the passes.
template <typename Ta, typename Tr>
__global__ void __launch_bounds__(kThreads) norm_residual_kernel(const NormParams p) {
    extern __shared__ float row[];
    __shared__ float sums[kThreads / 32];
    const long long t = blockIdx.x;
    const Ta* y = static_cast<const Ta*>(p.y) + t * p.ldy;
    const Ta* gate = static_cast<const Ta*>(p.gate) + t * p.ldg;
    const Tr* h = static_cast<const Tr*>(p.h) + t * p.H;
    float r = 1.f;
    if (p.y && p.post_w) {
        float ss = 0.f;
        for (int i = threadIdx.x; i < p.H; i += kThreads) {
            const float v = ld_act(y + i);
            ss = fmaf(v, v, ss);
        }
        r = 1.0f / sqrtf(block_sum(ss, sums) / p.H + p.eps);
    }
    float ss = 0.f;
    for (int i = threadIdx.x; i < p.H; i += kThreads) {
        float v = ld_act(h + i);
        if (p.y) {
            float u = ld_act(y + i) * r;
            if (p.post_w) u *= p.post_w[i];
            if (p.gate_cols) u *= sigmoidf_(ld_act(gate + (p.gate_cols == 1 ? 0 : i)));
            if (p.chan_scale) u *= p.chan_scale[i];
            v = fmaf(p.alpha, u, v);
        }
        row[i] = v;
        ss = fmaf(v, v, ss);
        if (p.h_out) st_out(static_cast<Tr*>(p.h_out) + t * p.H + i, v);
    }
    if (!p.x) return;
    r = 1.0f / sqrtf(block_sum(ss, sums) / p.H + p.eps);
    for (int i = threadIdx.x; i < p.H; i += kThreads) st_out(static_cast<Ta*>(p.x) + t * p.H + i, row[i] * r * p.pre_w[i]);
}

template <typename Ta, typename Tr>
cudaError_t norm(const NormParams& p, cudaStream_t stream) {
    const int smem = p.H * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(norm_residual_kernel<Ta, Tr>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    norm_residual_kernel<Ta, Tr><<<p.T, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_residual(const NormParams& p, int act_dtype, int res_dtype, cudaStream_t stream) {
    if (act_dtype == GDN_F32) return norm<float, float>(p, stream);
    return res_dtype == GDN_F32 ? norm<__nv_bfloat16, float>(p, stream) : norm<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace gdn
