// gdn_attn.cu -- attention of the last K tokens of each sequence over the paged key-value cache
// (include/gdn_attn.h, gdn_attn_decode).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_common.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 8;

// One CTA per (token row, query head).  Each warp walks every kWarps-th key with the channels spread
// over its lanes, keeping the running maximum m, sum l of e^(s-m) and the weighted sum of v; the warps'
// triples are joined in shared memory.
template <typename Ta, typename To, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_decode_kernel(const AttnParams p) {
    constexpr int kC = D / 32;
    __shared__ float ms[kWarps], ls[kWarps], os[kWarps][D];
    const int row = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, hk = h / p.G, b = row / p.K;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ps = p.cache.page_size;
    const long long cap = static_cast<long long>(p.max_pages) * ps;
    const int raw = p.seq_len[b];
    const int len = static_cast<int>(min(static_cast<long long>(max(raw, 0)), cap));
    bool bad = raw > cap;
    const int n = len - p.K + row % p.K + 1;
    const int* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
    float q[kC], o[kC], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        q[c] = ld_act(static_cast<const Ta*>(p.q) + row * p.ldq + h * D + c * 32 + lane);
        o[c] = 0.f;
    }
    for (int j = warp; j < n; j += kWarps) {
        const int page = table[j / ps];
        if (page < 0 || page >= p.cache.num_pages) {
            bad = true;
            continue;
        }
        const long long at = page * p.cache.page_stride + (j % ps) * p.cache.token_stride + hk * p.cache.head_stride;
        const Ta* k = static_cast<const Ta*>(p.cache.k) + at;
        const Ta* v = static_cast<const Ta*>(p.cache.v) + at;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) s = fmaf(q[c], ld_act(k + c * 32 + lane), s);
        s = warp_sum(s) * p.scale;
        if (s == -INFINITY) continue;   // no weight, and no maximum to be relative to
        const float m2 = fmaxf(m, s), f = expf(m - m2), e = expf(s - m2);
        l = l * f + e;
#pragma unroll
        for (int c = 0; c < kC; ++c) o[c] = o[c] * f + e * ld_act(v + c * 32 + lane);
        m = m2;
    }
    if (lane == 0) {
        ms[warp] = m;
        ls[warp] = l;
        if (bad && p.status) atomicOr(p.status + b, kKvBadIndex);
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) os[warp][c * 32 + lane] = o[c];
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
        float mm = -INFINITY, ll = 0.f, oo = 0.f;
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ms[w]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = ms[w] == -INFINITY ? 0.f : expf(ms[w] - mm);
            ll += f * ls[w];
            oo += f * os[w][i];
        }
        float y = ll > 0.f ? oo / ll : 0.f;
        if (p.gate) y *= sigmoidf_(ld_act(static_cast<const Ta*>(p.gate) + row * p.ldg + h * D + i));
        st_out(static_cast<To*>(p.out) + (static_cast<long long>(row) * p.Hq + h) * D + i, y);
    }
}

template <typename Ta, typename To, int D>
cudaError_t attn(const AttnParams& p, cudaStream_t stream) {
    attn_decode_kernel<Ta, To, D><<<p.B * p.K * p.Hq, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename Ta, typename To>
cudaError_t attn_d(const AttnParams& p, int head_dim, cudaStream_t stream) {
    if (head_dim == 64) return attn<Ta, To, 64>(p, stream);
    if (head_dim == 128) return attn<Ta, To, 128>(p, stream);
    return attn<Ta, To, 256>(p, stream);
}

}  // namespace

// Room for the counters of a split over the keys.
size_t attn_workspace_bytes(int, int, int, int, int, int) { return 4096; }

cudaError_t launch_attn_decode(const AttnParams& p, int head_dim, int act_dtype, int out_dtype, cudaStream_t stream) {
    if (act_dtype == GDN_BF16)
        return out_dtype == GDN_BF16 ? attn_d<__nv_bfloat16, __nv_bfloat16>(p, head_dim, stream)
                                     : attn_d<__nv_bfloat16, float>(p, head_dim, stream);
    return out_dtype == GDN_BF16 ? attn_d<float, __nv_bfloat16>(p, head_dim, stream)
                                 : attn_d<float, float>(p, head_dim, stream);
}

}  // namespace gdn
