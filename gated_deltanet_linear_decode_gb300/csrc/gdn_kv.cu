// gdn_kv.cu -- the paged key-value cache of include/gdn_attn.h: page bookkeeping
// (extend, truncate) and the append of new tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_common.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 1024;

// Exclusive prefix sum of one value a thread over the block; *total = the sum of all.
// Every thread of the block calls it; `warp_sums` is shared, 33 entries.
__device__ __forceinline__ long long block_prefix(long long v, long long* warp_sums, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // the last use of warp_sums is over
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const long long s = lane < n_warps ? warp_sums[lane] : 0;
        long long t = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        if (lane < n_warps) warp_sums[lane] = t - s;
        if (lane == 31) warp_sums[32] = t;
    }
    __syncthreads();
    *total = warp_sums[32];
    return warp_sums[warp] + x - v;
}

// What one sequence asks for: rows (tokens) and pages; -1 rows where the request is refused by itself.
struct Ask {
    int len, held, rows, pages;
};

__device__ __forceinline__ Ask extend_ask(const KvExtendParams& p, int b) {
    Ask a;
    a.len = p.seq_len[b];
    a.held = p.n_pages[b];
    a.rows = p.n_new[b];
    a.pages = 0;
    const long long total = (static_cast<long long>(a.len) + a.rows + p.page_size - 1) / p.page_size;
    const int most = min(p.max_pages, p.num_pages);
    if (a.len < 0 || a.rows < 0 || a.held < 0 || a.held > most || total > most) {
        a.rows = -1;
    } else if (a.rows > 0 && total > a.held) {
        a.pages = static_cast<int>(total) - a.held;
    }
    return a;
}

// One CTA; a thread owns a run of consecutive sequences.  Prefix sums over the asked pages and rows
// decide what is served, a third one over the served rows gives cu_seqlens; then the rows.
__global__ void __launch_bounds__(kThreads) kv_extend_kernel(const KvExtendParams p) {
    __shared__ long long sums[33];
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    const int free_n = min(max(*p.free_count, 0), p.num_pages);
    long long pages = 0, rows = 0, total;
    for (int b = b0; b < b1; ++b) {
        const Ask a = extend_ask(p, b);
        pages += a.pages;
        rows += max(a.rows, 0);
    }
    const long long pages0 = block_prefix(pages, sums, &total), rows0 = block_prefix(rows, sums, &total);
    long long served_rows = 0, served_pages = 0;
    {
        long long pg = pages0, rw = rows0;
        for (int b = b0; b < b1; ++b) {
            const Ask a = extend_ask(p, b);
            if (a.rows >= 0 && (a.pages == 0 || pg + a.pages <= free_n) && (a.rows == 0 || rw + a.rows <= p.T)) {
                served_rows += a.rows;
                served_pages += a.pages;
            }
            pg += a.pages;
            rw += max(a.rows, 0);
        }
    }
    long long total_rows, total_pages;
    long long row = block_prefix(served_rows, sums, &total_rows);
    block_prefix(served_pages, sums, &total_pages);
    long long pg = pages0, rw = rows0;
    for (int b = b0; b < b1; ++b) {
        const Ask a = extend_ask(p, b);
        const bool ok = a.rows >= 0 && (a.pages == 0 || pg + a.pages <= free_n) && (a.rows == 0 || rw + a.rows <= p.T);
        const int n = ok ? a.rows : 0, got = ok ? a.pages : 0;
        int* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
        for (int j = 0; j < got; ++j) table[a.held + j] = p.free_list[free_n - 1 - static_cast<int>(pg) - j];
        for (int i = 0; i < n; ++i) {
            const int pos = a.len + i;
            p.positions[row + i] = pos;
            p.slot_map[row + i] = table[pos / p.page_size] * p.page_size + pos % p.page_size;
        }
        p.cu_seqlens[b] = static_cast<int>(row);
        p.seq_len_out[b] = a.len + n;
        p.n_pages_out[b] = a.held + got;
        if (!ok && p.status) atomicOr(p.status + b, kKvRefused);
        pg += a.pages;
        rw += max(a.rows, 0);
        row += n;
    }
    if (threadIdx.x == 0) {
        p.cu_seqlens[p.B] = static_cast<int>(total_rows);
        *p.free_count_out = free_n - static_cast<int>(total_pages);
    }
    for (int t = static_cast<int>(total_rows) + threadIdx.x; t < p.T; t += kThreads) {
        p.slot_map[t] = -1;
        p.positions[t] = 0;
    }
}

__device__ __forceinline__ bool truncate_ask(const KvTruncateParams& p, int b, int* len, int* held, int* keep) {
    *len = p.seq_len[b];
    *held = p.n_pages[b];
    const int n = p.new_len[b];
    if (n < 0 || n > *len || *held < 0 || *held > p.max_pages) {
        *keep = *held;
        return false;
    }
    *keep = static_cast<int>(min((static_cast<long long>(n) + p.page_size - 1) / p.page_size, static_cast<long long>(*held)));
    *len = n;
    return true;
}

// One CTA; a thread owns a run of consecutive sequences.  The page that is given back as number g of n
// goes to free_list[free_count + n - 1 - g].
__global__ void __launch_bounds__(kThreads) kv_truncate_kernel(const KvTruncateParams p) {
    __shared__ long long sums[33];
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    const int free_n = min(max(*p.free_count, 0), p.num_pages);
    long long back = 0, total, asked;
    int len, held, keep;
    for (int b = b0; b < b1; ++b) {
        truncate_ask(p, b, &len, &held, &keep);
        back += held - keep;
    }
    const long long before = block_prefix(back, sums, &asked);
    // a sequence whose pages would not fit the stack is refused, as are all after it that give any back
    long long g = before, served = 0;
    for (int b = b0; b < b1; ++b) {
        truncate_ask(p, b, &len, &held, &keep);
        if (g + held - keep <= p.num_pages - free_n) served += held - keep;
        g += held - keep;
    }
    block_prefix(served, sums, &total);
    g = before;
    for (int b = b0; b < b1; ++b) {
        const int old = p.seq_len[b];
        bool ok = truncate_ask(p, b, &len, &held, &keep);
        const int n = held - keep;
        const bool fits = n == 0 || g + n <= p.num_pages - free_n;
        const int* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
        if (ok && fits)
            for (int j = 0; j < n; ++j) p.free_list[free_n + total - 1 - g - j] = table[keep + j];
        ok = ok && fits;
        p.seq_len_out[b] = ok ? len : old;
        p.n_pages_out[b] = ok ? keep : held;
        if (!ok && p.status) atomicOr(p.status + b, kKvRefused);
        g += n;
    }
    if (threadIdx.x == 0) *p.free_count_out = free_n + static_cast<int>(total);
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + i);
        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint4 x;
    x.x = StateIO<__nv_bfloat16>::pack(v[0], v[1]);
    x.y = StateIO<__nv_bfloat16>::pack(v[2], v[3]);
    x.z = StateIO<__nv_bfloat16>::pack(v[4], v[5]);
    x.w = StateIO<__nv_bfloat16>::pack(v[6], v[7]);
    *reinterpret_cast<uint4*>(p) = x;
}

// D/8 lanes hold one head of one token, 8 consecutive channels each (a 16-byte access, two for
// fp32).  The norm's sum is a butterfly over those lanes; the two halves of a rotary pair are
// rope_dim/2 channels, i.e. rope_dim/16 lanes, apart, so the partner's channels come by shuffle.
template <typename Ta, int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendParams p) {
    constexpr int kLanes = D / 8;
    const int n_heads = p.Hq + 2 * p.Hkv;
    const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes;
    const int i = threadIdx.x % kLanes;   // lane of the head
    const bool live = item < static_cast<long long>(p.T) * n_heads;
    const long long t = live ? item / n_heads : 0;
    const int h = live ? static_cast<int>(item % n_heads) : 0;
    const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;   // q, k, v
    const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
    const Ta* src = kind == 0   ? static_cast<const Ta*>(p.q) + t * p.ldq
                    : kind == 1 ? static_cast<const Ta*>(p.k) + t * p.ldk
                                : static_cast<const Ta*>(p.v) + t * p.ldv;
    float u[8];
    load8(src + static_cast<size_t>(hh) * D + i * 8, u);
    const int slot = p.slot_map[t], pos = p.positions[t];
    const bool pos_ok = p.rope_dim == 0 || (pos >= 0 && pos < p.n_pos);
    const bool ok = pos_ok && slot < static_cast<long long>(p.cache.num_pages) * p.cache.page_size;
    const float* w = kind == 0 ? p.q_norm_w : p.k_norm_w;
    // every lane of the warp takes part in the shuffles, whatever its head is
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) ss = fmaf(u[c], u[c], ss);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (kind != 2 && w) {
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
        float wv[8];
        load8(w + i * 8, wv);
#pragma unroll
        for (int c = 0; c < 8; ++c) u[c] = u[c] * r * wv[c];
    }
    if (p.rope_dim > 0) {
        const int half = p.rope_dim / 16;   // lanes in one half of the pairs
        const bool lo = i < half, in = i < 2 * half;
        const int from = (threadIdx.x & 31) - i + (lo ? i + half : in ? i - half : i);
        float co[8], si[8];
        if (in && pos_ok && kind != 2) {
            const size_t at = static_cast<size_t>(pos) * (p.rope_dim / 2) + (lo ? i : i - half) * 8;
            load8(p.rope_cos + at, co);
            load8(p.rope_sin + at, si);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float o = __shfl_sync(0xffffffffu, u[c], from);
            if (in && pos_ok && kind != 2) u[c] = lo ? u[c] * co[c] - o * si[c] : u[c] * co[c] + o * si[c];
        }
    }
    if (!live) return;
    if (!ok) {
        if (p.status && h == 0 && i == 0) atomicOr(p.status, kKvBadIndex);
        return;
    }
    if (kind == 0) {
        store8(static_cast<Ta*>(p.q_out) + (t * p.Hq + hh) * D + i * 8, u);
    } else if (slot >= 0) {
        const long long at = static_cast<long long>(slot / p.cache.page_size) * p.cache.page_stride +
                             static_cast<long long>(slot % p.cache.page_size) * p.cache.token_stride +
                             static_cast<long long>(hh) * p.cache.head_stride + i * 8;
        store8(static_cast<Ta*>(kind == 1 ? p.cache.k : p.cache.v) + at, u);
    }
}

template <typename Ta, int D>
cudaError_t append(const KvAppendParams& p, cudaStream_t stream) {
    const long long threads = static_cast<long long>(p.T) * (p.Hq + 2 * p.Hkv) * (D / 8);
    const long long blocks = (threads + 255) / 256;
    kv_append_kernel<Ta, D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_extend(const KvExtendParams& p, cudaStream_t stream) {
    kv_extend_kernel<<<1, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_truncate(const KvTruncateParams& p, cudaStream_t stream) {
    kv_truncate_kernel<<<1, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendParams& p, int head_dim, int act_dtype, cudaStream_t stream) {
    if (act_dtype == GDN_BF16) {
        if (head_dim == 64) return append<__nv_bfloat16, 64>(p, stream);
        if (head_dim == 128) return append<__nv_bfloat16, 128>(p, stream);
        return append<__nv_bfloat16, 256>(p, stream);
    }
    if (head_dim == 64) return append<float, 64>(p, stream);
    if (head_dim == 128) return append<float, 128>(p, stream);
    return append<float, 256>(p, stream);
}

}  // namespace gdn
