// gdn_kv.cu -- the paged key-value cache of include/gdn_attn.h: page bookkeeping
// (extend, truncate) and the append of new tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

// Page bookkeeping.  Integer work on a few kilobytes to a few megabytes: bound by the latency of a launch and of a
// handful of dependent loads, and for prompts by how many threads write the rows.  Every CTA of one cluster
// scans all of the sequences for itself (prefix sums over what they ask for, kept in shared memory), then the
// rows and pages -- not the sequences -- are spread over all threads, each finding its sequence by bisection
// (a prompt of 60,000 tokens beside a hundred of one keeps every thread busy).  The inputs may be the
// outputs, so lengths and counts are written only after a cluster barrier behind the last read.
constexpr int kMaxThreads = 1024;
// Measured: the next token of 64 sequences 3.5 us, 65,536 prompt rows 9.1 us, 3 drafted tokens of 64 sequences of up to
// 16,384 taken back 5.7 us.  Eight CTAs cost a cluster's launch and pay with many rows or pages: 8,128 empty rows 4.6 us
// against 4.7 by one, 65,536 prompt rows 9.1 against 42; pages of 64 sequences of 4096 tokens 5.6 against 5.3, of 16,384
// tokens 5.7 against 7.8 (256 threads).  A smaller CTA's barriers are cheaper: 256 threads against 1024, extension of 64
// sequences 3.4 us against 3.9 (but 7.9 against 5.5 for 1024 sequences), truncation 5.7 against 6.3 (1024 sequences 9.0
// against 8.8).
constexpr int kManyRows = 4096, kManyPages = 4096;   // above: 8 CTAs

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

// What one sequence asks for; rows = -1 where the request is refused by itself.
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

__global__ void __launch_bounds__(kMaxThreads) kv_extend_kernel(const KvExtendParams p) {
    extern __shared__ int smem[];
    int* const row_s = smem;               // [B + 1] first row of each sequence
    int* const page_s = smem + p.B + 1;    // [B + 1] pages served before it
    __shared__ Pair sums[33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    const int free_n = min(max(*p.free_count, 0), p.num_pages);
    Pair ask{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const Ask a = extend_ask(p, b);
        ask.rows += max(a.rows, 0);
        ask.pages += a.pages;
    }
    const Pair before = block_prefix(ask, sums, &total);
    // Where a request that would fit by itself is refused for want of pages or rows, so is every later one that
    // asks for any: what is served is a prefix of the asked pages, and of the asked rows.
    auto serve = [&](auto&& f) {
        Pair at = before;
        for (int b = b0; b < b1; ++b) {
            const Ask a = extend_ask(p, b);
            const bool ok = a.rows >= 0 && (a.pages == 0 || at.pages + a.pages <= free_n) &&
                            (a.rows == 0 || at.rows + a.rows <= p.T);
            f(b, a, ok);
            at.rows += max(a.rows, 0);
            at.pages += a.pages;
        }
    };
    Pair at = before;
    if (total.rows > p.T || total.pages > free_n) {   // some are refused: sums over the others
        Pair got{0, 0};
        serve([&](int, const Ask& a, bool ok) {
            got.rows += ok ? a.rows : 0;
            got.pages += ok ? a.pages : 0;
        });
        at = block_prefix(got, sums, &total);
    }
    const bool first_cta = cluster_ctarank() == 0;
    serve([&](int b, const Ask& a, bool ok) {
        row_s[b] = static_cast<int>(at.rows);
        page_s[b] = static_cast<int>(at.pages);
        at.rows += ok ? a.rows : 0;
        at.pages += ok ? a.pages : 0;
        if (!ok && first_cta && p.status) atomicOr(p.status + b, kKvRefused);
    });
    if (threadIdx.x == 0) {
        row_s[p.B] = static_cast<int>(total.rows);
        page_s[p.B] = static_cast<int>(total.pages);
    }
    __syncthreads();
    const int rows = row_s[p.B], pages = page_s[p.B];
    const int me = cluster_ctarank() * blockDim.x + threadIdx.x, all = cluster_ctas() * blockDim.x;
    for (int g = me; g < pages; g += all) {
        const int b = find(page_s, p.B, g);
        p.block_table[static_cast<size_t>(b) * p.max_pages + p.n_pages[b] + g - page_s[b]] = p.free_list[free_n - 1 - g];
    }
    for (int t = me; t < p.T; t += all) {
        int slot = -1, pos = 0;
        if (t < rows) {
            const int b = find(row_s, p.B, t);
            pos = p.seq_len[b] + t - row_s[b];
            const int i = pos / p.page_size, held = p.n_pages[b];
            // a page of this call is read where it comes from, not where another thread is writing it
            const int page = i < held ? p.block_table[static_cast<size_t>(b) * p.max_pages + i]
                                      : p.free_list[free_n - 1 - page_s[b] - (i - held)];
            if (page >= 0 && page < p.num_pages) slot = page * p.page_size + (pos - i * p.page_size);
            else if (p.status) atomicOr(p.status + b, kKvBadIndex);
        }
        p.slot_map[t] = slot;
        p.positions[t] = pos;
    }
    cluster_sync_all();
    if (!first_cta) return;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        p.cu_seqlens[b] = row_s[b];
        p.seq_len_out[b] = p.seq_len[b] + row_s[b + 1] - row_s[b];
        p.n_pages_out[b] = p.n_pages[b] + page_s[b + 1] - page_s[b];
    }
    if (threadIdx.x == 0) {
        p.cu_seqlens[p.B] = rows;
        *p.free_count_out = free_n - pages;
    }
}

// What a sequence gives back: pages keep..held-1, or nothing where it is refused by itself (ok false).
struct Back {
    int len, held, keep;
    bool ok;
};

__device__ __forceinline__ Back truncate_ask(const KvTruncateParams& p, int b) {
    Back r;
    r.len = p.seq_len[b];
    r.held = p.n_pages[b];
    r.keep = r.held;
    const int n = p.new_len[b];
    r.ok = n >= 0 && n <= r.len && r.held >= 0 && r.held <= p.max_pages;
    if (r.ok) {
        r.len = n;
        r.keep = static_cast<int>(min((static_cast<long long>(n) + p.page_size - 1) / p.page_size, static_cast<long long>(r.held)));
    }
    return r;
}

// The page that is given back as number g of n goes to free_list[free_count + n - 1 - g].
__global__ void __launch_bounds__(kMaxThreads) kv_truncate_kernel(const KvTruncateParams p) {
    extern __shared__ int smem[];
    int* const page_s = smem;   // [B + 1] pages given back before each sequence
    __shared__ Pair sums[33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    const int free_n = min(max(*p.free_count, 0), p.num_pages), room = p.num_pages - free_n;
    Pair ask{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const Back r = truncate_ask(p, b);
        ask.pages += r.held - r.keep;
    }
    Pair at = block_prefix(ask, sums, &total);
    const long long before = at.pages;
    // a sequence whose pages would not fit the stack is refused, as are all after it that give any back
    if (total.pages > room) {
        Pair got{0, 0};
        long long g = before;
        for (int b = b0; b < b1; ++b) {
            const Back r = truncate_ask(p, b);
            const int n = r.held - r.keep;
            if (g + n <= room) got.pages += n;
            g += n;
        }
        at = block_prefix(got, sums, &total);
    }
    const bool first_cta = cluster_ctarank() == 0;
    long long g = before;
    for (int b = b0; b < b1; ++b) {
        const Back r = truncate_ask(p, b);
        const int n = r.held - r.keep;
        const bool fits = n == 0 || g + n <= room;
        page_s[b] = static_cast<int>(at.pages);
        if (fits) at.pages += n;
        if (first_cta && p.status && !(r.ok && fits)) atomicOr(p.status + b, kKvRefused);
        g += n;
    }
    if (threadIdx.x == 0) page_s[p.B] = static_cast<int>(total.pages);
    __syncthreads();
    const int pages = page_s[p.B];
    // a warp takes 128 consecutive pages at a time: one bisection serves those of one sequence
    const int lane = threadIdx.x & 31;
    const int me = (cluster_ctarank() * blockDim.x + threadIdx.x) >> 5, all = (cluster_ctas() * blockDim.x) >> 5;
    for (int c = me * 128; c < pages; c += all * 128) {
        const int bc = find(page_s, p.B, c), end = page_s[bc + 1];
        const Back rc = truncate_ask(p, bc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int gg = c + i * 32 + lane;
            if (gg < pages) {
                int b = bc, keep = rc.keep;
                if (gg >= end) {
                    b = find(page_s, p.B, gg);
                    keep = truncate_ask(p, b).keep;
                }
                const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + keep + gg - page_s[b]];
                if ((page < 0 || page >= p.num_pages) && p.status) atomicOr(p.status + b, kKvBadIndex);
                p.free_list[free_n + pages - 1 - gg] = page;
            }
        }
    }
    cluster_sync_all();
    if (!first_cta) return;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const Back r = truncate_ask(p, b);
        const int n = page_s[b + 1] - page_s[b];
        const bool done = r.ok && n == r.held - r.keep;
        const int old = p.seq_len[b];
        p.seq_len_out[b] = done ? r.len : old;
        p.n_pages_out[b] = r.held - n;
    }
    if (threadIdx.x == 0) *p.free_count_out = free_n + pages;
}

// One cluster of `ctas` CTAs with room for `arrays` arrays of B + 1 words.  The kernel's limit is set to what the most sequences
// need, the same by every call: another thread's call may come between it and the launch.
template <typename P>
cudaError_t launch_cluster(void (*kernel)(P), const P& p, int ctas, int threads, size_t arrays, cudaStream_t stream) {
    const size_t smem = arrays * (static_cast<size_t>(p.B) + 1) * 4;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(arrays * (kKvMaxSeq + 1) * 4));
        if (e != cudaSuccess) return e;
    }
    return launch_dependent_cluster(kernel, ctas, dim3(ctas), dim3(threads), smem, stream, p);
}

// The append.  Elementwise over (2 H_q + 4 H_kv) head_dim elements a token, read and written once: bound by the
// memory for prompts -- where the instructions a head takes and the registers that hold back other warps
// matter -- and by latency for a decode batch.  A warp takes one job: up to kPass head sets of one token, all q
// or all k or all v, so that where they come from, where they go and what is done to them is settled once; all
// loads first.  D/8 lanes hold one head, 8 consecutive channels each (a 16-byte access, two for fp32).  The norm's sum is
// a butterfly over the lanes of a head.  The two halves of a rotary pair are rope_dim/2 channels, i.e. rope_dim/16
// lanes, apart: the partner's channels come by shuffle, as they lie in memory, and norm weight and rotation are
// one pair of factors a channel, u' = r (u A + partner B), the same for all heads of the job.
// Small CTAs, so that a finished warp's place is soon another's, and the registers of four head sets without spills.
// Measured, heads of 256, 64 channels rotated: 8192 tokens of 24/4 heads (271 MB) 50.1 us, 5.4 TB/s (fp32 83.8, 6.5 TB/s); 64 tokens of 16/2 heads
// 2.4 us.  8192 tokens by CTAs of 8 warps, four an SM 54.7 us; 4 warps, eight 52.5, nine 50.1, ten 49.7 (with spills; heads
// of 64 39 us against 34); 2 warps, sixteen 52.1, eighteen 49.6; 1 warp 66.  By CTAs of 8 warps two and eight head sets a
// job both 64 us.
constexpr unsigned kAppendWarps = 2;
constexpr int kPass = 4;

template <typename Ta, int D>
__global__ void __launch_bounds__(32 * kAppendWarps, sizeof(Ta) == 2 ? 18 : 12) kv_append_kernel(const KvAppendParams p, const int q_jobs, const int kv_jobs) {
    constexpr int kLanes = D / 8, kSet = 32 / kLanes;   // lanes of a head, heads of a set
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, i = lane % kLanes, sub = lane / kLanes;
    const int jobs = q_jobs + 2 * kv_jobs;
    const unsigned id = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int t = static_cast<int>(id / jobs);
    int job = static_cast<int>(id - static_cast<unsigned>(t) * jobs);
    if (t >= p.T) return;   // a whole warp
    const int slot = p.slot_map[t], pos = p.positions[t];
    const int kind = job < q_jobs ? 0 : job < q_jobs + kv_jobs ? 1 : 2;   // q, k, v
    if (kind) job -= kind == 1 ? q_jobs : q_jobs + kv_jobs;
    const int heads = kind == 0 ? p.Hq : p.Hkv, h0 = job * kPass * kSet + sub;
    const Ta* const src = (kind == 0   ? static_cast<const Ta*>(p.q) + t * p.ldq
                           : kind == 1 ? static_cast<const Ta*>(p.k) + t * p.ldk
                                       : static_cast<const Ta*>(p.v) + t * p.ldv) +
                          h0 * D + i * 8;
    Raw8<Ta> raw[kPass];
#pragma unroll
    for (int s = 0; s < kPass; ++s)
        if (h0 + s * kSet < heads) raw[s].load(src + s * kSet * D);
    if ((p.rope_dim != 0 && (pos < 0 || pos >= p.n_pos)) || slot >= p.cache.num_pages * p.cache.page_size) {
        if (p.status && lane == 0 && id == static_cast<unsigned>(t) * jobs) atomicOr(p.status, kKvBadIndex);
        return;
    }
    Ta* dst;
    long long step = D;   // elements from head to head
    if (kind == 0) {
        dst = static_cast<Ta*>(p.q_out) + (static_cast<long long>(t) * p.Hq + h0) * D;
    } else {
        if (slot < 0) return;
        const int page = slot / p.cache.page_size;
        step = p.cache.head_stride;
        dst = static_cast<Ta*>(kind == 1 ? p.cache.k : p.cache.v) + page * p.cache.page_stride +
              (slot - page * p.cache.page_size) * p.cache.token_stride + h0 * step;
    }
    dst += i * 8;
    step *= kSet;
    if (kind == 2) {   // copies, bit for bit
#pragma unroll
        for (int s = 0; s < kPass; ++s)
            if (h0 + s * kSet < heads) raw[s].store(dst + s * step);
        return;
    }
    const float* const w = kind == 0 ? p.q_norm_w : p.k_norm_w;
    const int half = p.rope_dim / 16;   // lanes in one half of the pairs
    int from = lane;
    float A[8], B[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        A[c] = 1.f;
        B[c] = 0.f;
    }
    if (w) load8(w + i * 8, A);
    if (i < 2 * half) {
        const int d = i < half ? half : -half;   // to the partner's lane
        from += d;
        const size_t tab = static_cast<size_t>(pos) * (p.rope_dim / 2) + (d > 0 ? i : i - half) * 8;
        float x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) B[c] = 1.f;
        if (w) load8(w + (i + d) * 8, B);
        load8(p.rope_cos + tab, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) A[c] *= x[c];
        load8(p.rope_sin + tab, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) B[c] *= d > 0 ? -x[c] : x[c];
    } else if (half > 0) {
        // Not rotated: the partner is the channel itself, and halves of the weight leave an infinite one what it is, where A = w and
        // B = 0 would make it NaN.  (Zeros for the partner instead: heads of 64 35.5 us against 33.9.)
#pragma unroll
        for (int c = 0; c < 8; ++c) A[c] = B[c] = 0.5f * A[c];
    }
#pragma unroll
    for (int s = 0; s < kPass; ++s) {
        if (h0 - sub + s * kSet >= heads) break;   // the same for the whole warp; its lanes shuffle together
        float u[8], r = 1.f;
        raw[s].get(u);
        if (w) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 8; c += 2) ss = fma2(make_float2(u[c], u[c + 1]), make_float2(u[c], u[c + 1]), ss);
            r = ss.x + ss.y;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
            r = rsqrtf(r * (1.0f / D) + p.eps);   // within 2 units in the last place
        }
        if (half > 0) {
            float x[8];
            raw[s].shuffled(from).get(x);
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                const float2 y = mul2(make_float2(r, r), fma2(make_float2(x[c], x[c + 1]), make_float2(B[c], B[c + 1]),
                                                              mul2(make_float2(u[c], u[c + 1]), make_float2(A[c], A[c + 1]))));
                u[c] = y.x;
                u[c + 1] = y.y;
            }
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) u[c] *= r * A[c];
        }
        if (h0 + s * kSet < heads) store8(dst + s * step, u);
    }
}

template <typename Ta, int D>
cudaError_t append(const KvAppendParams& p, cudaStream_t stream) {
    constexpr int kHeads = kPass * 256 / D;   // of a job
    const int q_jobs = (p.Hq + kHeads - 1) / kHeads, kv_jobs = (p.Hkv + kHeads - 1) / kHeads;
    const long long blocks = (static_cast<long long>(p.T) * (q_jobs + 2 * kv_jobs) + kAppendWarps - 1) / kAppendWarps;
    if (blocks > (1ll << 31) / kAppendWarps - 1) return cudaErrorInvalidConfiguration;   // a warp's number has 31 bits
    return launch_dependent(kv_append_kernel<Ta, D>, dim3(static_cast<unsigned>(blocks)), dim3(32 * kAppendWarps), 0, stream, p, q_jobs, kv_jobs);
}

}  // namespace

cudaError_t launch_kv_extend(const KvExtendParams& p, cudaStream_t stream) {
    const int ctas = p.T > kManyRows ? 8 : 1;
    const int threads = p.T <= 256 && p.B <= 256 ? 256 : kMaxThreads;
    return launch_cluster(kv_extend_kernel, p, ctas, threads, 2, stream);
}

cudaError_t launch_kv_truncate(const KvTruncateParams& p, cudaStream_t stream) {
    const int ctas = p.num_pages > kManyPages ? 8 : 1;
    const int threads = p.B <= 512 ? 256 : kMaxThreads;
    return launch_cluster(kv_truncate_kernel, p, ctas, threads, 1, stream);
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
