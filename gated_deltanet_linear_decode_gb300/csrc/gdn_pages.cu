// gdn_pages.cu -- pages that sequences share (include/gdn_pages.h): fork, release, compaction, and the copies of pages.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>

#include "gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_books.cuh"
#include "gdn_cluster_size.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {

namespace {

// The bookkeeping: whole numbers, a few words a sequence and a page entry.  As in gdn_kv.cu one cluster of CTAs, each of which
// scans all sequences for itself into prefix sums in shared memory; then the page entries -- not the sequences -- are spread
// over the cluster's threads.  Inputs are outputs: what the scan reads is written behind a cluster barrier.
constexpr int kBookThreads = 1024;
// CTAs by the entries of the tables (or pages) that there may be.  16 forks of 256 pages and their release (4,600 entries) by 1, 8, 16
// CTAs 15.2, 17.3, 18.6 us, 8 of 1,024 (9,400) 18.1, 18.2, 19.1, compaction of 16 sequences of up to 1,024 (16,600) 32, 18, 20, 63
// forks of 1,024 pages (66,000) 25 by 8 and 24 by 16, 400 forks on prefixes of up to 2,048 (890,000) 587, 86, 52.
int ctas_for(size_t entries) { return entries > 32768 ? 16 : entries > 8192 ? 8 : 1; }
// Pages whose counts are summed in shared memory before they go to page_refs, one addition a page and CTA.  Additions to a few
// lines of memory take their turn, some 20 ns each whoever makes them: 63 forks of 1024 pages of a cache of 1100 took 48 us
// by 8 and by 64 CTAs and their release 160, with counts in shared memory 12 and 21.  In larger caches the pages lie in more
// lines.
constexpr int kCountPages = 24 * 1024;
constexpr size_t kMostWords = 56 * 1024;   // of dynamic shared memory

__device__ __forceinline__ bool page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }
// Words that other CTAs of the cluster change: past L1, which keeps what it has read.
__device__ __forceinline__ int ld_l2(const int* p) { return __ldcg(p); }
__device__ __forceinline__ int ld_dsmem_int(const int* local, uint32_t rank) {
    return __float_as_int(ld_dsmem_f32(reinterpret_cast<const float*>(local), rank));
}
__device__ __forceinline__ int cluster_thread() { return static_cast<int>(cluster_ctarank() * blockDim.x + threadIdx.x); }
__device__ __forceinline__ int cluster_threads() { return static_cast<int>(cluster_ctas() * blockDim.x); }

// ---------------------------------------------------------------- fork
struct ForkAsk {
    int dst, full, part;
    bool ok;   // by itself
};

__device__ __forceinline__ ForkAsk fork_ask(const KvForkParams& p, int i) {
    ForkAsk a{-1, 0, 0, false};
    const int s = p.src[i], d = p.dst[i], n = p.len[i];
    if (s < 0 || s >= p.B || d < 0 || d >= p.B || s == d || n < 0 || n > p.seq_len[s]) return a;
    const int held = p.n_pages[s];
    a.dst = d;
    a.full = n / p.page_size;
    a.part = n - a.full * p.page_size > 0;
    a.ok = held <= p.max_pages && a.full + a.part <= held && p.seq_len[d] == 0 && p.n_pages[d] == 0;
    return a;
}

constexpr int kForkRun = 128;   // entries that a warp takes at a time

__global__ void __launch_bounds__(kBookThreads, 1) kv_fork_kernel(const KvForkParams p) {
    extern __shared__ int smem[];
    int* const first_s = smem;             // [B] the fork that a sequence is the dst of
    int* const run_s = first_s + p.B;      // [N + 1] runs of entries before each fork
    int* const page_s = run_s + p.N + 1;   // [N + 1] pages served before it
    int* const count_s = page_s + p.N + 1;   // [num_pages] if there are few
    __shared__ Pair sums[33];
    grid_dependency_wait();
    grid_launch_dependents();
    const bool counted = p.room > 0;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) first_s[b] = INT_MAX;
    if (counted)
        for (int g = threadIdx.x; g < p.num_pages; g += blockDim.x) count_s[g] = 0;
    __syncthreads();
    const int per = (p.N + blockDim.x - 1) / blockDim.x;
    const int i0 = min(p.N, static_cast<int>(threadIdx.x) * per), i1 = min(p.N, i0 + per);
    for (int i = i0; i < i1; ++i) {   // each thread's own forks, so far: runs (-1: refused by itself), pages
        const ForkAsk a = fork_ask(p, i);
        run_s[i] = a.ok ? (a.full + kForkRun - 1) / kForkRun : -1;
        page_s[i] = a.part;
        if (a.ok) atomicMin(first_s + a.dst, i);
    }
    __syncthreads();
    const int free_n = min(max(*p.free_count, 0), p.num_pages);
    const bool first_cta = cluster_ctarank() == 0;
    Pair ask{0, 0}, got{0, 0}, total;
    for (int i = i0; i < i1; ++i) {
        if (run_s[i] >= 0 && first_s[p.dst[i]] != i) run_s[i] = -1;   // another has its dst
        ask.pages += run_s[i] >= 0 ? page_s[i] : 0;
    }
    // what is served of the asked pages is a prefix of them
    long long used = block_prefix(ask, sums, &total).pages;
    for (int i = i0; i < i1; ++i) {
        used += run_s[i] >= 0 ? page_s[i] : 0;
        if (run_s[i] >= 0 && page_s[i] > 0 && used > free_n) {
            run_s[i] = -1;
            first_s[p.dst[i]] = INT_MAX;   // (only the first of a dst writes its word, and every other has been refused)
        }
        if (run_s[i] < 0) {
            run_s[i] = page_s[i] = 0;
            if (first_cta && p.status) atomicOr(p.status + i, kKvRefused);
        }
        got.rows += run_s[i];
        got.pages += page_s[i];
    }
    Pair at = block_prefix(got, sums, &total);
    for (int i = i0; i < i1; ++i) {
        const int n = run_s[i], k = page_s[i];
        run_s[i] = static_cast<int>(at.rows);
        page_s[i] = static_cast<int>(at.pages);
        at.rows += n;
        at.pages += k;
    }
    if (threadIdx.x == 0) {
        run_s[p.N] = static_cast<int>(total.rows);
        page_s[p.N] = static_cast<int>(total.pages);
    }
    __syncthreads();
    auto served = [&](int i) {
        const int d = p.dst[i];
        return d >= 0 && d < p.B && first_s[d] == i;
    };
    const int runs = run_s[p.N], lane = threadIdx.x & 31, ctas = static_cast<int>(cluster_ctas());
    // a CTA has consecutive runs: of forks of one sequence, as they often are, the same pages
    const int each = (runs + ctas - 1) / ctas, c0 = static_cast<int>(cluster_ctarank()) * each, c1 = min(runs, c0 + each);
    for (int c = c0 + static_cast<int>(threadIdx.x >> 5); c < c1; c += static_cast<int>(blockDim.x >> 5)) {
        const int i = find(run_s, p.N, c);
        const int full = p.len[i] / p.page_size, col0 = (c - run_s[i]) * kForkRun;
        const int* const from = p.block_table + static_cast<size_t>(p.src[i]) * p.max_pages;
        int* const to = p.block_table + static_cast<size_t>(p.dst[i]) * p.max_pages;
        int page[kForkRun / 32];
#pragma unroll
        for (int k = 0; k < kForkRun / 32; ++k) {
            const int col = col0 + k * 32 + lane;
            page[k] = col < full ? from[col] : 0;
        }
#pragma unroll
        for (int k = 0; k < kForkRun / 32; ++k) {
            const int col = col0 + k * 32 + lane;
            if (col >= full) continue;
            to[col] = page[k];
            if (page_ok(page[k], p.num_pages)) atomicAdd((counted ? count_s : p.page_refs) + page[k], 1);
            else if (p.status) atomicOr(p.status + i, kKvBadIndex);
        }
    }
    if (counted) {
        __syncthreads();
        for (int g = threadIdx.x; g < p.num_pages; g += blockDim.x)
            if (count_s[g] > 0) atomicAdd(p.page_refs + g, count_s[g]);
    }
    for (int i = cluster_thread(); i < p.N; i += cluster_threads()) {
        int a = -1, b = -1;
        if (served(i) && page_s[i + 1] > page_s[i]) {
            const int full = p.len[i] / p.page_size;
            a = p.block_table[static_cast<size_t>(p.src[i]) * p.max_pages + full];
            b = p.free_list[free_n - 1 - page_s[i]];
            p.block_table[static_cast<size_t>(p.dst[i]) * p.max_pages + full] = b;
            if (!page_ok(a, p.num_pages) || !page_ok(b, p.num_pages)) {
                a = b = -1;
                if (p.status) atomicOr(p.status + i, kKvBadIndex);
            }
        }
        p.copy_src[i] = a;
        p.copy_dst[i] = b;
    }
    cluster_sync_all();   // all have read the lengths
    if (!first_cta) return;
    for (int i = threadIdx.x; i < p.N; i += blockDim.x) {
        if (!served(i)) continue;
        const int n = p.len[i], d = p.dst[i];
        p.seq_len[d] = n;
        p.n_pages[d] = n / p.page_size + (page_s[i + 1] - page_s[i]);
    }
    if (threadIdx.x == 0) *p.free_count = free_n - page_s[p.N];
}

// ---------------------------------------------------------------- release
// A sequence gives up its entries from..held-1 (the first of them the kept one that a copy replaces, if `copy`).
struct ReleaseAsk {
    int from, held, stay;
    bool ok, copy;
};

__device__ __forceinline__ ReleaseAsk release_ask(const KvReleaseParams& p, int b) {
    ReleaseAsk r{0, p.n_pages[b], 0, false, false};
    const int n = p.new_len[b];
    r.stay = r.from = r.held;
    r.ok = n >= 0 && n <= p.seq_len[b] && r.held >= 0 && r.held <= p.max_pages;
    if (!r.ok) return r;
    const int need = n / p.page_size + (n % p.page_size > 0);
    r.stay = r.from = min(need, r.held);
    if (n % p.page_size > 0 && need <= r.held) {
        const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + need - 1];
        r.copy = page_ok(page, p.num_pages) && p.page_refs[page] > 0;
        r.from -= r.copy;
    }
    return r;
}

// Which of a page's holders gives it back?  Phase by phase, a cluster barrier between them: every entry given up takes one from
// its page's count; where that is below zero, the entries put in their numbers (INT_MIN + number, the least stays); the
// entry that finds its own there is the one.  So the count itself is all the scratch, and the result the same in any order.
constexpr int kHold = 6;              // blocks of a warp in registers
constexpr int kNone = INT_MIN;        // (pages below zero are taken as -1)
__global__ void __launch_bounds__(kBookThreads, 1) kv_release_kernel(const KvReleaseParams p) {
    extern __shared__ int smem[];
    int* const drop_s = smem;               // [B + 1] blocks of up to 128 entries given up before each sequence
    int* const copy_s = drop_s + p.B + 1;   // [B + 1] copies before it
    int* const from_s = copy_s + p.B + 1;   // [B] its first entry given up; -1 - that where it is refused
    int* const count_s = from_s + p.B + 1;  // [num_pages] if there are few
    __shared__ Pair sums[33];
    __shared__ int mine_s;
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    const int free_n = min(max(*p.free_count, 0), p.num_pages);
    Pair ask{0, 0}, got{0, 0}, total;
    for (int b = b0; b < b1; ++b) {   // each thread's own sequences, so far
        const ReleaseAsk r = release_ask(p, b);
        drop_s[b] = (r.held - r.from + 127) / 128;
        copy_s[b] = r.copy;
        from_s[b] = r.ok ? r.from : -1 - r.from;
        ask.pages += r.copy;
    }
    const Pair asked = block_prefix(ask, sums, &total);
    const bool first_cta = cluster_ctarank() == 0;
    long long used = asked.pages;
    for (int b = b0; b < b1; ++b) {
        used += copy_s[b];
        if (from_s[b] >= 0 && copy_s[b] && used > free_n) from_s[b] = -1 - from_s[b];   // the pages are out
        if (from_s[b] < 0) {
            drop_s[b] = copy_s[b] = 0;
            if (first_cta && p.status) atomicOr(p.status + b, kKvRefused);
        }
        got.rows += drop_s[b];
        got.pages += copy_s[b];
    }
    Pair at = block_prefix(got, sums, &total);
    for (int b = b0; b < b1; ++b) {
        const int n = drop_s[b], k = copy_s[b];
        drop_s[b] = static_cast<int>(at.rows);
        copy_s[b] = static_cast<int>(at.pages);
        at.rows += n;
        at.pages += k;
    }
    if (threadIdx.x == 0) {
        drop_s[p.B] = static_cast<int>(total.rows);
        copy_s[p.B] = static_cast<int>(total.pages);
    }
    cluster_sync_all();   // all have read the counts
    const int blocks = drop_s[p.B], copies = copy_s[p.B], all = cluster_threads(), lane = threadIdx.x & 31;
    // this warp's blocks: consecutive ones, of which the first kHold lie in registers, their loads issued together
    const int each = static_cast<int>((static_cast<long long>(blocks) * 32 + all - 1) / all);
    const long long k0 = static_cast<long long>(cluster_thread() >> 5) * each;
    const int k1 = static_cast<int>(min(static_cast<long long>(blocks), k0 + each));
    const bool counted = p.room > 0;
    auto sequence_of = [&](int k, int b) {   // from b, one that is not behind it, on
        if (k >= drop_s[b + 1] && k >= drop_s[++b + 1]) b = find(drop_s, p.B, k);
        return b;
    };
    int held[kHold][4];
    {
        int b = 0, n[kHold];
        const int* e[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            n[i] = 0;
            e[i] = nullptr;
            if (k0 + i < k1) {
                const int k = static_cast<int>(k0) + i;
                b = i == 0 ? find(drop_s, p.B, k) : sequence_of(k, b);
                const int col0 = (k - drop_s[b]) * 128 + lane;
                n[i] = p.n_pages[b] - from_s[b] - col0;
                e[i] = p.block_table + static_cast<size_t>(b) * p.max_pages + from_s[b] + col0;
            }
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) held[i][j] = 32 * j < n[i] ? max(e[i][32 * j], -1) : kNone;
    }
    // f(number, page) of the entries in order: the page, or kNone where there is none.  By whole warps; what is kNone in a register
    // stays so, and f may make it so.
    auto entries = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            if (k0 + i >= k1) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) f((static_cast<int>(k0) + i) * 128 + 32 * j + lane, held[i][j]);
        }
        int b = k0 + kHold < k1 ? find(drop_s, p.B, static_cast<int>(k0) + kHold) : 0;
        for (long long k = k0 + kHold; k < k1; ++k) {
            b = sequence_of(static_cast<int>(k), b);
            const int col0 = (static_cast<int>(k) - drop_s[b]) * 128 + lane, n = p.n_pages[b] - from_s[b] - col0;
            const int* const e = p.block_table + static_cast<size_t>(b) * p.max_pages + from_s[b] + col0;
            int page[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) page[j] = 32 * j < n ? max(e[32 * j], -1) : kNone;
#pragma unroll
            for (int j = 0; j < 4; ++j) f(static_cast<int>(k) * 128 + 32 * j + lane, page[j]);
        }
    };
    auto in_cache = [&](int page) { return page_ok(page, p.num_pages); };
    if (counted) {
        for (int g = threadIdx.x; g < p.num_pages; g += blockDim.x) count_s[g] = 0;
        __syncthreads();
    }
    entries([&](int at, int& page) {
        if (in_cache(page)) atomicAdd((counted ? count_s : p.page_refs) + page, counted ? 1 : -1);
        else if (page != kNone && p.status) atomicOr(p.status + find(drop_s, p.B, at >> 7), kKvBadIndex);
    });
    if (counted) {
        __syncthreads();
        for (int g = threadIdx.x; g < p.num_pages; g += blockDim.x)
            if (count_s[g] > 0) atomicSub(p.page_refs + g, count_s[g]);
    }
    for (int b = cluster_thread(); b < p.B; b += all) {
        int src = -1, dst = -1;
        if (copy_s[b + 1] > copy_s[b]) {
            src = p.block_table[static_cast<size_t>(b) * p.max_pages + from_s[b]];
            dst = p.free_list[free_n - 1 - copy_s[b]];
        }
        p.copy_src[b] = src;
        p.copy_dst[b] = dst;
    }
    cluster_sync_all();
    if (counted) {   // the counts as they are now
        for (int g = threadIdx.x; g < p.num_pages; g += blockDim.x) count_s[g] = ld_l2(p.page_refs + g);
        cluster_sync_all();
    }
    auto none_holds = [&](int page) { return in_cache(page) && (counted ? count_s[page] : ld_l2(p.page_refs + page)) < 0; };
    entries([&](int at, int& page) {
        if (none_holds(page)) atomicMin(p.page_refs + page, INT_MIN + at);
        else page = kNone;
    });
    cluster_sync_all();
    auto ours = [&](int page, int at) { return none_holds(page) && ld_l2(p.page_refs + page) == INT_MIN + at; };
    int back = 0;
    entries([&](int at, int& page) {
        const bool mine = ours(page, at);
        if (!mine) page = kNone;
        back += __popc(__ballot_sync(0xffffffffu, mine));
    });
    const Pair before = block_prefix(Pair{0, lane == 0 ? back : 0}, sums, &total);
    if (threadIdx.x == 0) mine_s = static_cast<int>(total.pages);
    cluster_sync_all();
    int rank = static_cast<int>(__shfl_sync(0xffffffffu, before.pages, 0)), pushed = 0;
    for (uint32_t c = 0; c < cluster_ctas(); ++c) {
        const int n = ld_dsmem_int(&mine_s, c);
        if (c < cluster_ctarank()) rank += n;
        pushed += n;
    }
    const int base = free_n - copies;   // the stack without the pages for copies
    entries([&](int at, int& page) {
        const bool mine = ours(page, at);
        const uint32_t set = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const long long place = static_cast<long long>(base) + pushed - 1 - (rank + __popc(set & ((1u << lane) - 1u)));
            p.page_refs[page] = 0;
            if (place < p.num_pages) p.free_list[place] = page;
            else if (p.status) atomicOr(p.status + find(drop_s, p.B, at >> 7), kKvBadIndex);
        }
        rank += __popc(set);
    });
    cluster_sync_all();   // the tables have been read
    for (int b = cluster_thread(); b < p.B; b += all) {
        if (copy_s[b + 1] == copy_s[b]) continue;
        const int fresh = ld_l2(p.copy_dst + b);
        p.block_table[static_cast<size_t>(b) * p.max_pages + from_s[b]] = fresh;
        if (!page_ok(fresh, p.num_pages)) {
            p.copy_src[b] = p.copy_dst[b] = -1;
            if (p.status) atomicOr(p.status + b, kKvBadIndex);
        }
    }
    if (first_cta)
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            if (from_s[b] < 0) continue;
            p.seq_len[b] = p.new_len[b];
            p.n_pages[b] = from_s[b] + (copy_s[b + 1] - copy_s[b]);
        }
    if (first_cta && threadIdx.x == 0) *p.free_count = min(base + pushed, p.num_pages);
    cluster_sync_all();   // no CTA ends while others read its shared memory
}

// ---------------------------------------------------------------- compaction
// The number of a page among those in use by ballots: a warp walks a run of pages, 32 at a time, and prefix sums over the
// warps' totals give each its start.  With `used` known, the r-th page from the top of those at `used` and above goes to the
// r-th place from the bottom that is not in use: each finds its own r, and writes itself into the pair of that number.
// Bound by the latency of its phases, some 4 us each of the larger of these: page_refs is zeroed, counted up, read twice and written,
// each time through L2 and behind a cluster barrier.  64 sequences of up to 1,024 pages in a cache half of it free take 23 us, of
// which the memory would need 0.2; 8 of up to 32 pages 8.6 us, one CTA.
__global__ void __launch_bounds__(kBookThreads, 1) kv_compact_kernel(const KvCompactParams p) {
    extern __shared__ int smem[];
    int* const held_s = smem;   // [B + 1] entries before each sequence
    __shared__ Pair sums[33];
    __shared__ int used_s, holes_s;
    grid_dependency_wait();
    grid_launch_dependents();
    const int me = cluster_thread(), all = cluster_threads(), lane = threadIdx.x & 31;
    const bool first_cta = cluster_ctarank() == 0;
    for (int g = me; g < p.num_pages; g += all) p.page_refs[g] = 0;
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    auto held = [&](int b) {
        const int n = p.n_pages[b];
        return n >= 0 && n <= p.max_pages ? n : 0;
    };
    Pair ask{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        ask.pages += held(b);
        if (first_cta && p.status && (p.n_pages[b] < 0 || p.n_pages[b] > p.max_pages)) atomicOr(p.status + b, kKvBadIndex);
    }
    Pair at = block_prefix(ask, sums, &total);
    for (int b = b0; b < b1; ++b) {
        held_s[b] = static_cast<int>(at.pages);
        at.pages += held(b);
    }
    if (threadIdx.x == 0) held_s[p.B] = static_cast<int>(total.pages);
    if (threadIdx.x == 0) holes_s = 0;
    cluster_sync_all();
    const int entries = held_s[p.B];
    // a warp takes 128 consecutive entries at a time: one bisection serves those of one sequence
    auto each_entry = [&](auto&& f) {
        for (long long c = static_cast<long long>(me >> 5) * 128; c < entries; c += static_cast<long long>(all >> 5) * 128) {
            const int bc = find(held_s, p.B, static_cast<int>(c)), end = held_s[bc + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long g = c + i * 32 + lane;
                if (g >= entries) continue;
                const int b = g < end ? bc : find(held_s, p.B, static_cast<int>(g));
                f(b, static_cast<size_t>(b) * p.max_pages + static_cast<size_t>(g - held_s[b]));
            }
        }
    };
    each_entry([&](int b, size_t e) {
        const int page = p.block_table[e];
        if (page_ok(page, p.num_pages)) atomicAdd(p.page_refs + page, 1);
        else if (p.status) atomicOr(p.status + b, kKvBadIndex);
    });
    cluster_sync_all();
    // this warp's run of pages
    const int warps = all >> 5, run = (p.num_pages / 32 + (p.num_pages % 32 > 0) + warps - 1) / warps;   // of 32 pages
    const long long p0 = static_cast<long long>(me >> 5) * run * 32, p1 = min(static_cast<long long>(p.num_pages), p0 + static_cast<long long>(run) * 32);
    int in_use = 0;
    for (long long g = p0; g < p1; g += 32) {
        const bool u = g + lane < p1 && ld_l2(p.page_refs + g + lane) > 0;
        in_use += __popc(__ballot_sync(0xffffffffu, u));
    }
    Pair before = block_prefix(Pair{lane == 0 ? in_use : 0, 0}, sums, &total);
    if (threadIdx.x == 0) used_s = static_cast<int>(total.rows);
    cluster_sync_all();
    int below = static_cast<int>(__shfl_sync(0xffffffffu, before.rows, 0)), used = 0;
    for (uint32_t c = 0; c < cluster_ctas(); ++c) {
        const int n = ld_dsmem_int(&used_s, c);
        if (c < cluster_ctarank()) below += n;
        used += n;
    }
    int holes = 0;
    for (long long g = p0; g < p1; g += 32) {
        const int page = static_cast<int>(g) + lane;
        const bool in = g + lane < p1;
        const int count = in ? ld_l2(p.page_refs + page) : 0;
        const uint32_t set = __ballot_sync(0xffffffffu, count > 0);
        if (in) {
            const int n = below + __popc(set & ((1u << lane) - 1u));   // in use below this page
            if (count > 0 && page < used) {
                p.page_map[page] = page;
                p.page_refs[page] = count - 1;
            } else if (count > 0) {
                p.copy_src[used - 1 - n] = page;
            } else {
                p.page_map[page] = -1;
                if (page < used) {
                    p.copy_dst[page - n] = page;
                    ++holes;
                }
            }
        }
        below += __popc(set);
    }
    for (int o = 16; o > 0; o >>= 1) holes += __shfl_xor_sync(0xffffffffu, holes, o);
    if (lane == 0 && holes > 0) atomicAdd(&holes_s, holes);
    cluster_sync_all();
    int moves = 0;
    for (uint32_t c = 0; c < cluster_ctas(); ++c) moves += ld_dsmem_int(&holes_s, c);
    for (int r = me; r < p.n_copy_max; r += all) {
        if (r < moves) {
            const int src = ld_l2(p.copy_src + r), dst = ld_l2(p.copy_dst + r);
            p.page_map[src] = dst;
            p.page_refs[dst] = ld_l2(p.page_refs + src) - 1;
            p.page_refs[src] = 0;
        } else {
            p.copy_src[r] = p.copy_dst[r] = -1;
        }
    }
    for (int i = me; i < p.num_pages - used; i += all) p.free_list[i] = p.num_pages - 1 - i;
    if (me == 0) {
        *p.free_count = p.num_pages - used;
        *p.n_copy = moves;
    }
    cluster_sync_all();
    each_entry([&](int, size_t e) {
        const int page = p.block_table[e];
        p.table_out[e] = page_ok(page, p.num_pages) ? ld_l2(p.page_map + page) : page;
    });
}

// One cluster of `ctas` CTAs (more than 8 have to be allowed, and 8 are taken where the device or a part of it has no room for more) with
// `words` words of shared memory, most of them `most` (the kernel's limit, the same by every call: another thread's call may come
// between it and the launch).
template <typename P>
cudaError_t launch_books(void (*kernel)(P), const P& p, int ctas, size_t words, size_t most, cudaStream_t stream) {
    const size_t smem = words * 4;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most * 4));
        if (e != cudaSuccess) return e;
    }
    if (ctas > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        ctas = cluster_that_fits(ctas, [&](int n) { return clusters_at_once(kernel, n, dim3(n), dim3(kBookThreads), smem, stream); });
    }
    return launch_dependent_cluster(kernel, ctas, dim3(ctas), dim3(kBookThreads), smem, stream, p);
}

// ---------------------------------------------------------------- copies
// Elementwise, every byte read and written once: bound by the memory (16,000 pages of 16 tokens of 4 heads of 256, 2.1 GB, 333 us,
// 6.3 TB/s, 93% of what one large copy reaches).  A CTA takes 256 x 8 accesses of 16 bytes of one
// page's keys or values at a time, all loads before the first store.  A page is `outer` runs of `inner` runs of `run`
// consecutive vectors (one run where it lies in one piece).
constexpr int kCopyThreads = 256, kCopyBatch = 8;

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const KvCopyParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long items = static_cast<long long>(p.n) * 2 * p.chunks;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int chunk = static_cast<int>(it % p.chunks);
        const long long pair = it / p.chunks;
        const int i = static_cast<int>(pair >> 1);
        const int src = p.copy_src[i], dst = p.copy_dst[i];
        if (src < 0 || dst < 0) continue;
        if (src >= p.cache.num_pages || dst >= p.cache.num_pages) {
            if (p.status && threadIdx.x == 0) atomicOr(p.status, kKvBadIndex);
            continue;
        }
        uint4* const half = static_cast<uint4*>(pair & 1 ? p.cache.v : p.cache.k);
        const uint4* const from = half + src * p.page_stride;
        uint4* const to = half + dst * p.page_stride;
        uint4 v[kCopyBatch];
        long long at[kCopyBatch];
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k) {
            const unsigned x = (static_cast<unsigned>(chunk) * kCopyBatch + k) * kCopyThreads + threadIdx.x;
            at[k] = -1;
            if (x < static_cast<unsigned>(p.vectors)) {
                const unsigned row = x / p.run, o = row / p.inner;
                at[k] = o * p.outer_stride + (row - o * p.inner) * p.inner_stride + (x - row * p.run);
                v[k] = from[at[k]];
            }
        }
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k)
            if (at[k] >= 0) to[at[k]] = v[k];
    }
}

}  // namespace

// Words for the counts of a cache's pages beside `books` others; 0 where there are too many.
int count_room(int num_pages, size_t books) { return num_pages <= kCountPages && books + num_pages <= kMostWords ? num_pages : 0; }

cudaError_t launch_kv_fork(KvForkParams p, cudaStream_t stream) {
    const size_t books = static_cast<size_t>(p.B) + 2 * (static_cast<size_t>(p.N) + 1);
    p.room = count_room(p.num_pages, books);
    return launch_books(kv_fork_kernel, p, ctas_for(static_cast<size_t>(p.N) * p.max_pages), books + p.room, kMostWords, stream);
}

cudaError_t launch_kv_release(KvReleaseParams p, cudaStream_t stream) {
    const size_t books = 3 * (static_cast<size_t>(p.B) + 1);
    p.room = count_room(p.num_pages, books);
    return launch_books(kv_release_kernel, p, ctas_for(static_cast<size_t>(p.B) * p.max_pages), books + p.room, kMostWords, stream);
}

cudaError_t launch_kv_compact(const KvCompactParams& p, cudaStream_t stream) {
    const size_t entries = static_cast<size_t>(p.B) * p.max_pages, pages = static_cast<size_t>(p.num_pages);
    return launch_books(kv_compact_kernel, p, ctas_for(entries > pages ? entries : pages), static_cast<size_t>(p.B) + 1, kKvMaxSeq + 1, stream);
}

cudaError_t launch_kv_copy(KvCopyParams p, cudaStream_t stream) {
    constexpr int kPiece = kCopyThreads * kCopyBatch;
    p.chunks = p.vectors / kPiece + (p.vectors % kPiece > 0);
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    const long long items = static_cast<long long>(p.n) * 2 * p.chunks;
    const int ctas = static_cast<int>(items < sms * 8ll ? items : sms * 8ll);
    return launch_dependent(kv_copy_kernel, dim3(ctas), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace gdn
