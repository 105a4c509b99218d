// gdn_chunk_tc.cu -- gdn_attn_chunk over a bf16 cache with a bf16 result: products on the 5th-generation tensor cores.
//
// A worker is a pair of CTAs (a cluster, two SMs) that work on one unit of up to 256 rows: S = Q . K^T and O += P . V with M = 256,
// 128 rows in each CTA's tensor memory.  The pair shares every tile of 128 keys: of the keys each CTA has 64 in its shared memory,
// of the values half of the channels, and the tensor cores read both.  So a key and a value come from L2 once for 256 rows
// (at d = 256, 4 x 256 operations a byte; with 128 rows a CTA the tensor cores' 2,048 cycles a tile would ask for 64 bytes a
// cycle of every SM).
//
// Roles of a CTA's 16 warps:
//   0-7   softmax: a thread has one row (tensor-memory lane) and 64 of a tile's 128 keys; the two threads of a row meet in shared
//         memory for the maximum.  The result is rescaled only when a row's maximum has risen by more than 2^kSlack.
//   8-11  load keys and values by cp.async, 16 bytes a lane, through the block table; any page size and strides
//   12    one thread: in the first CTA issues the products, in the second tells the first what has landed here
//   13    loads the queries of the next unit as soon as the last product with these has been made
//   14-15 nothing (registers are moved by groups of four warps)
//
// The products of one tile's S are issued before those of the O of the tile before (NS tiles before, where S has two places),
// so that the softmax of a tile runs beside products.  Every order between products that touch the same tensor memory goes
// through a barrier.
//
// A weight is rounded to bf16 (half a step, 2^-9 of it on average less than that; the sum of weights is of the unrounded ones):
// with a second part for what the rounding leaves, as gdn_attn_decode has it, which is bound by memory, the product with the values
// would take twice the time, half again as much for the whole.
#include "gdn_chunk.cuh"

namespace gdn {
namespace chunk {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kWaitLimit = 1 << 20;   // polls of a wait before it gives up
using tc::smem_u32;
constexpr float kSlack = 8.0f;   // how far a score may pass its row's base
constexpr int kRows = 256, kKeys = 128, kThreads = 512, kSoft = 256;
// Registers: 128 a thread at launch; the two softmax warpgroups take over some of the other two's (2 x 152 + 2 x 104 = 4 x 128).
constexpr int kSoftRegs = 152, kOtherRegs = 104;

template <int D_>
struct Tc {
    static constexpr int D = D_;
    static constexpr int NS = D == 256 ? 1 : 2;               // places of S; P has two
    static constexpr int kStage = kKeys * D;                  // bytes: 64 keys, or 128 keys' values of D/2 channels
    static constexpr int RK = D == 256 ? 2 : D == 128 ? 5 : 6;
    static constexpr int RV = D == 256 ? 3 : D == 128 ? 5 : 6;
    static constexpr int kQ = 128 * D * 2;
    static constexpr int kSmem = kQ + (RK + RV) * kStage + 3072;
    // tensor memory
    static constexpr int kO = 0, kS = D == 256 ? 256 : 128, kP = 384;
    static constexpr int kCost = 256;
    static_assert(kSmem <= 232448 && kS + NS * 128 <= kP, "shape");
};

struct Smem {
    float mx[2][2][128];              // by tile mod 2, half of the keys, row; at a part's end the sums, in [0]
    uint32_t valid[16][4];            // keys of a tile that are there, by tile mod 16
    uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
    uint64_t q_full, q_empty, s_full[2], p_ready[2], pv_done[2], drained, never;
    PlanSmem plan;
    uint32_t tmem;
    int last, stop, strays;           // stop: a softmax warp's wait has given up; strays: some were found; never taken back
    volatile int abort;
};
static_assert(sizeof(Smem) <= 3072, "fits");

// ---------------------------------------------------------------- the pair
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_cta(smem_u32(bar), rank)) : "memory");
}
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done != 0;
}
// Wait for phase `parity` of `bar`; false when it gives up or another warp of the CTA has.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, int limit = kWaitLimit) {
#pragma unroll 1
    for (int it = 0; it < limit; ++it) {
        if (try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    return false;
}
__device__ __forceinline__ bool warp_wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, wait_for(bar, parity, abort));
}

// Arrive at `bar` in both CTAs when every product issued so far is done.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}

// Upper words of the shared-memory descriptors: 128-byte swizzle, 8-row groups 1024 bytes apart; and no swizzle, core matrices
// 2048 bytes apart along N.  The lower word is the address / 16 and, for values, the stride of the other direction.
constexpr uint32_t kDescSwizzle = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescPlain = (2048u >> 4) | (1u << 14);

template <uint32_t kHiB>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc),
        "r"(static_cast<uint32_t>(add)), "n"(kDescSwizzle), "n"(kHiB));
}
template <uint32_t kHiB>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(idesc),
        "r"(static_cast<uint32_t>(add)), "n"(kHiB));
}

__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// A walk over the tiles of a worker's parts.
struct Walk {
    Part c;
    int t;
    bool more;
    template <class F>
    __device__ __forceinline__ void settle(const ChunkParams& p, const Line& ln, const Share& sh, F rows) {   // past parts without tiles
        while (more && c.t0 >= c.t1) more = next_part(ln, sh, p.B, p.Hkv, c, rows);
        t = c.t0;
    }
    template <class F>
    __device__ __forceinline__ void next(const ChunkParams& p, const Line& ln, const Share& sh, F rows) {
        if (++t < c.t1) return;
        more = next_part(ln, sh, p.B, p.Hkv, c, rows);
        settle(p, ln, sh, rows);
    }
    __device__ __forceinline__ bool first() const { return t == c.t0; }
    __device__ __forceinline__ bool last() const { return t + 1 == c.t1; }
};

// A row's channels ch..ch+7 of the result, gated.
template <int D>
__device__ __forceinline__ void put8(const ChunkParams& p, long long t, int h, int ch, float (&y)[8]) {
    if (p.gate) {
        float g[8];
        load8(static_cast<const bf16*>(p.gate) + t * p.ldg + static_cast<long long>(h) * D + ch, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= gate_of(g[i]);
    }
    store8(static_cast<bf16*>(p.out) + (t * p.Hq + h) * D + ch, y);
}

// The strays of a unit's late keys (gdn_attn.cuh; those that its first row does not see) are added to the rows that see them,
// in out or in the part at `part`.  A call, for the size of the code around it.
template <int D>
__device__ __noinline__ void add_strays(const ChunkParams& p, const Part& c, int tok0, int row0, int rows, float* part) {
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (D / 4); i += kSoft) {
        const int row = i / (D / 4), ch = i % (D / 4) * 4, tok = (row0 + row) / p.G, h = c.hk * p.G + row0 + row - tok * p.G;
        const int off = c.r.len - c.r.n;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int j = max(0, off + tok0 + 1); j <= off + tok0 + tok; ++j) {
            const int k = j / p.cache.page_size, page = p.block_table[static_cast<size_t>(c.b) * p.max_pages + k];
            if (page < 0 || page >= p.cache.num_pages) continue;
            const float4 v = StateIO<bf16>::ld(static_cast<const bf16*>(p.cache.v) + page * p.cache.page_stride +
                                               (j - k * p.cache.page_size) * p.cache.token_stride + c.hk * p.cache.head_stride + ch);
            y.x += isfinite(v.x) ? 0.f : v.x;
            y.y += isfinite(v.y) ? 0.f : v.y;
            y.z += isfinite(v.z) ? 0.f : v.z;
            y.w += isfinite(v.w) ? 0.f : v.w;
        }
        if (y.x == 0.f && y.y == 0.f && y.z == 0.f && y.w == 0.f) continue;
        if (!part) {
            put<bf16, D, true>(p, true, static_cast<long long>(c.r.row0) + tok0 + tok, h, ch, y);
        } else {
            float4* const at = reinterpret_cast<float4*>(part + static_cast<size_t>(row) * D + ch);
            *at = make_float4(at->x + y.x, at->y + y.y, at->z + y.z, at->w + y.w);
        }
    }
}

__device__ __forceinline__ void sync_row_halves(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory"); }
__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 5, %0;" ::"n"(kSoft) : "memory"); }

template <class S>
__global__ void __launch_bounds__(kThreads, 1) chunk_tc_kernel(const ChunkParams p) {
    constexpr int D = S::D, NS = S::NS, RK = S::RK, RV = S::RV;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const q_s = smem;
    uint8_t* const k_s = q_s + S::kQ;
    uint8_t* const v_s = k_s + RK * S::kStage;
    Smem& sm = *reinterpret_cast<Smem*>(v_s + RV * S::kStage);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_ctarank();
    const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);
    // the first CTA's barriers count the second one's word that it has the same
    if (threadIdx.x < 8) {
        tc::mbar_init(sm.k_full + threadIdx.x, 132 + (rank == 0));   // the loading lanes' copies, and one arrival a warp for the valid word
        tc::mbar_init(sm.v_full + threadIdx.x, 128 + (rank == 0));
        tc::mbar_init(sm.k_empty + threadIdx.x, 1);
        tc::mbar_init(sm.v_empty + threadIdx.x, 1);
    }
    if (threadIdx.x == 0) {
        tc::mbar_init(&sm.q_full, 32 + (rank == 0));
        tc::mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(sm.s_full + i, 1);
            tc::mbar_init(sm.p_ready + i, 16);   // the softmax warps of both CTAs
            tc::mbar_init(sm.pv_done + i, 1);
        }
        tc::mbar_init(&sm.drained, 1);
        tc::mbar_init(&sm.never, 1);
        sm.strays = 0;
        sm.abort = sm.stop = (smem_u32(smem) & 1023) != 0;   // the swizzle goes by address bits 7-9
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");   // the barriers are there before asynchronous arrivals on them
    const Line ln{kRows / p.G, kKeys, S::kCost};
    Share sh;
    Walk w;
    if (!my_share(p, ln, worker, workers, kKeys, sm.plan, sh, w.c)) return;   // both CTAs of a pair, or neither
    auto rows = [&](int b) { return rows_of(p, b); };
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync_all();   // the other CTA's barriers are there too
    tc::fence_after_sync();
    const uint32_t t_o = sm.tmem + S::kO, t_s = sm.tmem + S::kS, t_p = sm.tmem + S::kP;

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------ keys and values
        w.more = true;
        w.settle(p, ln, sh, rows);
        const int pw = warp - 8, ps = p.cache.page_size;
        // Of tile i: lane l's key 64 rank + 16 pw + l % 16 is one that this warp loads the key of, 32 pw + l the value of.
        // [0]: tile g (values), .. [NS]: tile g + NS (keys), [NS + 1]: the one being looked up.
        constexpr int A = NS + 2;
        int kp[A], ki[A], vp[A], vi[A], head[A], seq[A];   // page and place in it (-1: no key); seq -1: no tile
#pragma unroll
        for (int i = 0; i < A; ++i) ki[i] = vi[i] = seq[i] = -1, kp[i] = vp[i] = head[i] = 0;
        bool ok = true;
        const uint32_t ring_k = smem_u32(k_s), ring_v = smem_u32(v_s);
        auto look_up = [&](int a) {
            seq[a] = -1;
            if (!w.more) return;
            seq[a] = w.c.b;
            head[a] = w.c.hk;
            const int end = ln.seen(w.c.r, w.c.i), j0 = w.t * kKeys;   // keys from `end` on are nobody's
            const int* const table = p.block_table + static_cast<size_t>(w.c.b) * p.max_pages;
            auto find = [&](int j, int& page, int& in) {
                in = -1;
                if (j < end) {
                    const int k = j / ps;
                    in = j - k * ps;
                    page = table[k];   // looked at when it is used
                }
            };
            find(j0 + 64 * static_cast<int>(rank) + 16 * pw + (lane & 15), kp[a], ki[a]);
            find(j0 + 32 * pw + lane, vp[a], vi[a]);
            w.next(p, ln, sh, rows);
        };
        auto there_is = [&](int page, int in) { return in >= 0 && page >= 0 && page < p.cache.num_pages; };
        auto offset = [&](int page, int in, int h) {
            return static_cast<long long>(page) * p.cache.page_stride + static_cast<long long>(in) * p.cache.token_stride + static_cast<long long>(h) * p.cache.head_stride;
        };
        auto load_keys = [&](int a, int n) {   // tile number n
            const int st = n % RK;
            if (n >= RK) ok = warp_wait_for(sm.k_empty + st, (n / RK - 1) & 1, &sm.abort);
            if (!ok) return;
            const uint32_t v_there = __ballot_sync(0xffffffffu, there_is(vp[a], vi[a]));
            if (vi[a] >= 0 && !there_is(vp[a], vi[a]) && p.status) atomicOr(p.status + seq[a], kKvBadIndex);
            if (lane == 0) sm.valid[n & 15][pw] = v_there;
            const bool in_cache = there_is(kp[a], ki[a]);
            const uint32_t there = __ballot_sync(0xffffffffu, in_cache);
            const long long off = in_cache ? offset(kp[a], ki[a], head[a]) : 0;
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;   // lanes a row, rows an instruction
            const int ch = lane % kLanes, sub = lane / kLanes;
#pragma unroll
            for (int e = 0; e < 16 / kAtOnce; ++e) {
                const int i = e * kAtOnce + sub, row = 16 * pw + i;
                const long long o = __shfl_sync(0xffffffffu, off, i);
                tc::cp_async16_zfill(ring_k + st * S::kStage + (ch >> 3) * 8192 + row * 128 + ((ch ^ row) & 7) * 16,
                                     static_cast<const bf16*>(p.cache.k) + o + ch * 8, (there >> i) & 1 ? 16u : 0u);
            }
            tc::cp_async_mbar_arrive(sm.k_full + st);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(sm.k_full + st);
        };
        auto load_values = [&](int a, int n) {
            const int st = n % RV;
            if (n >= RV) ok = warp_wait_for(sm.v_empty + st, (n / RV - 1) & 1, &sm.abort);
            if (!ok) return;
            const bool in_cache = there_is(vp[a], vi[a]);
            const uint32_t there = __ballot_sync(0xffffffffu, in_cache);
            const long long off = (in_cache ? offset(vp[a], vi[a], head[a]) : 0) + rank * (D / 2);
            constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes;
            const int ch = lane % kLanes, sub = lane / kLanes;
#pragma unroll
            for (int e = 0; e < 32 / kAtOnce; ++e) {
                const int i = e * kAtOnce + sub, row = 32 * pw + i;
                const long long o = __shfl_sync(0xffffffffu, off, i);
                const uint32_t at = D == 64 ? (row >> 3) * 128 + ch * 2048 + (row & 7) * 16 : (ch >> 3) * 16384 + row * 128 + ((ch ^ row) & 7) * 16;
                tc::cp_async16_zfill(ring_v + st * S::kStage + at, static_cast<const bf16*>(p.cache.v) + o + ch * 8, (there >> i) & 1 ? 16u : 0u);
            }
            tc::cp_async_mbar_arrive(sm.v_full + st);
        };
#pragma unroll
        for (int i = 0; i <= NS; ++i) look_up(i);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (ok && seq[i] >= 0) load_keys(i, i);
#pragma unroll 1
        for (int g = 0; ok && seq[0] >= 0; ++g) {
            look_up(NS + 1);
            if (seq[NS] >= 0) load_keys(NS, g + NS);
            if (ok) load_values(0, g);
#pragma unroll
            for (int i = 0; i <= NS; ++i) {
                kp[i] = kp[i + 1];
                ki[i] = ki[i + 1];
                vp[i] = vp[i + 1];
                vi[i] = vi[i + 1];
                head[i] = head[i + 1];
                seq[i] = seq[i + 1];
            }
        }
        tc::cp_async_wait_all();   // nothing is in flight when the CTA ends
    } else if (warp == 13) {
        // ------------------------------------------------------------ queries
        bool more = true, ok = true;
        int n = 0;
        Part& c = w.c;
        while (more && ok) {
            if (c.t0 < c.t1) {
                if (n > 0) ok = warp_wait_for(&sm.q_empty, (n - 1) & 1, &sm.abort);
                if (!ok) break;
                const int n_rows = tokens_of(ln, c) * p.G;
                const long long t0 = static_cast<long long>(c.r.row0) + static_cast<long long>(c.i) * ln.tokens;
                constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
                const int ch = lane % kLanes, sub = lane / kLanes;
#pragma unroll 4
                for (int i = sub; i < 128; i += kAtOnce) {
                    const int r = static_cast<int>(rank) * 128 + i, tok = r / p.G;
                    const bool there = r < n_rows;
                    const long long o = there ? (t0 + tok) * p.ldq + static_cast<long long>(c.hk * p.G + r - tok * p.G) * D : 0;
                    tc::cp_async16_zfill(smem_u32(q_s) + (ch >> 3) * 16384 + i * 128 + ((ch ^ i) & 7) * 16,
                                         static_cast<const bf16*>(p.q) + o + ch * 8, there ? 16u : 0u);
                }
                tc::cp_async_mbar_arrive(&sm.q_full);
                ++n;
            }
            more = next_part(ln, sh, p.B, p.Hkv, c, rows);
        }
        tc::cp_async_wait_all();
    } else if (warp == 12) {
        if (lane == 0) {
            w.more = true;
            w.settle(p, ln, sh, rows);
            bool ok = true;
            int nq = 0, units = 0;   // S issued, units begun
            auto landed = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && wait_for(bar, parity, &sm.abort);
                tc::fence_proxy_async();   // its copies are there for the tensor cores
            };
            if (rank != 0) {
                // -------------------------------------------------------- the second CTA: tell the first, in the order of use
                auto tell = [&](uint64_t* bar, uint32_t parity) {
                    landed(bar, parity);
                    if (ok) arrive_at(bar, 0);
                };
                auto keys = [&]() {
                    if (w.first()) tell(&sm.q_full, units++ & 1);
                    tell(sm.k_full + nq % RK, (nq / RK) & 1);
                    ++nq;
                    w.next(p, ln, sh, rows);
                };
                for (int i = 0; i < NS && w.more && ok; ++i) keys();
#pragma unroll 1
                for (int g = 0; g < nq && ok; ++g) {
                    const bool after = !w.more || w.first();
                    if (!after) keys();
                    if (ok) tell(sm.v_full + g % RV, (g / RV) & 1);
                    if (after && w.more && ok) keys();
                }
            } else {
                // -------------------------------------------------------- the first: the products
                constexpr uint32_t id_s = tc::idesc_bf16(256, 128);
                constexpr uint32_t id_o = tc::idesc_f16(256, D, 0, 1, 0) | (1u << 7) | (1u << 10);
                constexpr uint32_t kHiV = D == 64 ? kDescPlain : kDescSwizzle;
                const uint32_t q_lo = (smem_u32(q_s) >> 4) + (1u << 16), k_lo = (smem_u32(k_s) >> 4) + (1u << 16);
                const uint32_t v_lo = (smem_u32(v_s) >> 4) + ((D == 64 ? 128u >> 4 : 16384u >> 4) << 16);
                uint32_t firsts = 0;   // by tile mod 32: the first of a part
                auto keys_landed = [&]() {
                    if (w.first()) landed(&sm.q_full, units++ & 1);
                    landed(sm.k_full + nq % RK, (nq / RK) & 1);
                };
                auto issue_s = [&]() {   // of tile number nq, whose operands have landed
                    const uint32_t d = t_s + nq % NS * 128, b = k_lo + nq % RK * (S::kStage >> 4);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss<kDescSwizzle>(d, q_lo + c * (16384 >> 4) + 2 * kk, b + c * (8192 >> 4) + 2 * kk, id_s, (c | kk) != 0);
                    commit_both(sm.s_full + nq % NS);
                    commit_both(sm.k_empty + nq % RK);
                    if (w.last()) commit_both(&sm.q_empty);
                    firsts = (firsts & ~(1u << (nq & 31))) | (static_cast<uint32_t>(w.first()) << (nq & 31));
                    ++nq;
                    w.next(p, ln, sh, rows);
                };
                for (int i = 0; i < NS && w.more && ok; ++i) {
                    keys_landed();
                    tc::fence_after_sync();
                    if (ok) issue_s();
                }
#pragma unroll 1
                for (int g = 0; g < nq && ok; ++g) {
                    const bool after = !w.more || w.first();   // a next unit's queries may be late: not before this tile's O
                    if (!after) keys_landed();
                    landed(sm.v_full + g % RV, (g / RV) & 1);
                    ok = ok && wait_for(sm.p_ready + (g & 1), (g >> 1) & 1, &sm.abort);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (!after) issue_s();   // into the place that the softmax has read
                    const uint32_t a = t_p + (g & 1) * 64, b = v_lo + g % RV * (S::kStage >> 4);
                    const bool add = !((firsts >> (g & 31)) & 1);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) mma_ts<kHiV>(t_o, a + ks * 8, b + ks * ((D == 64 ? 256 : 2048) >> 4), id_o, add || ks != 0);
                    commit_both(sm.pv_done + (g & 1));
                    commit_both(sm.v_empty + g % RV);
                    if (after && w.more) {
                        keys_landed();
                        tc::fence_after_sync();
                        if (ok) issue_s();
                    }
                }
                // everything issued is through before the pair ends
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&sm.drained)) : "memory");
                tc::mbar_wait(&sm.drained, 0, kWaitLimit);
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
        const uint32_t my_lanes = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t my_o = t_o + my_lanes + half * (D / 2);
        const float scale = p.scale * kLog2e;
        const Parts<kRows, D> parts(p.workspace, workers);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool done = warp_wait_for(bar, parity, &sm.abort);
            if (!done) sm.stop = 1;
            return done;
        };
        int g = 0;   // tile number
        Part& c = w.c;
        do {
            const int tok0 = c.i * ln.tokens, n_rows = tokens_of(ln, c) * p.G, off = c.r.len - c.r.n;
            const int row0 = static_cast<int>(rank) * 128, here = min(max(n_rows - row0, 0), 128);   // rows of this CTA
            const int tok = (row0 + row) / p.G;
            const int end = ln.seen(c.r, c.i);
            float m = -INFINITY, base = 0.f, limit = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int t = c.t0; t < c.t1; ++t, ++g) {
                if (!wait(sm.s_full + g % NS, (g / NS) & 1)) continue;
                tc::fence_after_sync();
                float s[64];
                {
                    const uint32_t at = t_s + my_lanes + g % NS * 128 + half * 64;
                    tc::tmem_ld32(at, reinterpret_cast<float(&)[32]>(s[0]));
                    tc::tmem_ld32(at + 32, reinterpret_cast<float(&)[32]>(s[32]));
                }
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 y = mul2(make_float2(s[i], s[i + 1]), make_float2(scale, scale));
                    s[i] = y.x;
                    s[i + 1] = y.y;
                }
                const uint32_t there[2] = {sm.valid[g & 15][2 * half], sm.valid[g & 15][2 * half + 1]};
                // late: some rows do not see some of the tile's keys
                const bool late = (t + 1) * kKeys > off + tok0 + 1;
                if (late || (there[0] & there[1]) != 0xffffffffu) {
                    const int sees = off + tok0 + tok + 1 - t * kKeys - half * 64;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = sees - i * 32;
                        const uint32_t x = n <= 0 ? 0u : n >= 32 ? there[i] : there[i] & ((1u << n) - 1u);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[i * 32 + e] = (x >> e) & 1 ? s[i * 32 + e] : -INFINITY;
                    }
                }
                float mx = fmaxf(s[0], s[1]);
#pragma unroll
                for (int i = 2; i < 64; i += 2) mx = fmaxf(mx, fmaxf(s[i], s[i + 1]));
                sm.mx[g & 1][half][row] = mx;
                sync_row_halves(quarter);
                mx = fmaxf(mx, sm.mx[g & 1][half ^ 1][row]);
                if (__any_sync(0xffffffffu, mx > limit)) {   // the same for both halves
                    const bool fresh = t == c.t0;
                    // the tile before has been added: O stands still
                    const bool through = fresh || wait(sm.pv_done + ((g - 1) & 1), ((g - 1) >> 1) & 1);
                    tc::fence_after_sync();
                    const float m2 = fmaxf(m, mx);
                    const bool none = m2 == -INFINITY;   // a row that has seen no key
                    const float f = none ? 0.f : ex2(m - m2);
                    m = m2;
                    base = none ? 0.f : m2;
                    limit = none ? -INFINITY : m2 + kSlack;
                    l *= f;
                    if (!fresh && through) {
#pragma unroll 1
                        for (int i = 0; i < D / 2; i += 32) {
                            float v[32];
                            tc::tmem_ld32(my_o + i, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= f;
                            tc::tmem_st32(my_o + i, v);
                        }
                    }
                }
                uint32_t w2[32];
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float x = ex2(s[2 * i] - base), y = ex2(s[2 * i + 1] - base);
                    sum.x += x;
                    sum.y += y;
                    w2[i] = StateIO<bf16>::pack(x, y);
                }
                l += sum.x + sum.y;
                if (g >= 2) wait(sm.pv_done + (g & 1), ((g >> 1) - 1) & 1);   // the weights that were in this place have been read
                tc::fence_after_sync();
                tmem_st32u(t_p + my_lanes + (g & 1) * 64 + half * 32, w2);
                if (late) {
                    // strays among the values that some rows do not see are taken out of this CTA's half of the channels
                    const int k0 = max(0, off + tok0 + 1 - t * kKeys), k1 = min(kKeys, end - t * kKeys);
                    if (k0 < k1 && wait(sm.v_full + g % RV, (g / RV) & 1)) {
                        uint8_t* const st = v_s + g % RV * S::kStage;
                        bool found = false;
#pragma unroll 1
                        for (int x = threadIdx.x; x < (k1 - k0) * (D / 16); x += kSoft) {
                            const int key = k0 + x / (D / 16), ch = x % (D / 16);
                            found |= attn::take_strays<bf16>(st + (D == 64 ? key / 8 * 128 + ch * 2048 + key % 8 * 16
                                                                           : ch / 8 * 16384 + key * 128 + ch % 8 * 16));
                        }
                        if (found) {
                            sm.strays = 1;
                            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(smem_u32(&sm.strays), rank ^ 1)), "r"(1) : "memory");
                        }
                        tc::fence_proxy_async();
                    }
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_at(sm.p_ready + (g & 1), 0);
            }
            // -------------------------------------------------------- the part's end
            const bool any = c.t0 < c.t1, whole = c.whole();
            const size_t place = parts.place(worker, c);
            if (any) wait(sm.pv_done + ((g - 1) & 1), ((g - 1) >> 1) & 1);
            tc::fence_after_sync();
            if (p.test_stall && warp == 3 && !wait_for(&sm.never, 0, &sm.abort, 256)) sm.stop = 1;
            sm.mx[0][half][row] = l;   // (all have read the last tile's maximum: its weights were waited for)
            sync_softmax();
            if (sm.stop) {   // a wait gave up: nothing of this part is written
                if (threadIdx.x == 0 && p.status) atomicOr(p.status + c.b, 16);
            } else {
                const float sum = sm.mx[0][0][row] + sm.mx[0][1][row], f = sum == 0.f ? 0.f : 1.0f / sum;
                const long long tr = static_cast<long long>(c.r.row0) + tok0 + tok;
                const int h = c.hk * p.G + row0 + row - tok * p.G;
                float* const part = parts.o + (place * kRows + row0) * D;
#pragma unroll 1
                for (int i = 0; i < D / 2; i += 32) {
                    float v[32];
                    if (any) tc::tmem_ld32(my_o + i, v);
                    if (row < here) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float y[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) y[x] = any ? v[e + x] * (whole ? f : 1.0f) : 0.f;
                            const int ch = half * (D / 2) + i + e;
                            if (whole) put8<D>(p, tr, h, ch, y);
                            else store8(part + static_cast<size_t>(row) * D + ch, y);
                        }
                    }
                }
                if (!whole && half == 0 && row < here) parts.ml[place * kRows + row0 + row] = make_float2(m, sum);
                if (sm.strays) {
                    sync_softmax();
                    add_strays<D>(p, c, tok0, row0, here, whole ? nullptr : part);
                }
                if (!whole) {   // the worker that arrives last joins this CTA's rows of all parts, in their order
                    const long long first = c.at + ln.cost;
                    const int w0 = sh.owner(first), n = sh.owner(first + static_cast<long long>(kKeys) * (c.tiles - 1)) - w0 + 1;
                    sync_softmax();
                    if (threadIdx.x == 0) {
                        unsigned old;
                        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(parts.counters + 2 * w0 + rank), "r"(n - 1) : "memory");
                        sm.last = old == static_cast<unsigned>(n - 1);
                    }
                    sync_softmax();
                    if (sm.last) {
                        auto at = [&](int k) { return (k == 0 ? 2 * static_cast<size_t>(w0) + 1 : 2 * static_cast<size_t>(w0 + k)) * kRows + row0; };
#pragma unroll 1
                        for (int i = threadIdx.x; i < here * (D / 4); i += kSoft) {
                            const int r = i / (D / 4), ch = i % (D / 4) * 4, tk = (row0 + r) / p.G;
                            float mm = -INFINITY, ll = 0.f;
                            for (int k = 0; k < n; ++k) mm = fmaxf(mm, __ldcg(parts.ml + at(k) + r).x);
                            const float b0 = mm == -INFINITY ? 0.f : mm;
                            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                            for (int k = 0; k < n; ++k) {
                                const float2 z = __ldcg(parts.ml + at(k) + r);
                                const float fk = ex2(z.x - b0);
                                const float4 v = __ldcg(reinterpret_cast<const float4*>(parts.o + (at(k) + r) * D + ch));
                                ll = fmaf(fk, z.y, ll);
                                y = make_float4(fmaf(fk, v.x, y.x), fmaf(fk, v.y, y.y), fmaf(fk, v.z, y.z), fmaf(fk, v.w, y.w));
                            }
                            put<bf16, D>(p, true, static_cast<long long>(c.r.row0) + tok0 + tk, c.hk * p.G + row0 + r - tk * p.G, ch,
                                         attn::times(y, ll == 0.f ? 0.f : 1.0f / ll));
                        }
                    }
                }
                tc::fence_before_sync();
            }
            sync_softmax();   // the sums and sm.last have been read
        } while (next_part(ln, sh, p.B, p.Hkv, c, rows));
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync_all();   // no product, copy or arrival concerns this pair any more
    tc::fence_after_sync();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem), "r"(512));
}

template <int D>
cudaError_t launch(const ChunkParams& p, int sms, cudaStream_t stream) {
    using S = Tc<D>;
    const cudaError_t e = cudaFuncSetAttribute(chunk_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    const int pairs = min(sms / 2, kMaxWorkers / 2);
    return launch_dependent_cluster(chunk_tc_kernel<S>, 2, dim3(2 * pairs), dim3(kThreads), S::kSmem, stream, p);
}

}  // namespace

size_t tc_workspace_bytes(int head_dim) {
    if (head_dim == 64) return parts_bytes<kRows, 64>(kMaxWorkers / 2);
    if (head_dim == 128) return parts_bytes<kRows, 128>(kMaxWorkers / 2);
    return parts_bytes<kRows, 256>(kMaxWorkers / 2);
}

cudaError_t launch_tc(const ChunkParams& p, int head_dim, int sms, cudaStream_t stream) {
    if (head_dim == 64) return launch<64>(p, sms, stream);
    if (head_dim == 128) return launch<128>(p, sms, stream);
    return launch<256>(p, sms, stream);
}

}  // namespace chunk
}  // namespace gdn
