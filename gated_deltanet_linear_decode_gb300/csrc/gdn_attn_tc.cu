// gdn_attn_tc.cu -- gdn_attn_decode over a bf16 cache, with a bf16 result, for more than 32 rows a kv head (a speculative
// verify of wide groups): the products on the 5th-generation tensor cores.  The division of the keys over the CTAs, the page look-ups
// and the join of split groups are those of gdn_attn.cuh.
//
// With R rows the products take 4 R d operations a key of 4 d bytes.  On mma.sync every 16 rows read the keys and
// values from shared memory again (and the queries once per 16 keys): at 24 rows and d = 256 that is 2,050 cycles of a
// tile of 64 keys, against 1,500 at the memory's rate, and it grows with R.  tcgen05.mma reads each operand once.
//
// A tile is 128 keys; S = Q . K^T and O += P . V have M = 128 tensor-memory lanes.  A block of NR = 64 or 128 rows
// takes the lanes 128/NR times: lane x holds row x % NR and, of every tile, only the NR keys from (x / NR) NR on; the
// other keys' weights in its lane of P are zeros.  So a thread a lane has its keys' scores, maximum and sum to itself -- the
// softmax has no shuffle and no barrier -- and the copies of a row meet once, at a group's end, as key groups do.  The
// tensor cores do 128 rows' work whatever R is: 48 products a tile at d = 256, 4,240 cycles measured, under the 5,500
// its 128 KB take.  (With the keys or channels on the M side and R on the N side, a product of N = 32 took as long as one
// of N = 128, and the softmax needed its maximum over lanes.)
//
// Measured, 64 ragged sequences of up to 8192 keys (0.54 GB, floor 82 us), 16/2 heads of 256: 64 rows 163 us, 128 rows 249 us (277
// TFLOP/s); 64/8 heads of 64: 248 and 492.  What bounds it: 128 rows the softmax (a thread's 128 keys a tile, 8,300 cycles when they
// were counted); 64 rows a group's end, much of it the fetch of code that runs about twice a CTA: 100 to 130 KB of it, and where it
// was 160 to 190 KB all of these took 10 to 40% longer.
// Roles, one persistent CTA per SM:
//   warps 0-3   a thread a lane: S from tensor memory, weights e^(s - base) as two bf16 parts back into its place;
//   warps 4-11  load: cp.async into a ring of 16 KB units, 128 keys x 64 channels each in the 128-byte swizzle
//               layout, in the order of their use, with zero fill for keys that are not there;
//   warp 12     one thread issues S (both operands K-major in shared memory) two tiles ahead of O (P in tensor memory, V as
//               it lies in the ring, MN-major); a commit hands each unit back.
// The base of a lane is its running maximum, but it is raised (and its O and l scaled) only when a score passes it by
// more than 8 in base 2: then all weights stay under 2^8, the sums in 32 bits are as exact as with the maximum
// itself, and O is hardly ever read before the end.  (The tensor cores' sums drop what is below the last bit: 4.5e-5 of the
// result at 16,000 keys a CTA, a fortieth of a bf16 result's own rounding.)
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kUnit = 16384;      // 128 keys x 64 channels
constexpr float kSlack = 8.0f;    // how far a score may pass its row's base

template <int D_, int NR_>
struct TcShape {
    using Ta = bf16;
    static constexpr int D = D_, NR = NR_;
    static constexpr int kRows = NR;          // rows of a block
    static constexpr int kThreads = 128;      // softmax
    static constexpr int kLoaders = 8;        // warps that load, 16 keys of a tile each
    static constexpr int kAll = 32 * (4 + kLoaders + 1);
    static constexpr int kTile = 128;         // keys
    // at d = 256, with the larger code (above): 64 rows 2 tiles 204 us, 8 tiles 174, 16 tiles 187; 128 rows 8 tiles 288 us, 12 tiles 275
    static constexpr int kGroupCost = D == 256 ? (NR == 64 ? 8 : 12) : D == 128 ? 6 : 4;
    static constexpr int kCols = D / 64;      // units of a tile's keys, and of its values
    static constexpr int NV = D > 64 ? 128 : 64;   // channels of one product with V: two units side by side, or one
    static constexpr int kPerV = NV / 64;
    static constexpr int kPart = (kMaxFan * 4 + 8) * NR;   // join of parts
    static constexpr int kQBytes = 256 * D > kPart ? 256 * D : kPart;   // Q; at a group's end the copies of its rows, then parts
    static constexpr int kFit = (232448 - 3072 - kQBytes) / kUnit;
    static constexpr int kUnits = kFit > 12 ? 12 : kFit / 2 * 2;        // even: two units of values lie side by side
    static constexpr int kSmem = kUnits * kUnit + kQBytes + 3072;
    // Tensor memory: twice 128 columns where a tile's S and then its P lie, and O.
    static constexpr int kColO = 256;
    static_assert(kUnits >= 6 && kSmem <= 232448 && kColO + D <= 512, "shape");
};

// What follows the operands in shared memory.
struct TcSmem {
    float2 ml[128];                           // of a lane: maximum and sum; then of a row
    float f[128];                             // of a lane: its share's weight in the row
    uint16_t valid[16][8];                    // keys of a tile that are there, by tile mod 16
    uint64_t full[16], empty[12];             // of half a tile (its keys or its values), by number mod 16; of a unit
    uint64_t q_ready, s_full[2], p_ready[2], o_done, drained, never;
    PlanSmem plan;
    uint32_t tmem;
    int flag, stop, strays;                   // stop: a softmax warp's wait has given up, strays: some were found; never taken back
    volatile int abort;
};
static_assert(sizeof(TcSmem) <= 3072, "fits");

// The issuing thread's instructions are on the critical path, so a descriptor is put together from its two words: the
// upper one a constant of the layout, the lower one (address / 16, and for MN-major the step along M/N) one addition.
// K-major, 128-byte swizzle, 8-row groups 1024 bytes apart:
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescLoK = 1u << 16;
// MN-major, 128-byte swizzle: rows (along K) of 64 elements, 8-row groups 1024 bytes apart, the next 64 elements along
// N one unit on:
constexpr uint32_t kDescLoN = static_cast<uint32_t>(kUnit >> 4) << 16;

// D (+)= A . B with both operands in shared memory, and with A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc),
        "r"(static_cast<uint32_t>(add)), "n"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(idesc),
        "r"(static_cast<uint32_t>(add)), "n"(kDescHi));
}

// Add the strays to the results of a group's rows.  A call, for the size of the code around it.
template <class S>
__device__ __noinline__ void add_strays(const AttnParams& p, int b, int hk, int row0, int len, int rows) {
    constexpr int D = S::D;
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (D / 4); i += S::kThreads) {
        const int row = i / (D / 4), c = i % (D / 4) * 4;
        const float4 x = strays_of<bf16>(p, b, hk, len, row0 + row, c);
        if (x.x == 0.f && x.y == 0.f && x.z == 0.f && x.w == 0.f) continue;
        put<bf16, D, true>(p, true, b, hk, row0 + row, c, x);
    }
}

template <class S>
__global__ void __launch_bounds__(S::kAll, 1) attn_tc_kernel(const AttnParams p) {
    constexpr int D = S::D, NR = S::NR, kUnits = S::kUnits;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const q_s = smem + kUnits * kUnit;
    TcSmem& sm = *reinterpret_cast<TcSmem*>(q_s + S::kQBytes);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.G * p.K, row_blocks = (R + NR - 1) / NR;
    if (threadIdx.x < kUnits) {
        tc::mbar_init(sm.empty + threadIdx.x, 1);
    }
    // each loading lane's copies, and one arrival a warp for the valid word
    if (threadIdx.x < 16) tc::mbar_init(sm.full + threadIdx.x, S::kLoaders * 33);
    if (threadIdx.x == 0) {
        tc::mbar_init(&sm.q_ready, 128);
        tc::mbar_init(&sm.s_full[0], 1);
        tc::mbar_init(&sm.s_full[1], 1);
        tc::mbar_init(&sm.p_ready[0], 128);   // by a tile's place, as s_full: the threads may be a tile ahead
        tc::mbar_init(&sm.p_ready[1], 128);
        tc::mbar_init(&sm.o_done, 1);
        tc::mbar_init(&sm.drained, 1);
        tc::mbar_init(&sm.never, 1);
        sm.strays = 0;
        sm.abort = sm.stop = (tc::smem_u32(smem) & 1023) != 0;   // the swizzle goes by address bits 7-9
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");   // the barriers are there before asynchronous arrivals on them
    Cursor cc;
    Share sh;
    if (!my_share<S>(p, row_blocks, sm.plan, cc, sh)) return;
    const long long last = sh.last;
    bool over;
    constexpr int kIssuer = 4 + S::kLoaders;
    if (warp == kIssuer) tc::tmem_alloc(&sm.tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t t_s = sm.tmem, t_o = t_s + S::kColO;

    if (warp >= 4 && warp < kIssuer) {
        // ------------------------------------------------------------ the loading warps; lane l < 16 of warp w knows key 16 w + l
        const int pw = warp - 4, ps = p.cache.page_size;
        const uint32_t ring = tc::smem_u32(smem);
        // Tile i is at [0], those after it at [1] and [2], the one being looked up at [3].
        int page[4] = {0, 0, 0, 0}, in_page[4] = {0, 0, 0, 0}, head[4] = {0, 0, 0, 0}, seq[4] = {-1, -1, -1, -1};   // seq -1: no key
        int tiles = 0, unit = 0, halves = 0;
        uint32_t round = 0;
        uint32_t begins = 0, ends = 0;   // bit k: tile [k] is the first, the last of a group in this CTA
        bool ok = true, first_tile = true;
        // half a tile: its keys' channels (of tile number i) or its values', kCols units, 4 rows of 128 bytes an instruction
        auto load = [&](const void* half, int k, int i) {
            const bool in_cache = page[k] >= 0 && page[k] < p.cache.num_pages;
            const uint32_t there = __ballot_sync(0xffffffffu, seq[k] >= 0 && in_cache);
            if (seq[k] >= 0 && !in_cache && p.status) atomicOr(p.status + seq[k], kKvBadIndex);
            const long long off = page[k] * p.cache.page_stride + in_page[k] * p.cache.token_stride + head[k] * p.cache.head_stride;
            const bf16* src[4];
            int n[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = e * 4 + (lane >> 3);
                const long long o = __shfl_sync(0xffffffffu, off, key);
                n[e] = (there >> key) & 1 ? 16 : 0;
                src[e] = static_cast<const bf16*>(half) + (n[e] ? o : 0) + (lane & 7) * 8;
            }
            const int row = pw * 16 + (lane >> 3);
            // row + 4 e: its swizzle is that of row with bit 2 flipped for odd e
            const uint32_t d0 = ring + row * 128 + ((lane & 7) ^ (row & 7)) * 16, d1 = d0 ^ 64;
#pragma unroll 1
            for (int c = 0; c < S::kCols; ++c) {
                if (c % 2 == 0 || S::kCols == 1) {   // units are handed back in order: one wait for two of them
                    const int u = S::kCols == 1 ? unit : unit + 1;
                    if (round > 0) ok = warp_wait(sm.empty + u, (round - 1) & 1, &sm.abort);
                    if (!ok) return;
                }
                if (c == 0 && i >= 0 && lane == 0) sm.valid[i & 15][pw] = static_cast<uint16_t>(there);
#pragma unroll
                for (int e = 0; e < 4; ++e) tc::cp_async16_zfill((e & 1 ? d1 : d0) + unit * kUnit + e * 512, src[e] + c * 64, n[e]);
                if (++unit == kUnits) {
                    unit = 0;
                    ++round;
                }
            }
            tc::cp_async_mbar_arrive(sm.full + (halves & 15));
            if (lane == 0) tc::mbar_arrive(sm.full + (halves & 15));
            ++halves;
        };
#pragma unroll 1
        for (int t = 0; ok; ++t) {   // turn t looks up the pages of tile t and loads for tile t - 3
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                page[k] = page[k + 1];
                in_page[k] = in_page[k + 1];
                head[k] = head[k + 1];
                seq[k] = seq[k + 1];
            }
            seq[3] = -1;
            begins >>= 1;
            ends >>= 1;
            if (cc.at < last) {
                const int j = cc.tile * 128 + pw * 16 + lane;
                if (lane < 16 && j < cc.len) {
                    const int k = j / ps;
                    in_page[3] = j - k * ps;
                    head[3] = cc.hk;
                    seq[3] = cc.b;
                    page[3] = p.block_table[static_cast<size_t>(cc.b) * p.max_pages + k];   // looked at when it is used
                }
                begins |= first_tile || cc.tile == 0 ? 8u : 0u;
                ends |= cc.tile + 1 == cc.tiles || cc.at + 1 == last ? 8u : 0u;
                first_tile = false;
                advance<S>(p, cc, row_blocks);
                ++tiles;
            }
            if (t < 3) continue;
            const int i = t - 3;
            if (i >= tiles) break;
            // in the order of their use: S is two tiles ahead of O
            if (begins & 1) {
                load(p.cache.k, 0, i);
                if (!(ends & 1) && ok) load(p.cache.k, 1, i + 1);
            }
            if (ok) load(p.cache.v, 0, -1);
            if (ok && !(ends & 3)) load(p.cache.k, 2, i + 2);
        }
        tc::cp_async_wait_all();   // nothing is in flight when the CTA ends
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------ the issuing thread
        if (lane == 0) {
            constexpr uint32_t id_s = tc::idesc_bf16(128, 128);
            constexpr uint32_t id_o = tc::idesc_f16(128, S::NV, 0, 1, 0) | (1u << 7) | (1u << 10);
            const uint32_t ring_lo = tc::smem_u32(smem) >> 4, q_lo = (tc::smem_u32(q_s) >> 4) + kDescLoK;
            int unit = 0, halves = 0, done = 0;   // done: tiles whose O has been issued
            uint32_t q_phase = 0;
            bool ok = true;
            // The first unit of the next half tile, when it has landed; the fence makes its copies visible to the tensor cores.
            // (A wait costs 230 cycles even where there is nothing to wait for: one for a half tile, not one for a unit.)
            auto landed = [&]() {
                ok = ok && stage_wait(sm.full + (halves & 15), (halves >> 4) & 1, &sm.abort);
                ++halves;
                const int u = unit;
                if ((unit += S::kCols) >= kUnits) unit -= kUnits;
                tc::fence_proxy_async();
                tc::fence_after_sync();
                return u;
            };
            auto issue_s = [&](int i) {   // of tile i, the next one
                const uint32_t d = t_s + (i & 1) * 128;
                int u = landed();
                if (!ok) return;
#pragma unroll
                for (int c = 0; c < S::kCols; ++c) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(d, q_lo + c * (16384 >> 4) + 2 * kk, ring_lo + u * (kUnit >> 4) + 2 * kk + kDescLoK, id_s, (c | kk) != 0);
                    tc::mma_commit(sm.empty + u);
                    if (++u == kUnits) u = 0;
                }
                tc::mma_commit(&sm.s_full[(i & 1)]);
            };
            // S is issued two tiles ahead of O, within a group: it runs while the threads compute, and they do not wait for O.
            bool first_of_group = true;
#pragma unroll 1
            while (cc.at < last && ok) {
                // tiles of the group in this CTA after this one
                const long long more = min(static_cast<long long>(cc.tiles - cc.tile), last - cc.at) - 1;
                const bool group_done = cc.tile + 1 == cc.tiles;
                if (first_of_group) {
                    ok = stage_wait(&sm.q_ready, q_phase, &sm.abort);
                    q_phase ^= 1;
                    issue_s(done);
                    if (more >= 1) issue_s(done + 1);
                }
                ok = ok && stage_wait(&sm.p_ready[(done & 1)], (done >> 1) & 1, &sm.abort);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t t_p = t_s + (done & 1) * 128;
                int u = landed();
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < D / S::NV; ++h) {
                    const uint32_t v_lo = ring_lo + u * (kUnit >> 4) + kDescLoN;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(t_o + h * S::NV, t_p + ks / 2 * 32 + q * 16 + ks % 2 * 8, v_lo + ks * (2048 >> 4), id_o,
                                   !first_of_group || (q | ks) != 0);
                    tc::mma_commit(sm.empty + u);
                    if (S::kPerV == 2) tc::mma_commit(sm.empty + u + 1);
                    if ((u += S::kPerV) == kUnits) u = 0;
                }
                tc::mma_commit(&sm.o_done);
                if (more >= 2) {   // into the place that O's product has read P from
                    ok = stage_wait(&sm.o_done, done & 1, &sm.abort);
                    tc::fence_after_sync();
                    issue_s(done + 2);
                }
                ++done;
                advance<S>(p, cc, row_blocks);
                first_of_group = group_done;
            }
            tc::mma_commit(&sm.drained);   // everything issued is through before the CTA ends
            tc::mbar_wait(&sm.drained, 0, kWaitLimit);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ the softmax warps
        const Split sp = split_of<S>(p);
        constexpr int kChunks = NR / 32;           // of 32 keys, a thread's share of a tile
        const uint32_t my_lanes = static_cast<uint32_t>(32 * warp) << 16;
        const int r = threadIdx.x % NR, key0 = threadIdx.x / NR * NR;   // this lane's row, its first key of a tile
        const uint32_t my_o = t_o + my_lanes;
        const float c = p.scale * kLog2e;
        float m = -INFINITY, base = 0.f, limit = -INFINITY, l = 0.f;
        // A wait of a softmax warp; what it gives up is told before the barrier at the group's end.
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool done = warp_wait(bar, parity, &sm.abort);
            if (!done) sm.stop = 1;
            return done;
        };
        bool fresh = true, first_seg = true, new_seq = cc.tile == 0 && cc.hk == 0 && cc.rb == 0;
        int count = 0;   // tiles of this CTA
        long long seg_first = cc.at;
        int half0 = 0;   // halves of the tiles of the CTA's groups before this one
#pragma unroll 1
        while (cc.at < last) {
            const int row0 = cc.rb * NR, rows = min(NR, R - row0);
            if (fresh) {
                const bf16* const q = static_cast<const bf16*>(p.q) + static_cast<long long>(cc.b) * p.K * p.ldq + static_cast<long long>(cc.hk) * p.G * D;
                for (int i = threadIdx.x; i < NR * D / 8; i += 128) {
                    const int qr = i / (D / 8), ch = i % (D / 8), row = row0 + qr, tok = token_of(p, row);
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (row < R) v = *reinterpret_cast<const uint4*>(q + tok * p.ldq + (row - tok * p.G) * D + ch * 8);
#pragma unroll
                    for (int x = 0; x < 128; x += NR)   // row x + qr has the swizzle of row qr
                        *reinterpret_cast<uint4*>(q_s + ch / 8 * 16384 + (x + qr) * 128 + ((ch & 7) ^ (qr & 7)) * 16) = v;
                }
                m = limit = -INFINITY;
                base = l = 0.f;
                tc::fence_proxy_async();
                tc::mbar_arrive(&sm.q_ready);
                if (new_seq && threadIdx.x == 0 && p.status) {
                    seq_keys(p, cc.b, &over);
                    if (over) atomicOr(p.status + cc.b, kKvBadIndex);
                }
            }
            if (wait(&sm.s_full[(count & 1)], (count >> 1) & 1)) {
                const uint32_t my_s = t_s + my_lanes + (count & 1) * 128;
                tc::fence_after_sync();
                // this row sees the keys of the tile before `sees` that are there
                const int sees = cc.len - p.K + token_of(p, row0 + r) + 1 - cc.tile * 128 - key0;
                uint32_t there[kChunks], all = 0xffffffffu;
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    there[i] = *reinterpret_cast<const uint32_t*>(&sm.valid[count & 15][key0 / 16 + 2 * i]);
                    all &= there[i];
                }
                const bool masked = all != 0xffffffffu || (cc.tile + 1) * 128 > cc.len - p.K + 1;   // the same for the warp
                // 32 scores in base 2
                auto scores = [&](int i, float (&s)[32]) {
                    tc::tmem_ld32(my_s + key0 + i * 32, s);
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[e] *= c;
                    if (masked) {
                        const int n = sees - i * 32;
                        const uint32_t w = n <= 0 ? 0u : n >= 32 ? there[i] : there[i] & ((1u << n) - 1u);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[e] = (w >> e) & 1 ? s[e] : -INFINITY;
                    }
                };
                float w[32], mx = -INFINITY;   // scores for the maximum, read again for the weights
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    scores(i, w);
#pragma unroll
                    for (int e = 0; e < 32; ++e) mx = fmaxf(mx, w[e]);
                }
                if (__any_sync(0xffffffffu, mx > limit)) {
                    // the tiles before have been added: O stands still
                    const bool through = fresh || wait(&sm.o_done, (count - 1) & 1);
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
                        for (int i = 0; i < D; i += 32) {
                            float v[32];
                            tc::tmem_ld32(my_o + i, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= f;
                            tc::tmem_st32(my_o + i, v);
                        }
                    }
                }
                // Weights: two bf16 parts, the second the rounding of what the first leaves (2^-17 together, below a bf16
                // result's own rounding), two keys a column: those of 32 keys take the columns of their scores.
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    scores(i, w);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        w[e] = ex2(w[e] - base);
                        l += w[e];
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float x[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint32_t u = StateIO<bf16>::pack(w[2 * e], w[2 * e + 1]);
                            if (q == 0) {
                                w[2 * e] -= __uint_as_float(u << 16);
                                w[2 * e + 1] -= __uint_as_float(u & 0xffff0000u);
                            }
                            x[e] = __uint_as_float(u);
                        }
                        tc::tmem_st16(my_s + key0 + i * 32 + q * 16, x);
                    }
                }
                if ((cc.tile + 1) * 128 > cc.len - p.K + 1) {
                    // Strays are taken out here and not by the loading warps, whose loop would grow (64 rows 179 us against 188).  The
                    // values have landed when their barrier says so, and the issuing thread waits for all lanes before it uses them.
                    const int i = static_cast<int>(cc.at - seg_first), n = static_cast<int>(min(static_cast<long long>(cc.tiles - cc.tile + i), last - seg_first));
                    const int h = half0 + 2 * i + (i + 1 < n ? 2 : 1);   // the keys of the next tile come before these values, but for the last one's
                    const int k0 = max(0, cc.len - p.K + 1 - cc.tile * 128), k1 = min(128, cc.len - cc.tile * 128);
                    if (k0 < k1 && wait(sm.full + (h & 15), (h >> 4) & 1)) {
                        const int u0 = h * S::kCols % kUnits;
                        bool found = false;
#pragma unroll 1
                        for (int x = threadIdx.x; x < (k1 - k0) * (D / 8); x += 128) {
                            const int ch = x % (D / 8);
                            found |= take_strays<bf16>(smem + (u0 + ch / 8) % kUnits * kUnit + (k0 + x / (D / 8)) * 128 + ch % 8 * 16);
                        }
                        if (found) sm.strays = 1;
                        tc::fence_proxy_async();
                    }
                }
                if (NR < 128) {   // zeros for the keys that are other lanes'
                    float z[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) z[e] = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i / kChunks != key0 / NR)
#pragma unroll
                            for (int q = 0; q < 2; ++q) tc::tmem_st16(my_s + i * 32 + q * 16, z);
                }
                tc::tmem_wait_st();
                // Before the last tile of a group goes off: the one before it has been added, so that the wait for the last
                // one cannot take the wrong phase for its own.
                if (!fresh && (cc.tile + 1 == cc.tiles || cc.at + 1 == last)) wait(&sm.o_done, (count - 1) & 1);
                tc::fence_before_sync();
                tc::mbar_arrive(&sm.p_ready[(count & 1)]);
            }
            ++count;
            const bool group_done = cc.tile + 1 == cc.tiles;
            if (group_done || cc.at + 1 == last) {
                const long long g_first = cc.at - cc.tile, g_last = g_first + cc.tiles;   // the group's tiles
                const bool whole = seg_first == g_first && cc.at + 1 == g_last;
                const int part = 2 * blockIdx.x + (first_seg ? 0 : 1);
                wait(&sm.o_done, (count - 1) & 1);
                tc::fence_after_sync();
                if (p.test_stall && warp == 3 && !stage_wait(&sm.never, 0, &sm.abort, 256)) sm.stop = 1;
                sm.ml[threadIdx.x] = make_float2(m, l);
                sync_computing<S>();
                if (sm.stop) {   // a wait gave up: nothing of this group is written
                    if (threadIdx.x == 0 && p.status) atomicOr(p.status + cc.b, 16);
                } else {
                    // the copies of a row meet in the queries' place, a quarter of the channels at a time
                    constexpr int CH = D / 4, kPitch = CH + 4;
                    float* const buf = reinterpret_cast<float*>(q_s);
                    float mm = -INFINITY, ll = 0.f;
#pragma unroll
                    for (int x = 0; x < 128; x += NR) mm = fmaxf(mm, sm.ml[x + r].x);
                    const float b0 = mm == -INFINITY ? 0.f : mm, f = ex2(m - b0);
#pragma unroll
                    for (int x = 0; x < 128; x += NR) ll = fmaf(ex2(sm.ml[x + r].x - b0), sm.ml[x + r].y, ll);
                    if (threadIdx.x < NR) {
                        sm.f[r] = ll == 0.f ? 0.f : 1.0f / ll;
                        if (!whole) sp.ml[static_cast<size_t>(part) * NR + r] = make_float2(mm, ll);
                    }
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
#pragma unroll 1
                        for (int c0 = 0; c0 < CH; c0 += 16) {
                            float v[16];
                            tc::tmem_ld16(my_o + h * CH + c0, v);
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                *reinterpret_cast<float4*>(buf + threadIdx.x * kPitch + c0 + i) = make_float4(f * v[i], f * v[i + 1], f * v[i + 2], f * v[i + 3]);
                        }
                        sync_computing<S>();
#pragma unroll 1
                        for (int i = threadIdx.x; i < rows * (CH / 4); i += 128) {
                            const int row = i / (CH / 4), ch = i % (CH / 4) * 4;
                            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                            for (int x = 0; x < 128; x += NR) {
                                const float4 v = *reinterpret_cast<const float4*>(buf + (x + row) * kPitch + ch);
                                y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
                            }
                            if (whole) put<bf16, D>(p, true, cc.b, cc.hk, row0 + row, h * CH + ch, times(y, sm.f[row]));
                            else *reinterpret_cast<float4*>(sp.o + (static_cast<size_t>(part) * NR + row) * D + h * CH + ch) = y;
                        }
                        sync_computing<S>();
                    }
                    if (!whole) join_group<S>(p, true, sp, sh, cc, g_first, g_last, rows, buf, &sm.strays, &sm.flag);
                    if (whole ? sm.strays : sm.flag == (kFinished | kStrays)) add_strays<S>(p, cc.b, cc.hk, row0, cc.len, rows);
                }
                first_seg = false;
            }
            const int b = cc.b;
            advance<S>(p, cc, row_blocks);
            fresh = group_done;
            if (group_done) {
                half0 = 2 * count;
                new_seq = cc.b != b;
                seg_first = cc.at;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kIssuer) tc::tmem_dealloc(sm.tmem, 512);
}

template <int D, int NR>
cudaError_t launch_shape(const AttnParams& p, int sms, cudaStream_t stream) {
    using S = TcShape<D, NR>;
    const cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_tc_kernel<S>, dim3(sms), dim3(S::kAll), S::kSmem, stream, p);
}

template <int D>
cudaError_t by_rows(const AttnParams& p, int sms, cudaStream_t stream) {
    return block_rows(p.G * p.K, true) == 64 ? launch_shape<D, 64>(p, sms, stream) : launch_shape<D, 128>(p, sms, stream);
}

}  // namespace

cudaError_t launch_tc(const AttnParams& p, int head_dim, int sms, cudaStream_t stream) {
    if (head_dim == 64) return by_rows<64>(p, sms, stream);
    if (head_dim == 128) return by_rows<128>(p, sms, stream);
    return by_rows<256>(p, sms, stream);
}

}  // namespace attn
}  // namespace gdn
