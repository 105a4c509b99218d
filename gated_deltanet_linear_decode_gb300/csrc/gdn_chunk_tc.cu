// gdn_chunk_tc.cu -- gdn_attn_chunk over a bf16 cache: products on the 5th-generation tensor cores.
//
// A worker is a pair of CTAs (a cluster, two SMs) that work on one unit of up to 256 rows: S = Q . K^T and O += P . V with M = 256,
// 128 rows in each CTA's tensor memory.  The pair shares every tile of 128 keys: of the keys each CTA has 64 in its shared memory,
// of the values half of the channels, and the tensor cores read both.  So a key and a value come from L2 once for 256 rows
// (at d = 256 a tile's products take 2,048 cycles and its copies 32 bytes a cycle of every SM; with 128 rows a CTA it were 64).
//
// Roles of a CTA's 12 warps:
//   0-7   softmax, two groups that take turns: a thread has one row (tensor-memory lane) of every other tile.  A tile's maximum needs
//         the base that the other group had for the tile before; the weights' powers of one run beside the maxima of the next.
//         The result is rescaled only when a row's maximum has risen by more than 2^kSlack.
//   8     copies keys by TMA, from a tensor map that serves any strides; each lane looks up its keys' pages and copies them.  Keys
//         past the end and pages outside the cache are coordinates outside the map, which read as zeros
//   10    copies values
//   11    copies queries (with the keys' copies a part's first keys had to wait for the last part's queries to be done with, and
//         came 2 us late)
//   9     one thread of the first CTA: issues the products
//
// Bound by the products where units are long: 8,192 tokens, 24/4 heads of 256, 539 us, 1.53 PFLOP/s, 80% of what a large matrix product
// reaches (in a run of 20; after half a second of them the power limit has the clock at 1.85 GHz, and they take 577, 1.43
// PFLOP/s); a tile of 128 keys takes some 2,400 cycles.  Elsewhere by a part's begin and end: 8 ragged prompts of up to 4,096
// tokens, 64/8 heads of 128, 1,161 us, 1.02 PFLOP/s; tiles take 0.82 us each, the rest of a part 5 us.  And where calls are small by
// a chain of latencies: 37 tokens behind 740, 16/2 heads of 256, 27 us.
//
// S has two or three places, as the tensor memory allows, so that the softmax of tiles runs beside the products of others.  The
// weights take the place of scores that have been read; the S that comes into their place waits for the product with them.
//
// For a bf16 result a weight is rounded to bf16 (2^-8 of it at most): with a second part for what the rounding leaves, as
// gdn_attn_decode has it, which is bound by memory, the product with the values would take twice the time, half again as much
// for the whole.
//
// For an fp32 result a weight is three bf16 parts, which together have all its bits.  They take 192 columns a place of S, and a sum
// over many tiles in tensor memory would be cut at every product (2^-24 or so of it, always towards zero: 1e-4 after 32,768 keys).
// So a unit has 64 channels of the values -- a head of 256 is four units, which compute the same weights -- and a tile's O is
// its own; a thread adds it to its row's 64 sums in registers, each group those of its tiles, relative to a base of its own.
// (Heads of 64, 64 tokens each of 16 sequences of up to 4,096: 42 us; in fp32 on the CUDA cores 186.)
#include <cuda.h>

#include "gdn_chunk.cuh"
#include "gdn_chunk_strays.h"
#include "gdn_internal.h"

namespace gdn {
namespace chunk {

namespace {

using bf16 = __nv_bfloat16;
using attn::kWaitLimit;
using tc::smem_u32;
constexpr int kDrainLimit = 1 << 14;   // polls for what is in flight at the end
constexpr int kDrainCycles = 1 << 17;  // and a time for it after a give-up
constexpr int kMinShare = 512;        // keys of a worker, at least
constexpr int kJoin = 8;              // parts that are joined at a time, of units with many of them
constexpr unsigned kStrayPart = 1 << 16;   // in a counter of parts
static_assert(kMaxWorkers < static_cast<int>(kStrayPart), "parts of a unit");
constexpr float kSlack = 8.0f;   // how far a score may pass its row's base
constexpr int kRows = 256, kKeys = 128, kThreads = 384, kSoft = 256;
constexpr int kRest = 3 * 1024;   // bytes of shared memory beside queries, keys and values

template <int D_, bool kF32_>
struct Tc {
    static constexpr int D = D_;
    static constexpr bool kF32 = kF32_;                       // the result
    static constexpr int DV = kF32 ? 64 : D, kSlices = D / DV;   // channels of the values that a unit has
    static constexpr int NS = kF32 || D == 256 ? 2 : 3;       // places of S, and of the weights that take a part of it
    static constexpr int kVCh = kF32 ? 32 : D == 256 ? 128 : 64;   // channels of a CTA's values (bf16 results of heads of 64: all of them, in both)
    static constexpr int kBlock = kF32 ? 32 : 64;             // channels of a row of a box of values
    static constexpr int kStageK = kKeys * D, kStageV = kKeys * 2 * kVCh;   // bytes: 64 keys, 128 keys' values
    static constexpr int RK = kF32 ? (D == 256 ? 4 : 6) : D == 256 ? 2 : D == 128 ? 5 : 6;
    static constexpr int RV = kF32 ? (D == 256 ? 3 : 6) : D == 256 ? 3 : D == 128 ? 5 : 6;
    static constexpr int kQ = 128 * D * 2;
    static constexpr int kSmem = kQ + RK * kStageK + RV * kStageV + kRest;
    // tensor memory: O (of fp32 results two, by tile mod 2), the places; in a place of fp32 results S is behind 64 columns
    static constexpr int kO = 0, kS = kF32 ? 128 : D == 256 ? 256 : 128;
    static constexpr int kPlace = kF32 ? 192 : 128, kScores = kF32 ? 64 : 0;
    static constexpr int kCost = D == 256 ? 768 : 512;        // of a unit: its begin and end take as long as so many keys
    static constexpr bool kGates = DV <= 128;                 // a row's gates are loaded before its sums are there (ragged prompts 1,221 -> 1,158 us)
    static_assert(kSmem <= 232448 && kS + NS * kPlace <= 512, "shape");
};

struct Smem {
    float base[2][128];               // of a row's weights, by tile mod 2
    float sum[2][128];                // at a part's end the groups' shares, relative to their base
    uint32_t valid[16][4];            // keys of a tile that are there, by tile mod 16
    uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
    uint64_t q_full, q_empty, s_full[3], p_ready[3], pv_done[3], drained, never;   // by place of S
    uint64_t v_told[6];               // by tile mod 6: one of them is always the same group's, and not passed twice before it has looked
    union {
        PlanSmem plan;                // until the roles begin
        struct {
            int tiles[16];            // of a part that has some, by its number mod 16; 0: there is none
            Part next;                // at a part's end what comes then, if there is more
            int more;
        } way;
    };
    uint32_t tmem;
    int last, stop;                   // last: this CTA finishes the part's rows; stop: a softmax warp has seen abort
    Strays strays;
    volatile int abort;
};
static_assert(sizeof(Smem) <= kRest, "fits");

// ---------------------------------------------------------------- the pair
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// An arrival at the CTA `rank`'s barrier.  It orders what this CTA sees; what the tensor cores see of registers and shared memory
// is ordered by their own fences before it.  (With .release.cluster, which waits until the whole GPU could see this thread's
// writes, an arrival took 1,280 cycles.)
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_cta(smem_u32(bar), rank)) : "memory");
}

// A box of the map at (0, c1, .. c4) into this CTA's shared memory, its bytes counted by the first CTA's barrier (at cluster address
// `bar`).
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int c1, int c2, int c3, int c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_q(uint32_t dst, const CUtensorMap* map, int ch, int head, int token, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ch), "r"(head), "r"(token), "r"(bar)
        : "memory");
}

// Wait for phase `parity` of `bar`.  A wait that gives up, or finds that another of the CTA has, returns as well: who goes on to
// use what it waited for looks at `abort` first.  (Made like this a wait for what is there takes 73 cycles; with an answer
// that the caller branches on 184, by one lane and a shuffle 290.)
__device__ __forceinline__ bool is_there(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}
__device__ __noinline__ void long_wait(uint32_t bar, uint32_t parity, volatile int* abort, int limit) {
#pragma unroll 1
    for (int it = 0; it < limit; ++it) {
        if (is_there(bar, parity) || *abort) return;
    }
    *abort = 1;
}
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (!is_there(smem_u32(bar), parity)) long_wait(smem_u32(bar), parity, abort, kWaitLimit);
}

// One lane of a converged warp (the compiler knows that it is one).
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Arrive at `bar` in both CTAs when every product issued so far is done.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}

// Upper word of the shared-memory descriptors: 128-byte swizzle, 8-row groups 1024 bytes apart.  The lower word is the address / 16
// and, for values, how far the next 64 channels are.
constexpr uint32_t kDesc128 = (1024u >> 4) | (1u << 14) | (2u << 29);
// 64-byte swizzle, for values of 32 channels.
constexpr uint32_t kDesc64 = (512u >> 4) | (1u << 14) | (4u << 29);

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc),
        "r"(static_cast<uint32_t>(add)), "n"(kDesc128), "r"(b_hi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(idesc),
        "r"(static_cast<uint32_t>(add)), "r"(b_hi));
}

// 32 consecutive columns of this thread's lane, to be waited for; 32 words to such columns.
__device__ __forceinline__ void tmem_ask32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// The wait names the registers, so that nothing that uses them moves ahead of it.
__device__ __forceinline__ void tmem_wait_for(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
          "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
          "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
          "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
        :: "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}

// The boxes that are copied.  A stage holds groups of 8 tokens, of each its blocks of 64 channels, of each 8 rows of 128 bytes: with
// that, keys and values have one distance from a group to the next and one from a block to the next, as the tensor cores want it.
// Where pages are a multiple of 8 tokens and follow one another, or the heads of one do, the map is (64 channels, 8 tokens, block,
// group of 8, page and head) and a box is all the blocks of as many tokens as always lie in one page.  (A copy takes its thread
// 150 cycles: pages of 16 by boxes of 8 keys, or 16 tokens' one block, were bound by that.)  Otherwise it is (64 channels, token,
// block, head, page) and a box one block of 1 to 8 tokens, which the copies then bound: 4 x 1,024 tokens behind 1,024, bf16 results, heads
// of 256, 128, 64: pages of 16 106, 121, 106 us, of 100 (boxes of 4) 171, 196, 158, of 1 and 5 (boxes of 1) 469, 488, 456.
struct Boxes {
    int tokens;        // of a box
    int whole;         // the first kind of map
    int group, head;   // what a page adds to the coordinates of group and head there
};
struct Division {   // by the page size, of 31 bits: x -> x * mul >> 32 >> shift, or x where mul is 0
    uint32_t mul, shift;
    __device__ __forceinline__ int of(int x) const { return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(x), mul) >> shift) : x; }
};

// 16 bf16 of a row: one access of 32 bytes where rows begin on such, else two of 16.  (A part's end is bound by these: each
// of a warp's lanes has another row, and an access of a lane takes its turn whatever its size.)
__device__ __forceinline__ void load16(const void* at, bool whole, uint32_t (&v)[8]) {
    if (whole) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "l"(at));
    } else {
        const uint4 a = static_cast<const uint4*>(at)[0], b = static_cast<const uint4*>(at)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}
__device__ __forceinline__ void store16(void* at, bool whole, const uint32_t (&v)[8]) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                     "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
    } else {
        static_cast<uint4*>(at)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4*>(at)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
__device__ __forceinline__ bool on32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// A walk over the tiles of a worker's parts.  The part lies in memory (to_next_part is a call), what every tile asks for does not.
struct Walk {
    Part& c;
    int t, t0, t1;
    bool more;
    __device__ __forceinline__ Walk(Part& first, const ChunkParams& p, const Line& ln, const Share& sh) : c(first), more(true) { settle(p, ln, sh); }
    __device__ __forceinline__ void settle(const ChunkParams& p, const Line& ln, const Share& sh) {   // past parts without tiles
        while (more && c.t0 >= c.t1) more = to_next_part(p, ln, sh, c);
        t = t0 = c.t0;
        t1 = c.t1;
    }
    __device__ __forceinline__ void next(const ChunkParams& p, const Line& ln, const Share& sh) {
        if (++t < t1) return;
        more = to_next_part(p, ln, sh, c);
        settle(p, ln, sh);
    }
    __device__ __forceinline__ bool first() const { return t == t0; }
    __device__ __forceinline__ bool last() const { return t + 1 == t1; }
};

// A part in the workspace: of each CTA by 8 channels its 128 rows' -- what a warp's lanes, of a row each, write and read is
// consecutive.  (By rows a part of 128 KB took 4.3 us to write, and six of them 28 to join.)
__device__ __forceinline__ uint32_t part_at(int row, int ch) { return static_cast<uint32_t>((ch >> 3) * 128 + row) * 8 + (ch & 7); }

// All softmax warps.
__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 9, %0;" ::"n"(kSoft) : "memory"); }

// The strays of a unit's late keys (gdn_attn.cuh; those that its first row does not see) are added to the results of the rows that
// see them: this CTA's rows, whose first token is the unit's token cta_tok.  By whoever finishes the rows, behind the join of a unit's
// parts, and not to a part: its weight in the join may be zero, in a row that sees none of its keys or far larger scores
// elsewhere, and would make NaN of an infinity.  A thread has 4 channels of a run of consecutive tokens: of the keys before the run it
// needs the sum, then a token sees one key more than the token before.  Loads of several keys go out together: each is a table entry, then a
// value.  (8,192 tokens, 4/4 heads of 256, 116 us; with one NaN token, in the last unit of each head, 206, and 2,147 where each row's keys
// were walked one after another; with NaN in all tokens 594 and 10,418.)  A call, for the size of the code around it.
template <class S>
__device__ __noinline__ void add_strays(const ChunkParams& p, const Part& c, int tok0, int cta_tok, int rows) {
    constexpr int DV = S::DV, kQuads = DV / 4, kRuns = kSoft / kQuads, kAt = 4;
    const int hk = c.hk / S::kSlices, ch = c.hk % S::kSlices * DV + static_cast<int>(threadIdx.x) % kQuads * 4;
    const int tokens = rows / p.G, each = (tokens + kRuns - 1) / kRuns;
    const int first = static_cast<int>(threadIdx.x) / kQuads * each, last = min(tokens, first + each);
    if (first >= last) return;
    const int seen = c.r.len - c.r.n + tok0;   // the last key that the unit's first token sees; below 0: none
    const int from = max(0, seen + 1), mine = seen + cta_tok;
    auto strays_of = [&](int j) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const int k = j / p.cache.page_size, page = p.block_table[static_cast<size_t>(c.b) * p.max_pages + k];
        if (page >= 0 && page < p.cache.num_pages)
            v = StateIO<bf16>::ld(static_cast<const bf16*>(p.cache.v) + page * p.cache.page_stride +
                                  (j - k * p.cache.page_size) * p.cache.token_stride + hk * p.cache.head_stride + ch);
        return make_float4(isfinite(v.x) ? 0.f : v.x, isfinite(v.y) ? 0.f : v.y, isfinite(v.z) ? 0.f : v.z, isfinite(v.w) ? 0.f : v.w);
    };
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float4 v) { y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w); };
#pragma unroll 8
    for (int j = from; j < mine + first; ++j) add(strays_of(j));
#pragma unroll 1
    for (int i0 = first; i0 < last; i0 += kAt) {
        float4 v[kAt];
#pragma unroll
        for (int u = 0; u < kAt; ++u) v[u] = i0 + u < last && mine + i0 + u >= from ? strays_of(mine + i0 + u) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int u = 0; u < kAt && i0 + u < last; ++u) {
            add(u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3]);
            if (y.x == 0.f && y.y == 0.f && y.z == 0.f && y.w == 0.f) continue;
            for (int g = 0; g < p.G; ++g) put<bf16, S::D, true>(p, !S::kF32, static_cast<long long>(c.r.row0) + tok0 + cta_tok + i0 + u, hk * p.G + g, ch, y);
        }
    }
}

// The join of n parts of a few rows, by items of a row's 4 channels: eight parts' loads together.  A call, for the size of the
// code around it.
template <class S>
__device__ __noinline__ void join_few(const ChunkParams& p, const Part& c, const Parts<kRows, S::DV>& parts, int w0, int n, int tok0, int cta_tok, int rows, int row0) {
    constexpr int kAt = 8, D = S::DV;
    auto row_of = [&](int k) { return (k == 0 ? 2 * static_cast<size_t>(w0) + 1 : 2 * static_cast<size_t>(w0 + k)) * kRows + row0; };
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (D / 4); i += kSoft) {
        const int r = i / 2 % rows, ch = i / 2 / rows * 8 + i % 2 * 4, in = r / p.G;
        float mm = -INFINITY, ll = 0.f;
#pragma unroll 8
        for (int k = 0; k < n; ++k) mm = fmaxf(mm, __ldcg(&parts.ml[row_of(k) + r].x));
        mm = mm == -INFINITY ? 0.f : mm;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = 0; k0 < n; k0 += kAt) {   // past the last part it again, without weight
            float2 z[kAt];
            float4 x[kAt];
#pragma unroll
            for (int v = 0; v < kAt; ++v) {
                const size_t at = row_of(min(k0 + v, n - 1));
                z[v] = __ldcg(parts.ml + at + r);
                x[v] = __ldcg(reinterpret_cast<const float4*>(parts.o + at * D + part_at(r, ch)));
            }
#pragma unroll
            for (int v = 0; v < kAt; ++v) {
                if (k0 + v >= n) break;
                const float f = ex2(z[v].x - mm);
                ll = fmaf(f, z[v].y, ll);
                y = make_float4(fmaf(f, x[v].x, y.x), fmaf(f, x[v].y, y.y), fmaf(f, x[v].z, y.z), fmaf(f, x[v].w, y.w));
            }
        }
        put<bf16, S::D>(p, !S::kF32, static_cast<long long>(c.r.row0) + tok0 + cta_tok + in, c.hk / S::kSlices * p.G + r - in * p.G, c.hk % S::kSlices * D + ch,
                        attn::times(y, ll == 0.f ? 0.f : 1.0f / ll));
    }
}

// A group's warp lets the other group's warp of the same rows have its base (barriers 1 to 8).
__device__ __forceinline__ void give_base(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(1 + id) : "memory"); }
__device__ __forceinline__ void take_base(int id) { asm volatile("bar.sync %0, 64;" ::"r"(1 + id) : "memory"); }

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                    const __grid_constant__ CUtensorMap q_map, const Boxes kb, const Boxes vb, const Division by_page) {
    constexpr int D = S::D, DV = S::DV, NS = S::NS, RK = S::RK, RV = S::RV;
    constexpr int kKBlocks = D / 64, kVBlocks = S::kVCh / S::kBlock;   // blocks of channels in a CTA's stages
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const q_s = smem;
    uint8_t* const k_s = q_s + S::kQ;
    uint8_t* const v_s = k_s + RK * S::kStageK;
    Smem& sm = *reinterpret_cast<Smem*>(v_s + RV * S::kStageV);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_ctarank();
    const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);
    // What lands is counted by the first CTA's barriers, with an arrival of each CTA.
    if (threadIdx.x < 8) {
        tc::mbar_init(sm.k_full + threadIdx.x, 2);
        tc::mbar_init(sm.v_full + threadIdx.x, 2);
        tc::mbar_init(sm.k_empty + threadIdx.x, 1);
        tc::mbar_init(sm.v_empty + threadIdx.x, 1);
    }
    if (threadIdx.x == 0) {
        tc::mbar_init(&sm.q_full, 2);
        tc::mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(sm.s_full + i, 1);
            tc::mbar_init(sm.p_ready + i, 8);   // a tile's softmax warps of both CTAs
            tc::mbar_init(sm.pv_done + i, 1);
        }
        for (int i = 0; i < 6; ++i) tc::mbar_init(sm.v_told + i, 1);
        tc::mbar_init(&sm.drained, 1);
        tc::mbar_init(&sm.never, 1);
        sm.strays.clear();
        sm.abort = sm.stop = (smem_u32(smem) & 1023) != 0;   // the swizzle goes by address bits 7-9
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");   // the barriers are there before asynchronous arrivals on them
    const int cta_tokens = 128 / p.G, cta_rows = cta_tokens * p.G;   // of a unit, in each CTA
    const Line ln{2 * cta_tokens, 7, S::kCost};
    static_assert(kKeys == 1 << 7, "keys of a tile");
    Share sh;
    Part c;
    if (!my_share(p, ln, worker, workers, kMinShare, sm.plan, sh, c)) return;   // both CTAs of a pair, or neither
    // rows past cta_rows, which no copy writes
    for (int i = threadIdx.x; i < (128 - cta_rows) * (D / 8); i += kThreads)
        *reinterpret_cast<uint4*>(q_s + i / ((128 - cta_rows) * 8) * 16384 + cta_rows * 128 + i % ((128 - cta_rows) * 8) * 16) = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async();
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync_all();   // the other CTA's barriers are there too
    tc::fence_after_sync();
    const uint32_t t_o = sm.tmem + S::kO, t_s = sm.tmem + S::kS;

    // The bytes of both CTAs are expected by the first one, and the second one arrives.
    auto announce = [&](uint64_t* bar, uint32_t bytes) {
        if (lane == 0) {
            if (rank == 0) tc::mbar_expect_tx(bar, bytes);
            else arrive_at(bar, 0);
        }
        __syncwarp();
        return in_cta(smem_u32(bar), 0);
    };
    auto rest = [&]() {   // after a give-up: more time than any copy takes
        if (!sm.abort) return;
        const long long from = clock64();
        while (clock64() - from < kDrainCycles) {
        }
    };
    if (warp == 8 || warp == 10) {
        // ------------------------------------------------------------ copies: warp 8 keys, warp 10 values
        Walk w(c, p, ln, sh);
        const bool keys = warp == 8;
        const Boxes bx = keys ? kb : vb;
        const int ps = p.cache.page_size, groups = kKeys / bx.tokens;
        // Lane l has the tile's groups of bx.tokens keys l + 32 k, [0] of the tile to be copied, [1] of the one being looked up.
        constexpr int kPer = 4;
        int page[2][kPer] = {}, in[2][kPer] = {}, head[2] = {}, slice[2] = {}, seq[2] = {}, tiles[2] = {};   // in -1: no key; seq -1: no tile
        int parts = 0, part_seq = 0, part_head = 0, part_slice = 0;
        int end = 0;               // keys from `end` on are nobody's
        const int* table = nullptr;   // the sequence's pages
        auto look_up = [&](int a) {
            seq[a] = -1;
            if (!w.more) return;
            if (w.first()) {
                part_seq = c.b;
                part_head = c.hk / S::kSlices;
                part_slice = c.hk % S::kSlices;
                end = c.seen;
                table = p.block_table + static_cast<size_t>(c.b) * p.max_pages;
            }
            seq[a] = part_seq;
            head[a] = part_head;
            slice[a] = part_slice;
            tiles[a] = w.first() ? w.t1 - w.t0 : 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (k > 0 && groups <= 32 * k) break;
                const int i = lane + 32 * k, j = w.t * kKeys + i * bx.tokens;
                in[a][k] = page[a][k] = -1;
                if (i < groups && j < end) {
                    const int x = by_page.of(j);
                    in[a][k] = j - x * ps;
                    page[a][k] = table[x];   // looked at when it is used
                }
            }
            w.next(p, ln, sh);
        };
        // copies of the tile at [0]: boxes [g0, g0 + n), all blocks from `block` on, by the lanes that have them
        const int row_bytes = keys ? 128 : 2 * S::kBlock;
        auto copy = [&](uint32_t stage, const CUtensorMap* map, int g0, int n, int block, int blocks, uint32_t bar) {
#pragma unroll 1
            for (int k = g0 >> 5; k <= (g0 + n - 1) >> 5; ++k) {
                const int pg = k == 0 ? page[0][0] : k == 1 ? page[0][1] : k == 2 ? page[0][2] : page[0][3];
                const int tk = max(k == 0 ? in[0][0] : k == 1 ? in[0][1] : k == 2 ? in[0][2] : in[0][3], 0);
                const int r = lane + 32 * k - g0, row = r * bx.tokens;
                uint32_t dst = stage + (row >> 3) * blocks * 8 * row_bytes + (row & 7) * row_bytes;
                if (r >= 0 && r < n) {
                    if (bx.whole) {
                        const bool there = pg >= 0 && pg < p.cache.num_pages;   // (the coordinates of another would be some other's)
                        tma_load(dst, map, 0, block, there ? pg * bx.group + (tk >> 3) : 0, there ? pg * bx.head + head[0] : -1, bar);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < blocks; ++c, dst += 8 * row_bytes) tma_load(dst, map, tk, block + c, head[0], pg, bar);
                    }
                }
                __syncwarp();
            }
        };
        int n = -1;   // tiles copied
#pragma unroll 1
        for (;; ++n) {
            head[0] = head[1];
            slice[0] = slice[1];
            seq[0] = seq[1];
            tiles[0] = tiles[1];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                page[0][k] = page[1][k];
                in[0][k] = in[1][k];
            }
            if (n >= 0 && seq[0] < 0) break;
            look_up(1);
            if (n < 0) continue;
            if (keys) {
                if (n >= RK) wait_for(sm.k_empty + n % RK, (n / RK - 1) & 1, &sm.abort);
                if (sm.abort) break;
                if (tiles[0] > 0) {   // a part's first
                    if (lane == 0) sm.way.tiles[parts & 15] = tiles[0];
                    ++parts;
                }
                if (lane < 4) sm.valid[n & 15][lane] = 0xffffffffu;
                bool bad = false;
#pragma unroll
                for (int k = 0; k < kPer; ++k) bad |= in[0][k] >= 0 && (page[0][k] < 0 || page[0][k] >= p.cache.num_pages);
                if (__any_sync(0xffffffffu, bad)) {
                    if (bad && p.status) atomicOr(p.status + seq[0], kKvBadIndex);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kPer; ++k)
                        if (in[0][k] >= 0 && (page[0][k] < 0 || page[0][k] >= p.cache.num_pages))
                            for (int key = (lane + 32 * k) * bx.tokens; key < (lane + 32 * k + 1) * bx.tokens; ++key)
                                atomicAnd(&sm.valid[n & 15][key >> 5], ~(1u << (key & 31)));
                }
                __syncwarp();
            } else {
                if (n >= RV) wait_for(sm.v_empty + n % RV, (n / RV - 1) & 1, &sm.abort);
                if (sm.abort) break;
            }
            const uint32_t bar = announce(keys ? sm.k_full + n % RK : sm.v_full + n % RV, keys ? 2 * S::kStageK : 2 * S::kStageV);
            copy(keys ? smem_u32(k_s) + n % RK * S::kStageK : smem_u32(v_s) + n % RV * S::kStageV, keys ? &k_map : &v_map,
                 keys ? static_cast<int>(rank) * groups / 2 : 0, keys ? groups / 2 : groups, keys ? 0 : S::kF32 ? 2 * slice[0] + static_cast<int>(rank) : D > 64 ? static_cast<int>(rank) * kVBlocks : 0,
                 keys ? kKBlocks : kVBlocks, bar);
        }
        int landed = max(0, n - (keys ? RK : RV));   // tiles before this one have been used
        if (keys && !sm.abort) {   // the products' warp learns that there are no more
            if (n >= RK) wait_for(sm.k_empty + n % RK, (n / RK - 1) & 1, &sm.abort);
            if (lane == 0) sm.way.tiles[parts & 15] = 0;
            announce(sm.k_full + n % RK, 0);
            landed = max(0, n + 1 - RK);
        }
        // Nothing is in flight when the pair ends: the last copies of every stage have landed.  After a give-up the two CTAs may have
        // stopped at different tiles, and no barrier tells of those that only one has copied.
        if (rank == 0) {
            const int r = keys ? RK : RV;
            for (int i = landed; i < n; ++i) tc::mbar_wait((keys ? sm.k_full : sm.v_full) + i % r, (i / r) & 1, kDrainLimit);
        }
        rest();
    } else if (warp == 11) {
        // ------------------------------------------------------------ queries
        int n = 0, before = 0;   // parts with tiles, tiles of the last one
        for (bool more = true; more; more = to_next_part(p, ln, sh, c)) {
            if (c.t0 >= c.t1) continue;
            if (n > 0) {   // for all of the last part: with a limit more for every 32,768 tiles, which take some 40 ms
                for (int i = 0; i < before >> 15; ++i)
                    for (int it = 0; it < kWaitLimit && !is_there(smem_u32(&sm.q_empty), (n - 1) & 1) && !sm.abort; ++it) {
                    }
                wait_for(&sm.q_empty, (n - 1) & 1, &sm.abort);
            }
            if (sm.abort) break;
            before = c.t1 - c.t0;
            const uint32_t bar = announce(&sm.q_full, 2 * cta_rows * D * 2);
            if (elected()) {
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load_q(smem_u32(q_s) + x * 16384, &q_map, x * 64, c.hk / S::kSlices * p.G, c.r.row0 + c.i * ln.tokens + static_cast<int>(rank) * cta_tokens, bar);
            }
            __syncwarp();
            ++n;
        }
        if (rank == 0 && n > 0) tc::mbar_wait(&sm.q_full, (n - 1) & 1, kDrainLimit);
        rest();
    } else if (warp == 9) {
        if (rank == 0) {
            // -------------------------------------------------------- products
            // (How many tiles a part has the keys' copier tells: the way to the next part, in code that is not at hand then, takes 2 us.)
            int nq = 0, units = 0, left = 0;   // S issued, parts begun, tiles of the newest one to come
            bool end = false;
            uint32_t firsts = 0;     // by tile mod 32: the first of a part
            constexpr uint32_t id_s = tc::idesc_bf16(256, 128);
            constexpr uint32_t id_o = tc::idesc_f16(256, 2 * S::kVCh, 0, 1, 0) | (1u << 7) | (1u << 10);
            const uint32_t q_lo = (smem_u32(q_s) >> 4) + (1u << 16), k_lo = (smem_u32(k_s) >> 4) + (1u << 16);
            // from one group of 8 to the next; from one block of 64 channels to the next, 1024 bytes
            constexpr uint32_t k_hi = (kDesc128 & ~0x3FFFu) | (kKBlocks * 1024 >> 4), v_hi = S::kF32 ? kDesc64 : (kDesc128 & ~0x3FFFu) | (kVBlocks * 1024 >> 4);
            const uint32_t v_lo = (smem_u32(v_s) >> 4) + ((1024u >> 4) << 16);
            auto issue_s = [&]() {   // of tile number nq, whose operands have landed
                const uint32_t d = t_s + nq % NS * S::kPlace + S::kScores, b = k_lo + nq % RK * (S::kStageK >> 4);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(d, q_lo + c * (16384 >> 4) + 2 * kk, b + c * (1024 >> 4) + 2 * kk, k_hi, id_s, (c | kk) != 0);
                commit_both(sm.s_full + nq % NS);
                commit_both(sm.k_empty + nq % RK);
                if (left == 1) commit_both(&sm.q_empty);
            };
            auto issue_o = [&](int g) {
                const uint32_t a = t_s + g % NS * S::kPlace, b = v_lo + g % RV * (S::kStageV >> 4);
                if constexpr (S::kF32) {   // a tile's own O, of the weights' smallest parts first
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(t_o + (g & 1) * 64, a + (part == 0 ? ks * 8 : 48 + part * 16 + ks / 2 * 32 + ks % 2 * 8), b + ks * (1024 >> 4), v_hi, id_o, part != 2 || ks != 0);
                } else {
                    const bool add = !((firsts >> (g & 31)) & 1);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) mma_ts(t_o, a + ks * 8, b + ks * (kVBlocks * 2048 >> 4), v_hi, id_o, add || ks != 0);
                }
                commit_both(sm.pv_done + g % NS);
                commit_both(sm.v_empty + g % RV);
            };
            // Turn g: the product with tile g's weights, then S of tile g + NS into the place that these had.
#pragma unroll 1
            for (int g = -NS; g < nq; ++g) {
                if (g >= 0) {
                    wait_for(sm.v_full + g % RV, (g / RV) & 1, &sm.abort);
                    wait_for(sm.p_ready + g % NS, (g / NS) & 1, &sm.abort);
                    if (sm.abort) break;
                    tc::fence_after_sync();
                    if (elected()) issue_o(g);
                    __syncwarp();
                }
                if (!end) {
                    wait_for(sm.k_full + nq % RK, (nq / RK) & 1, &sm.abort);
                    if (sm.abort) break;
                    const bool first = left == 0;
                    if (first) {
                        left = sm.way.tiles[units & 15];
                        end = left == 0;
                    }
                    if (!end) {
                        if (first) wait_for(&sm.q_full, units++ & 1, &sm.abort);
                        if (g >= 0) wait_for(sm.pv_done + g % NS, (g / NS) & 1, &sm.abort);
                        if (sm.abort) break;
                        tc::fence_after_sync();
                        if (elected()) issue_s();
                        __syncwarp();
                        firsts = (firsts & ~(1u << (nq & 31))) | (static_cast<uint32_t>(first) << (nq & 31));
                        ++nq;
                        --left;
                    }
                }
            }
            // everything issued is through before the pair ends
            if (elected())
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&sm.drained)) : "memory");
            tc::mbar_wait(&sm.drained, 0, kDrainLimit);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
        const uint32_t my_lanes = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t my_o = t_o + my_lanes + half * (DV / 2);   // at a part's end a thread has half of its row's channels
        const float scale = p.scale * kLog2e, size = scale == 0.f ? 1.f : fabsf(scale);
        const int in = row / p.G;   // token of this CTA's
        const int cta_tok = static_cast<int>(rank) * cta_tokens, tok = cta_tok + in;   // of the unit's
        auto wait = [&](uint64_t* bar, uint32_t parity) { wait_for(bar, parity, &sm.abort); };
        int g = 0;           // tile number
        uint32_t told = 0;   // phases of v_told
        // acc = acc * f + tile's O, of which `at` has 64 columns
        auto add_o = [&](float (&acc)[S::kF32 ? 64 : 1], uint32_t at, int tile, float f) {
            wait(sm.pv_done + tile % NS, (tile / NS) & 1);
            tc::fence_after_sync();
            if constexpr (S::kF32) {
#pragma unroll
                for (int i = 0; i < 64; i += 32) {
                    float v[32];
                    tc::tmem_ld32(at + i, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x = fma2(make_float2(acc[i + e], acc[i + e + 1]), make_float2(f, f), make_float2(v[e], v[e + 1]));
                        acc[i + e] = x.x;
                        acc[i + e + 1] = x.y;
                    }
                }
            }
        };
        do {
            const int t0 = c.t0, t1 = c.t1;
            const int tok0 = c.i * ln.tokens, n_tok = tokens_of(ln, c), off = c.r.len - c.r.n;
            const int here = min(max(n_tok - cta_tok, 0), cta_tokens) * p.G;   // rows of this CTA
            const int end = c.seen;
            float acc[S::kF32 ? 64 : 1] = {};   // fp32 results: the row's sums over this group's tiles but for the newest,
            float to_next = 1.0f;                    // relative to the base of the newest but one; times this to that of the newest
            float m = -INFINITY, l = 0.f;   // of a row: the base of its weights, -inf before it has seen a key; this thread's share of their sum
#pragma unroll 1
            for (int t = t0; t < t1; ++t, ++g) {
                if ((g & 1) != half) continue;   // the other group's
                wait(sm.s_full + g % NS, (g / NS) & 1);
                tc::fence_after_sync();
                const uint32_t my_s = t_s + my_lanes + g % NS * S::kPlace + S::kScores;
                // late: some rows do not see some of the tile's keys
                const bool late = (t + 1) * kKeys > off + tok0 + 1;
                const uint4 there = *reinterpret_cast<const uint4*>(sm.valid[g & 15]);
                if (late || (there.x & there.y & there.z & there.w) != 0xffffffffu || !(scale > 0.f)) {
                    // scores of keys that a row does not see, and the scale's sign, are seen to in place
                    const int sees = min(off + tok0 + tok + 1, end) - t * kKeys;
                    const float sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
                    // (the warp's first row sees the least; where that costs registers that the sums of fp32 results need, it is not asked)
                    const int all_see = !S::kF32 && scale > 0.f ? __shfl_sync(0xffffffffu, sees, 0) : 0;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = sm.valid[g & 15][i];
                        const int n = sees - i * 32;
                        if (all_see - i * 32 >= 32 && w == 0xffffffffu) continue;
                        float s[32];
                        tc::tmem_ld32(my_s + i * 32, s);
                        const uint32_t x = n <= 0 ? 0u : n >= 32 ? w : w & ((1u << n) - 1u);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[e] = (x >> e) & 1 ? s[e] * sign : -INFINITY;
                        tc::tmem_st32(my_s + i * 32, s);
                    }
                    tc::tmem_wait_st();
                }
                float s0[32], s1[32];   // scores for the maximum, read again for the weights
                tmem_ask32(my_s, s0);
                tmem_ask32(my_s + 32, s1);
                float ma = -INFINITY, mb = -INFINITY;
                auto larger = [&](const float (&s)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        ma = max3(ma, s[e], s[e + 1]);
                        mb = max3(mb, s[e + 2], s[e + 3]);
                    }
                };
                tmem_wait_for(s0);
                tmem_wait_for(s1);
                larger(s0);
                tmem_ask32(my_s + 64, s0);
                larger(s1);
                tmem_ask32(my_s + 96, s1);
                tmem_wait_for(s0);
                tmem_wait_for(s1);
                larger(s0);
                larger(s1);
                const float mx = fmaxf(ma, mb) * size;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                if constexpr (S::kF32) {
                    // The groups' bases and sums are apart until the part's end.  The tile before of this group has its O by now, or soon.
                    const float now = fmaxf(m, mx);
                    if (t >= t0 + 2) add_o(acc, t_o + my_lanes + half * 64, g - 2, to_next);
                    to_next = now == m ? 1.0f : ex2(m - now);
                    l *= to_next;
                    m = now;
                    const float base = m == -INFINITY ? 0.f : m;
                    // 32 weights: bf16 parts, each of what the ones before leave -- all bits of a weight.  The first parts go before the
                    // scores, the other two into the place of the scores that they are from
                    auto weights = [&](int i, const float (&s)[32]) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t w[3][8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int at = 16 * h + 2 * e;
                                const float2 x = fma2(make_float2(s[at], s[at + 1]), make_float2(size, size), make_float2(-base, -base));
                                float2 y = make_float2(ex2(x.x), ex2(x.y));
                                sum[e & 1] = add2(sum[e & 1], y);
#pragma unroll
                                for (int part = 0; part < 3; ++part) {
                                    const uint32_t z = w[part][e] = StateIO<bf16>::pack(y.x, y.y);
                                    if (part < 2) y = fma2(make_float2(__uint_as_float(z << 16), __uint_as_float(z & 0xffff0000u)), make_float2(-1.f, -1.f), y);
                                }
                            }
                            tmem_st8u(my_s - 64 + i * 16 + 8 * h, w[0]);
                            tmem_st8u(my_s + i * 32 + 8 * h, w[1]);
                            tmem_st8u(my_s + i * 32 + 16 + 8 * h, w[2]);
                        }
                    };
                    tmem_ask32(my_s, s0);
                    tmem_wait_for(s0);
                    tmem_ask32(my_s + 32, s1);
                    weights(0, s0);
                    tmem_wait_for(s1);
                    tmem_ask32(my_s + 64, s0);
                    weights(1, s1);
                    tmem_wait_for(s0);
                    tmem_ask32(my_s + 96, s1);
                    weights(2, s0);
                    tmem_wait_for(s1);
                    weights(3, s1);
                } else {
                    tmem_ask32(my_s, s0);
                    // the base that the other group had for the tile before, and this tile's for it
                    if (g > 0) take_base(quarter + 4 * (half ^ 1));
                    const float before = t == t0 ? -INFINITY : sm.base[half ^ 1][row];
                    // (a row's base moves by its own scores alone: its result does not depend on the rows beside it)
                    const bool up = mx > before + kSlack;   // (above -inf, at a row's first keys)
                    const float now = up ? mx : before;
                    sm.base[half][row] = now;
                    give_base(quarter + 4 * half);
                    if (t > t0 && __any_sync(0xffffffffu, up)) {
                        wait(sm.pv_done + (g - 1) % NS, ((g - 1) / NS) & 1);   // the tile before has been added: O stands still
                        tc::fence_after_sync();
                        const float f = up ? ex2(before - now) : 1.0f;
#pragma unroll 1
                        for (int i = 0; i < D; i += 32) {
                            float v[32];
                            tc::tmem_ld32(t_o + my_lanes + i, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= f;
                            tc::tmem_st32(t_o + my_lanes + i, v);
                        }
                    }
                    if (now != m) {
                        l *= ex2(m - now);   // (m -inf: there is none yet)
                        m = now;
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    auto weights = [&](int i, const float (&s)[32]) {   // two keys a column, in the place of scores that have been read
                        uint32_t w2[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 x = fma2(make_float2(s[2 * e], s[2 * e + 1]), make_float2(size, size), make_float2(-base, -base));
                            const float2 y = make_float2(ex2(x.x), ex2(x.y));
                            sum[e & 1] = add2(sum[e & 1], y);
                            w2[e] = StateIO<bf16>::pack(y.x, y.y);
                        }
                        tmem_st16u(my_s + i * 16, w2);
                    };
                    tmem_wait_for(s0);
                    tmem_ask32(my_s + 32, s1);
                    tmem_wait_for(s1);
                    weights(0, s0);
                    tmem_ask32(my_s + 64, s0);
                    tmem_wait_for(s0);
                    weights(1, s1);
                    tmem_ask32(my_s + 96, s1);
                    tmem_wait_for(s1);
                    weights(2, s0);
                    weights(3, s1);
                }
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                if (late) {
                    // Strays among the values that some rows do not see are taken out of this CTA's channels, and what the boxes brought from
                    // behind the last key that anyone sees.
                    const int k0 = max(0, off + tok0 + 1 - t * kKeys), kend = end - t * kKeys, k1 = min(kKeys, (kend + vb.tokens - 1) / vb.tokens * vb.tokens);
                    bool landed = k0 < k1;
                    if (landed) {   // the first CTA's barrier tells of both; it tells the second one
                        if (rank == 0) {
                            wait(sm.v_full + g % RV, (g / RV) & 1);
                            landed = !sm.abort;
                            if (landed && (threadIdx.x & 127) == 0) arrive_at(sm.v_told + g % 6, 1);
                        } else {
                            wait(sm.v_told + g % 6, (told >> (g % 6)) & 1);
                            landed = !sm.abort;
                        }
                        told ^= 1u << (g % 6);
                    }
                    if (landed) {
                        uint8_t* const st = v_s + g % RV * S::kStageV;
                        bool found = false;
#pragma unroll 1
                        for (int x = threadIdx.x & 127; x < (k1 - k0) * (S::kVCh / 8); x += 128) {
                            const int key = k0 + x / (S::kVCh / 8), ch = x % (S::kVCh / 8);
                            uint8_t* const at = S::kF32 ? st + key * 64 + (ch ^ ((key >> 1) & 3)) * 16
                                                        : st + (key >> 3) * (kVBlocks * 1024) + ch / 8 * 1024 + (key & 7) * 128 + ((ch ^ key) & 7) * 16;
                            if (key < kend) found |= attn::take_strays<bf16>(at);
                            else *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
                        }
                        if (found) {
                            volatile int* const mark = sm.strays.mark();
                            *mark = 1;
                            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(smem_u32(const_cast<int*>(mark)), rank ^ 1)), "r"(1) : "memory");
                            asm volatile("fence.acq_rel.cluster;" ::: "memory");
                        }
                        tc::fence_proxy_async();
                    }
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_at(sm.p_ready + g % NS, 0);
            }
            // -------------------------------------------------------- the part's end
            const bool any = t0 < t1, whole = c.whole();
            const long long tr = static_cast<long long>(c.r.row0) + tok0 + tok;
            const int h = c.hk / S::kSlices * p.G + row - in * p.G, ch0 = half * (DV / 2), col0 = c.hk % S::kSlices * DV + ch0;   // of the part, of the head
            const bool gated = p.gate && row < here, gate32 = on32(p.gate) && p.ldg % 16 == 0;
            const bf16* const gate = static_cast<const bf16*>(p.gate) + (tr * p.ldg + static_cast<long long>(h) * D + col0);
            if (gated)   // the gate's lines, while the last products run
                for (int i = 0; i < DV / 2; i += 64) prefetch_l2(gate + i);
            if constexpr (S::kF32) {   // the groups' sums to where their last O was
                const int mine = (g - 1 - half) & 1 ? g - 2 : g - 1;
                if (mine >= g - (t1 - t0)) add_o(acc, t_o + my_lanes + half * 64, mine, to_next);
#pragma unroll
                for (int i = 0; i < 64; i += 32) tc::tmem_st32(t_o + my_lanes + half * 64 + i, reinterpret_cast<float(&)[32]>(acc[i]));
                tc::tmem_wait_st();
                tc::fence_before_sync();
            }
            if ((g & 1) == half && quarter == 0) {   // the way to the next part, by a warp of the group that did not have the last tile
                Part next = c;
                const bool more = to_next_part(p, ln, sh, next);
                if ((threadIdx.x & 127) == 0) {
                    sm.way.next = next;
                    sm.way.more = more;
                }
            }
            uint32_t gt[DV / 64][2][8];   // the gates of this thread's channels; all of them now where there are few
            auto gates = [&](int i) {
                load16(gate + 32 * i, gate32, gt[i][0]);
                load16(gate + 32 * i + 16, gate32, gt[i][1]);
            };
            if (S::kGates && whole && gated) {
#pragma unroll
                for (int i = 0; i < DV / 64; ++i) gates(i);
            }
            if constexpr (!S::kF32) {
                if (any) wait(sm.pv_done + (g - 1) % NS, ((g - 1) / NS) & 1);
                tc::fence_after_sync();
            }
            if (p.test_stall && warp == 3) long_wait(smem_u32(&sm.never), 0, &sm.abort, 256);
            if (sm.abort) sm.stop = 1;   // told before the barrier, behind which all look
            if (((g - 1) & 1) == half && (threadIdx.x & 127) == 0) {   // by the group that had the last tile
                sm.strays.take_over(any);
                sm.last = whole;
            }
            // the sum relative to the last tile's base, which the group of that tile has
            sm.sum[half][row] = l;
            sm.base[half][row] = m;
            sync_softmax();
            if (sm.stop) {   // a wait gave up: nothing of this part is written
                if (threadIdx.x == 0 && p.status) atomicOr(p.status + c.b, 16);
            } else {
                m = S::kF32 ? fmaxf(sm.base[0][row], sm.base[1][row]) : sm.base[any ? (g - 1) & 1 : 0][row];
                float sum = 0.f, fg[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    fg[i] = sm.base[i][row] == -INFINITY ? 0.f : ex2(sm.base[i][row] - m);
                    sum += fg[i] == 0.f ? 0.f : sm.sum[i][row] * fg[i];
                }
                if constexpr (S::kF32) tc::fence_after_sync();
                auto load_o = [&](int i, float (&v)[32]) {   // columns i.. of this thread's half, relative to m
                    tc::tmem_ld32(my_o + i, v);
                    if constexpr (S::kF32) {
                        float w[32];
                        tc::tmem_ld32(my_o + 64 + i, w);
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = fmaf(v[e], fg[0], w[e] * fg[1]);
                    }
                };
                const Parts<kRows, DV> parts(p.workspace, workers);
                const size_t place = Parts<kRows, DV>::place(worker, c);
                float* const part = parts.o + (place * kRows + rank * 128) * DV;
                bool result = whole;   // this CTA finishes the rows
                if (!whole) {
#pragma unroll 1
                    for (int i = 0; i < DV / 2; i += 32) {
                        float v[32];
                        load_o(i, v);
                        if (row < here) {
                            float* const to = part + part_at(row, ch0 + i);
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t y[8];
#pragma unroll
                                for (int q = 0; q < 8; ++q) y[q] = __float_as_uint(v[e + q]);
                                store16(to + e * 128, true, y);
                            }
                        }
                    }
                    if (half == 0 && row < here) parts.ml[place * kRows + rank * 128 + row] = make_float2(m, sum);
                    // the worker that arrives last joins this CTA's rows of all parts; of many parts with many rows the last of each kJoin
                    // joins those first, for one CTA reads no more than some 70 bytes a ns
                    const long long first = c.at + ln.cost;
                    const int w0 = sh.owner(first), n = sh.owner(first + static_cast<long long>(kKeys) * (c.tiles - 1)) - w0 + 1;
                    const bool few = here * (DV / 4) <= 4 * kSoft;
                    const int row0 = static_cast<int>(rank) * 128;
                    const bool twice = n > kJoin && !few;
#pragma unroll 1
                    for (bool first_time = twice;; first_time = false) {
                        // parts `from`, `from` + step, .. of the unit, `these` of them, to the first one's place or at last to tensor memory
                        const int from = first_time ? (worker - w0) / kJoin * kJoin : 0, step = twice && !first_time ? kJoin : 1;
                        const int these = first_time ? min(kJoin, n - from) : (n + step - 1) / step;
                        sync_softmax();
                        if (threadIdx.x == 0) {
                            // counts the parts, and those with strays above them; zero again behind the last one
                            unsigned old;
                            int* const counter = parts.counters + (first_time ? kMaxWorkers + 4 * (w0 + from) + 2 * (from == 0) : 2 * w0) + rank;
                            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(sm.strays.now ? kStrayPart + 1 : 1) : "memory");
                            sm.last = old % kStrayPart == static_cast<unsigned>(these - 1);
                            if (sm.last) {
                                *counter = 0;
                                if (old >= kStrayPart) sm.strays.now = 1;
                            }
                        }
                        sync_softmax();
                        if (!sm.last) break;
                        if (few) {
                            join_few<S>(p, c, parts, w0, n, tok0, cta_tok, here, row0);
                            break;
                        }
                        auto row_of = [&](int k) {
                            const int at = from + k * step;
                            return static_cast<uint32_t>((at == 0 ? 2 * w0 + 1 : 2 * (w0 + at)) * kRows + row0);
                        };
                        // in their order, whoever was last: statistics first
                        m = -INFINITY;
                        sum = 0.f;
                        if (row < here)
#pragma unroll 2
                            for (int k = 0; k < these; ++k) m = fmaxf(m, __ldcg(&parts.ml[row_of(k) + row].x));
                        const float base = m == -INFINITY ? 0.f : m;
                        if (row < here)
#pragma unroll 2
                            for (int k = 0; k < these; ++k) {
                                const float2 z = __ldcg(parts.ml + row_of(k) + row);
                                sum = fmaf(ex2(z.x - base), z.y, sum);
                            }
#pragma unroll 1
                        for (int i = 0; i < DV / 2; i += 32) {
                            float v[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = 0.f;
                            if (row < here)
#pragma unroll 1
                                for (int k = 0; k < these; k += 2) {   // two parts' loads together; past the last part it again
                                    uint32_t y[2][4][8];
                                    float mk[2];
#pragma unroll
                                    for (int x = 0; x < 2; ++x) {
                                        const uint32_t at = row_of(min(k + x, these - 1));
                                        mk[x] = __ldcg(&parts.ml[at + row].x);
#pragma unroll
                                        for (int q = 0; q < 4; ++q) load16(parts.o + at * DV + part_at(row, ch0 + i + 8 * q), true, y[x][q]);
                                    }
#pragma unroll
                                    for (int x = 0; x < 2; ++x) {
                                        if (k + x == these) break;   // (not added with a weight of zero: it may be infinite)
                                        const float fk = ex2(mk[x] - base);
#pragma unroll
                                        for (int q = 0; q < 32; ++q) v[q] = fmaf(fk, __uint_as_float(y[x][q / 8][q % 8]), v[q]);
                                    }
                                }
                            if (first_time) {
                                if (row < here) {
                                    float* const to = parts.o + row_of(0) * DV + part_at(row, ch0 + i);
#pragma unroll
                                    for (int e = 0; e < 32; e += 8) {
                                        uint32_t y[8];
#pragma unroll
                                        for (int q = 0; q < 8; ++q) y[q] = __float_as_uint(v[e + q]);
                                        store16(to + e * 128, true, y);
                                    }
                                }
                            } else {
                                __syncwarp();
                                tc::tmem_st32(my_o + i, v);
                            }
                        }
                        if (!first_time) {
                            tc::tmem_wait_st();
                            result = true;
                            break;
                        }
                        sync_softmax();   // all have read the statistics
                        if (half == 0 && row < here) parts.ml[row_of(0) + row] = make_float2(m, sum);
                    }
                }
                if (result) {   // in tensor memory
                    const float f = sum == 0.f ? 0.f : 1.0f / sum;
                    const bool out32 = on32(p.out);
                    const long long to = (tr * p.Hq + h) * D + col0;
                    auto finish = [&](int i, const uint32_t (&gt)[2][8]) {   // channels i.. of this thread's
                        float v[32];
                        if (!whole) tc::tmem_ld32(my_o + i, v);
                        else if (any) load_o(i, v);
                        if (row < here) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = any ? v[e] * f : 0.f;
                            if (gated) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const uint32_t x = gt[e / 16][e % 16 / 2];
                                    v[e] *= gate_of<S::kF32>(__uint_as_float(x << 16));
                                    v[e + 1] *= gate_of<S::kF32>(__uint_as_float(x & 0xffff0000u));
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += S::kF32 ? 8 : 16) {
                                uint32_t y[8];
#pragma unroll
                                for (int q = 0; q < 8; ++q) y[q] = S::kF32 ? __float_as_uint(v[e + q]) : StateIO<bf16>::pack(v[e + 2 * q & 31], v[e + 2 * q + 1 & 31]);
                                if constexpr (S::kF32) store16(static_cast<float*>(p.out) + to + i + e, out32, y);
                                else store16(static_cast<bf16*>(p.out) + to + i + e, out32, y);
                            }
                        }
                    };
                    if constexpr (S::kGates) {
                        if (!whole && gated) {
#pragma unroll
                            for (int i = 0; i < DV / 64; ++i) gates(i);
                        }
#pragma unroll
                        for (int i = 0; i < DV / 64; ++i) finish(32 * i, gt[i]);
                    } else {
#pragma unroll 1
                        for (int i = 0; i < DV / 2; i += 32) {
                            if (gated) {
                                load16(gate + i, gate32, gt[0][0]);
                                load16(gate + i + 16, gate32, gt[0][1]);
                            }
                            finish(i, gt[0]);
                        }
                    }
                }
                if (sm.strays.now && sm.last) {
                    sync_softmax();
                    add_strays<S>(p, c, tok0, cta_tok, here);
                }
                tc::fence_before_sync();
            }
            const bool more = sm.way.more;
            if (more) c = sm.way.next;
            sync_softmax();   // the sums, sm.last and sm.way.next have been read
            if (!more) break;
        } while (true);
        if (!S::kF32 && g > 0 && (g & 1) == half) take_base(quarter + 4 * (half ^ 1));   // the last one given
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync_all();   // no product, copy or arrival concerns this pair any more
    tc::fence_after_sync();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem), "r"(512));
}

// The map of a half of the cache, and the boxes of up to `most` tokens and `blocks` blocks of `block` channels; false if there can be none.
bool cache_map(CUtensorMap* m, Boxes* b, const ChunkParams& p, const void* half, int D, int most, int blocks, uint32_t block) {
    const KvCache& c = p.cache;
    auto bytes = [&](long long stride) { return stride ? static_cast<uint64_t>(stride) * 2 : static_cast<uint64_t>(D) * 2; };
    const uint64_t ps = c.page_size, pages = c.num_pages, heads = p.Hkv, parts = D / block;
    int two = 128;   // tokens that always lie in one page
    while (c.page_size % two != 0) two /= 2;
    const bool pages_follow = pages == 1 || c.page_stride == c.page_size * c.token_stride;
    const bool heads_follow = pages == 1 || heads == 1 || c.page_stride == p.Hkv * c.head_stride;
    *b = Boxes{two < most ? two : most, two >= 8 && (pages_follow || (heads_follow && pages * heads <= INT32_MAX)), 0, 0};
    if (b->whole) {
        b->group = pages_follow ? c.page_size / 8 : 0;
        b->head = pages_follow ? 0 : p.Hkv;
        const uint64_t dims[5] = {block, 8, parts, pages_follow ? pages * ps / 8 : ps / 8, pages_follow ? heads : pages * heads};
        const uint64_t strides[4] = {bytes(c.token_stride), 2 * block, bytes(c.token_stride) * 8, pages_follow || heads > 1 ? bytes(c.head_stride) : bytes(c.page_stride)};
        const uint32_t boxes[5] = {block, 8, static_cast<uint32_t>(blocks), static_cast<uint32_t>(b->tokens / 8), 1};
        return make_tensor_map_bf16(m, half, 5, dims, strides, boxes);
    }
    b->tokens = two < 8 ? two : 8;
    if (b->tokens * block * 2 < 128) return false;   // where a box goes is a multiple of 128 bytes
    const uint64_t dims[5] = {block, ps, parts, heads, pages};
    const uint64_t strides[4] = {bytes(c.token_stride), 2 * block, bytes(c.head_stride), bytes(c.page_stride)};
    const uint32_t boxes[5] = {block, static_cast<uint32_t>(b->tokens), 1, 1, 1};
    return make_tensor_map_bf16(m, half, 5, dims, strides, boxes);
}

template <class S>
cudaError_t launch(const ChunkParams& from, int sms, bool* done, cudaStream_t stream) {
    constexpr int D = S::D;
    ChunkParams p = from;
    p.heads = p.Hkv * S::kSlices;
    *done = false;
    Boxes kb, vb;
    Division by_page{0, 0};
    int bits = 0;   // of page_size, rounded up
    while ((1ll << bits) < p.cache.page_size) ++bits;
    if (bits > 0) by_page = Division{static_cast<uint32_t>(((1ull << (31 + bits)) + p.cache.page_size - 1) / p.cache.page_size), static_cast<uint32_t>(bits - 1)};
    CUtensorMap k, v, q;
    const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.Hq), static_cast<uint64_t>(p.T)};
    const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(p.ldq) * 2};
    const uint32_t boxes[3] = {64, static_cast<uint32_t>(p.G), static_cast<uint32_t>(128 / p.G)};
    if (!cache_map(&k, &kb, p, p.cache.k, D, 64, D / 64, 64) || !cache_map(&v, &vb, p, p.cache.v, D, 128, S::kVCh / S::kBlock, S::kBlock) || !make_tensor_map_bf16(&q, p.q, 3, dims, strides, boxes))
        return cudaSuccess;
    *done = true;
    const cudaError_t e = cudaFuncSetAttribute(chunk_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    const int pairs = min(sms / 2, kMaxWorkers / 2);
    return launch_dependent_cluster(chunk_tc_kernel<S>, 2, dim3(2 * pairs), dim3(kThreads), S::kSmem, stream, p, k, v, q, kb, vb, by_page);
}

}  // namespace

size_t tc_workspace_bytes(int head_dim, bool out_bf16) {
    if (head_dim == 64 || !out_bf16) return parts_bytes<kRows, 64>(kMaxWorkers / 2);
    if (head_dim == 128) return parts_bytes<kRows, 128>(kMaxWorkers / 2);
    return parts_bytes<kRows, 256>(kMaxWorkers / 2);
}

cudaError_t launch_tc(const ChunkParams& p, int head_dim, bool out_bf16, int sms, bool* done, cudaStream_t stream) {
    if (head_dim == 64) return out_bf16 ? launch<Tc<64, false>>(p, sms, done, stream) : launch<Tc<64, true>>(p, sms, done, stream);
    if (head_dim == 128) return out_bf16 ? launch<Tc<128, false>>(p, sms, done, stream) : launch<Tc<128, true>>(p, sms, done, stream);
    return out_bf16 ? launch<Tc<256, false>>(p, sms, done, stream) : launch<Tc<256, true>>(p, sms, done, stream);
}

}  // namespace chunk
}  // namespace gdn
