// gdn_attn.cuh -- attention of the last K tokens of each sequence over the paged key-value cache
// (include/gdn_attn.h, gdn_attn_decode): the kernel, instantiated per type in gdn_attn_bf16.cu and
// gdn_attn_f32.cu; gdn_attn_tc.cu builds on it for many rows.
//
// Mathematics.  A kv head's G query heads times K tokens are R = G*K rows that share its keys.  Over any set of
// keys a row has m = max s, l = sum e^(s-m), o = sum e^(s-m) v; two sets join as m = max(m1, m2),
// l = l1 e^(m1-m) + l2 e^(m2-m), o likewise, and o / l is the result once.  Scores are kept in base 2
// (s log2 e).  One pass over the keys; every key and value is read from memory once per block of rows.
//
// Strays.  A key that a row does not see has the weight 0 in it, which keeps its value out only if that is finite.  Of the keys
// that some rows of a block see and others do not -- the last K - 1 of a sequence -- the values are looked at before
// the products; an infinite or NaN element is zeroed in shared memory, and added, from the cache, to the results of the rows that see
// its key, by the CTA that finishes them: not to a part, whose weight in the join may be zero (a row that sees none of
// its keys, far larger scores elsewhere) and would make NaN of an infinity.  (Three tokens, 24 rows, 64 ragged sequences: 107.7
// us, 105.5 without; looked at by the computing warps 111, whose registers do not suffice for it.  One token has no such
// keys and a kernel without all this.)
//
// What bounds it: the cache's bytes.  A bf16 key and value of head size d are 4 d bytes for 4 R d operations: the stream is the
// time up to 16 rows (64 ragged sequences of 0.54 GB, heads of 256, floor 80 us: 8 rows 94 us, 16 rows 96); with more the
// operands' way from shared memory to the products shows (24 rows 108, 32 rows 121).  The layout serves the stream:
//   * one persistent CTA per SM; the keys of all (sequence, kv head, row block) groups, cut into tiles, are
//     divided evenly over the CTAs whatever the lengths, from the lengths on the device (no host plan).  A group
//     counts kGroupCost tiles more than it has, for its begin and end;
//   * four producer warps issue cp.async (16 bytes a lane, zero fill for keys that are not there) into rings of 16 KB
//     stages (8 KB for bf16 heads of 64) that fill 192 KB of shared memory (160 or 128 KB beside the queries of many rows), most of
//     it in flight; the loads run across group borders.  They have
//     warps of their own because a warp stands still while the memory takes its requests: with the loads in the computing
//     warps, those spent 175 of 305 us there (64 ragged sequences, 2.2 GB) and the two times added up;
//   * the other warps are key groups x row groups: KG key groups each walk their own tiles with their own ring, so
//     their only meeting is the join of the triples (m, l, o) at a group's end; RG warps of a key group hold
//     different rows and share its stages;
//   * a group whose tiles span several CTAs is joined through the workspace by the CTA that arrives last.
//
// Waits.  Producers and consumers meet at an mbarrier pair a stage.  Every wait has a limit; a warp whose wait gives up
// sets a flag that ends all waits of the CTA, nothing more is written, and the sequences concerned get bit 4 of
// their status words.  What a computing warp missed is told by the warp itself (stop) before the barrier at its group's end,
// behind which all of them look: a copy of the flag taken before that barrier misses a warp that gives up later.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "gdn_tc.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxCtas = 256;
constexpr int kFanOne = 16, kMaxFan = 32;         // parts joined at once: all of up to kFanOne, at most kMaxFan
constexpr size_t kCounterBytes = 3 * kMaxCtas * 4;   // at the start of the workspace
static_assert(kMaxCtas / 12 < kMaxFan, "parts of the second step");
constexpr unsigned kStrayPart = 1 << 16;          // in a counter of parts
static_assert(kMaxCtas < static_cast<int>(kStrayPart), "parts of a group");
constexpr int kFinished = 1, kStrays = 2;         // what join_group leaves

// Shape of a kernel: Ta cache type, D head size, NT blocks of 8 rows a warp holds, RG row groups, KG key
// groups, PIECES bf16 parts of a softmax weight (bf16 only), FR rows a warp holds (fp32; NT is 1).
template <typename Ta_, int D_, int NT_, int RG_, int KG_, int PIECES_, int FR_ = 8>
struct Shape {
    using Ta = Ta_;
    static constexpr bool kBf16 = std::is_same<Ta_, __nv_bfloat16>::value;
    static constexpr int D = D_, NT = NT_, RG = RG_, KG = KG_, PIECES = PIECES_;
    static constexpr int kWarpRows = kBf16 ? 8 * NT : FR_, kPassRows = kBf16 ? 8 : FR_;   // of a warp, of a join pass
    static constexpr int kThreads = RG * KG * 32;                      // that compute
    static constexpr int kAll = kThreads + 128;                        // and four warps that load
    static constexpr int PW = 4 / KG;                                  // of them, a key group's
    static constexpr int kRows = kWarpRows * RG < 8 ? 8 : kWarpRows * RG;   // rows of a block (of 8, some are not used by fewer)
    static constexpr int kRowBytes = D * static_cast<int>(sizeof(Ta));
    static constexpr int KT = kBf16 ? (D == 256 ? 16 : 32) : 2048 / D;   // keys of a stage
    static constexpr int kHalfBytes = KT * kRowBytes;                  // the keys of a stage, then the values
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kQBytes = kBf16 ? kRows * kRowBytes : 0;      // queries, bf16 kernels only
    static constexpr int kRing = kQBytes > 32768 ? 131072 : kQBytes > 16384 || kRows == 128 ? 163840 : 196608;
    static constexpr int kStages = kRing / kStageBytes / KG;           // of one key group
    static constexpr int kTile = KG * KT;                              // keys of a tile
    // A group's begin and end, in tiles.  A tile is KG stages: 64 KB where it was measured (KG = 4; bf16 heads of 64 32 KB); with the
    // two and one key groups of many fp32 rows or fp32 results it is a half or a quarter of that, and so is the weight, not measured
    // apart.  64 ragged sequences, heads of 256, 24 rows: 3 tiles 118 us, 5 tiles 108,
    // 8 tiles 106; heads of 128, 24 rows: 3 tiles 121, 8 tiles 132.  fp32, 16 sequences, 8 rows: heads of 64 1 tile 48.7,
    // 2 tiles 49.9, 5 tiles 56 (9 sequences in pages of 11: 15.8, 15.0, 16.4); of 128 1 tile 68, 2 and 3 tiles 64, 5 tiles 68; of
    // 256 2 tiles 119, 3 tiles 110, 5 tiles 102, 8 tiles 107.
    static constexpr int kGroupCost = kBf16 ? (D == 64 ? 3 : D == 128 ? 4 : RG > 1 ? 8 : 6) : D == 64 ? 2 : D == 128 ? 3 : 5;
    static constexpr int JC = D < 128 ? D : 128;                       // channels of a join pass
    static constexpr int kJPitch = JC + 4;                             // 8t+g banks for the writes below
    static constexpr int kPartBytes = (kMaxFan * 4 + 8) * kRows;       // weights and totals of a join of parts
    static constexpr int kJoinBytes = KG * 8 * kJPitch * 4 > kPartBytes ? KG * 8 * kJPitch * 4 : kPartBytes;
    static constexpr int kMlBytes = KG * kRows * 8;
    static constexpr int kBarBytes = (2 * KG * kStages + 1) * 8;       // full and empty of each stage, and one that nothing arrives on
    static constexpr int kValidBytes = KG * kStages * PW * 4;
    static constexpr int kSmem = KG * kStages * kStageBytes + kQBytes + kJoinBytes + kMlBytes + kBarBytes + kValidBytes;
    // With more than 8 warps the computing ones take over registers of the loading ones: 168 a thread at launch for 12
    // warps are 2/3 of 224 and 1/3 of 56, 128 for 16 are 3/4 of 152 and 1/4 of 56.
    static constexpr bool kMoveRegs = kAll > 256;
    static constexpr int kRegs = kAll == 384 ? 224 : 152;
    static_assert(!kMoveRegs || kAll == 384 || kAll == 512, "registers");
    static_assert(kStages >= 3 && KT % PW == 0 && KT / PW <= 32 && kSmem + 512 <= 232448, "shape");
};

using tc::smem_u32;

constexpr int kWaitLimit = 1 << 22;   // polls of a wait before it gives up

// Wait for phase `parity` of `bar`; false when it gives up or another warp has.  A loop that is not unrolled: there are a score of
// waits in a kernel, and with 16 polls each written out the tcgen05 kernel had 160 to 190 KB of code, now 100 to 130 (64 rows,
// heads of 64: 350 us against 262).
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int limit = kWaitLimit) {
#pragma unroll 1
    for (int it = 0; it < limit; ++it) {
        if (tc::mbar_wait(bar, parity, 1)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    return false;
}
// The same by a whole warp, with one answer for all of it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, stage_wait(bar, parity, abort));
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// c[16x8] += a[16x16] . b[16x8], bf16 operands
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kLate = 1 << 30;   // beside a key's head: one of the last K - 1 of its sequence

// Where a walk over the tiles stands: group (b, hk, rb), tile of the group.  `at` numbers the tiles of all groups one
// after another, each group's followed by cost numbers that no tile has.
struct Cursor {
    int b, hk, rb, tile, tiles, len;
    long long at;
};

__device__ __forceinline__ int seq_keys(const AttnParams& p, int b, bool* over) {
    const long long cap = static_cast<long long>(p.max_pages) * p.cache.page_size;
    const int n = p.seq_len[b];
    *over = n > cap;
    return static_cast<int>(min(static_cast<long long>(max(n, 0)), cap));
}

template <int kTile>
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }   // an empty sequence has one

template <class S>
__device__ __forceinline__ void next_group(const AttnParams& p, Cursor& c, int row_blocks) {
    c.tile = 0;
    if (++c.rb < row_blocks) return;
    c.rb = 0;
    if (++c.hk < p.Hkv) return;
    c.hk = 0;
    if (++c.b < p.B) {
        bool over;
        c.len = seq_keys(p, c.b, &over);
        c.tiles = tiles_of<S::kTile>(c.len);
    }
}

template <class S>
__device__ __forceinline__ void advance(const AttnParams& p, Cursor& c, int row_blocks) {
    ++c.at;
    if (++c.tile < c.tiles) return;
    c.at += S::kGroupCost;
    next_group<S>(p, c, row_blocks);
}

struct Split {
    int* counters;     // [2 kMaxCtas] by a part's place, [kMaxCtas] by CTA
    float* o;          // [2 * ctas][kRows][D]
    float2* ml;        // [2 * ctas][kRows]
};

// row / G for rows under 4096 and G <= 16 (g_inv = 65536 / G rounded up).
__device__ __forceinline__ int token_of(const AttnParams& p, int row) { return static_cast<int>((static_cast<unsigned>(row) * p.g_inv) >> 16); }

// The result of a row's channels c..c+3, gated, into out; added to what is there if `add`.
template <typename Ta, int D, bool add = false>
__device__ __forceinline__ void put(const AttnParams& p, bool out_bf16, int b, int hk, int row, int c, float4 y) {
    const int tok = token_of(p, row), h = hk * p.G + row - tok * p.G;
    const long long t = static_cast<long long>(b) * p.K + tok;
    if (p.gate) {
        const float4 g = StateIO<Ta>::ld(static_cast<const Ta*>(p.gate) + t * p.ldg + static_cast<long long>(h) * D + c);
        y.x *= gate_of(g.x);
        y.y *= gate_of(g.y);
        y.z *= gate_of(g.z);
        y.w *= gate_of(g.w);
    }
    const long long at = (t * p.Hq + h) * D + c;
    if (add) {
        const float4 x = out_bf16 ? StateIO<__nv_bfloat16>::ld(static_cast<const __nv_bfloat16*>(p.out) + at)
                                  : StateIO<float>::ld(static_cast<const float*>(p.out) + at);
        y = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    if (out_bf16) StateIO<__nv_bfloat16>::st(static_cast<__nv_bfloat16*>(p.out) + at, y);
    else StateIO<float>::st(static_cast<float*>(p.out) + at, y);
}

// Words of two bf16 or one fp32: bits 15 and 31 (bit 31) of the result are set where an element is infinite or NaN.
template <typename Ta>
__device__ __forceinline__ uint32_t stray_bits(uint32_t w) {
    return sizeof(Ta) == 4 ? (w & 0x7f800000u) + 0x00800000u : (w & 0x7f807f80u) + 0x00800080u;
}
template <typename Ta>
__device__ __forceinline__ bool has_strays(uint4 v) {
    const uint32_t any = stray_bits<Ta>(v.x) | stray_bits<Ta>(v.y) | stray_bits<Ta>(v.z) | stray_bits<Ta>(v.w);
    return (any & (sizeof(Ta) == 4 ? 0x80000000u : 0x80008000u)) != 0;
}
// Whether there are strays among the values of the keys `late` (bits) of a warp, lane k holding key k's offset.  kChunks: of 16
// bytes, a value's.  Small, for the registers of the loading warps: in batches of loads 24 rows took 108 us instead of 105.
template <typename Ta, int kChunks>
__device__ __forceinline__ bool find_strays(const Ta* v, long long off, uint32_t late) {
    constexpr int kAtOnce = kChunks < 32 ? 32 / kChunks : 1;   // keys
    const int lane = threadIdx.x & 31;
    bool any = false;
#pragma unroll 1
    for (int key = (__ffs(late) - 1) / kAtOnce * kAtOnce; key < 32 && late >> key; key += kAtOnce) {
        const int k = key + lane / kChunks;
        const long long o = __shfl_sync(0xffffffffu, off, k) + lane % kChunks * (16 / static_cast<int>(sizeof(Ta)));
        if ((late >> k) & 1) {
            any |= has_strays<Ta>(*reinterpret_cast<const uint4*>(v + o));
            if (kChunks > 32) any |= has_strays<Ta>(*reinterpret_cast<const uint4*>(v + o + 32 * (16 / static_cast<int>(sizeof(Ta)))));
        }
    }
    return __any_sync(0xffffffffu, any);
}
// Zero what is not finite among 16 bytes in shared memory; true if anything was.
template <typename Ta>
__device__ __forceinline__ bool take_strays(uint8_t* at) {
    uint4* const x = reinterpret_cast<uint4*>(at);
    if (!has_strays<Ta>(*x)) return false;
    uint32_t w[4] = {x->x, x->y, x->z, x->w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = stray_bits<Ta>(w[i]);
        w[i] = sizeof(Ta) == 4 ? (b >> 31 ? 0u : w[i]) : w[i] & ((b >> 31 ? 0u : 0xffff0000u) | ((b >> 15) & 1 ? 0u : 0xffffu));
    }
    *x = make_uint4(w[0], w[1], w[2], w[3]);
    return true;
}

// The strays of the keys that a row sees, in its channels c..c+3; zeros elsewhere.
template <typename Ta>
__device__ __forceinline__ float4 strays_of(const AttnParams& p, int b, int hk, int len, int row, int c) {
    const int end = len - p.K + token_of(p, row);   // the last key that it sees
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int j = max(0, len - p.K + 1); j <= end; ++j) {
        const int k = j / p.cache.page_size, page = p.block_table[static_cast<size_t>(b) * p.max_pages + k];
        if (page < 0 || page >= p.cache.num_pages) continue;
        const float4 v = StateIO<Ta>::ld(static_cast<const Ta*>(p.cache.v) + page * p.cache.page_stride +
                                         (j - k * p.cache.page_size) * p.cache.token_stride + hk * p.cache.head_stride + c);
        y.x += isfinite(v.x) ? 0.f : v.x;
        y.y += isfinite(v.y) ? 0.f : v.y;
        y.z += isfinite(v.z) ? 0.f : v.z;
        y.w += isfinite(v.w) ? 0.f : v.w;
    }
    return y;
}

__device__ __forceinline__ float4 times(float4 y, float f) { return make_float4(y.x * f, y.y * f, y.z * f, y.w * f); }

// The barrier of the computing warps.
template <class S>
__device__ __forceinline__ void sync_computing() {
    asm volatile("bar.sync 1, %0;" ::"n"(S::kThreads) : "memory");
}

// a / b with the short division where it will do.
__device__ __forceinline__ long long quot(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// Join `count` parts of a group's rows (part k's rows begin at row_at(k)): into the result if `final`, else into place
// `to`.  The loads of a step are issued together: a round trip for the statistics, then one for every eight parts of
// kBatch * kThreads float4s.  Parts have all kRows rows; those past `rows` hold nothing and go nowhere.
template <class S, class F>
__device__ __forceinline__ void join_parts(const AttnParams& p, bool out_bf16, const Split& sp, int rows, int b, int hk, int row0,
                                           float* w_s, int count, bool final, int to, F row_at) {
    using Ta = typename S::Ta;
    constexpr int D = S::D, kItems = S::kRows * D / 4, kShare = kItems / S::kThreads;
    constexpr int kBatch = kShare < 1 ? 1 : kShare < 4 ? kShare : 4;
    constexpr int kTpr = 8;   // threads a row for the statistics
    static_assert(kBatch == 1 || kItems % (S::kThreads * kBatch) == 0, "a batch ends with the rows of a part");
    float2* const t_s = reinterpret_cast<float2*>(w_s + kMaxFan * S::kRows);   // [kRows]; w_s [kMaxFan][kRows]
#pragma unroll 1
    for (int r = threadIdx.x / kTpr; r < rows; r += S::kThreads / kTpr) {
        const int sub = threadIdx.x % kTpr;
        const uint32_t group = 0xffu << (threadIdx.x & 24);
        float2 t[kMaxFan / kTpr];
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxFan / kTpr; ++i) {
            const int k = i * kTpr + sub;
            t[i] = make_float2(-INFINITY, 0.f);
            if (k < count) t[i] = __ldcg(sp.ml + row_at(k) + r);
        }
#pragma unroll
        for (int i = 0; i < kMaxFan / kTpr; ++i) mm = fmaxf(mm, t[i].x);
#pragma unroll
        for (int d = 1; d < kTpr; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(group, mm, d));
        const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int i = 0; i < kMaxFan / kTpr; ++i) {
            const float f = ex2(t[i].x - base);
            ll = fmaf(f, t[i].y, ll);
            w_s[(i * kTpr + sub) * S::kRows + r] = f;
        }
#pragma unroll
        for (int d = 1; d < kTpr; d <<= 1) ll += __shfl_xor_sync(group, ll, d);
        if (sub == 0) {
            t_s[r] = make_float2(mm, ll);
            if (!final) sp.ml[static_cast<size_t>(to) * S::kRows + r] = make_float2(mm, ll);
        }
    }
    sync_computing<S>();
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < rows * (D / 4); i0 += S::kThreads * kBatch) {
        float4 y[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = 0; k0 < count; k0 += 8) {   // past the last part it again, with the weight 0
            float4 v[8][kBatch];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float4* const x = reinterpret_cast<const float4*>(sp.o + row_at(min(k0 + u, count - 1)) * D) + i0;
#pragma unroll
                for (int j = 0; j < kBatch; ++j) v[u][j] = __ldcg(x + j * S::kThreads);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const float f = w_s[(k0 + u) * S::kRows + (i0 + j * S::kThreads) / (D / 4)];
                    y[j].x = fmaf(f, v[u][j].x, y[j].x);
                    y[j].y = fmaf(f, v[u][j].y, y[j].y);
                    y[j].z = fmaf(f, v[u][j].z, y[j].z);
                    y[j].w = fmaf(f, v[u][j].w, y[j].w);
                }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * S::kThreads, r = i / (D / 4);
            if (!final) {
                reinterpret_cast<float4*>(sp.o + static_cast<size_t>(to) * S::kRows * D)[i] = y[j];
            } else if (r < rows) {
                const float ll = t_s[r].y, inv = ll == 0.f ? 0.f : 1.0f / ll;
                put<Ta, D>(p, out_bf16, b, hk, row0 + r, i % (D / 4) * 4, times(y[j], inv));
            }
        }
    }
    sync_computing<S>();
}

template <class S>
__device__ __forceinline__ Split split_of(const AttnParams& p) {
    uint8_t* const w = static_cast<uint8_t*>(p.workspace);
    return {reinterpret_cast<int*>(w), reinterpret_cast<float*>(w + kCounterBytes),
            reinterpret_cast<float2*>(w + kCounterBytes + static_cast<size_t>(2) * gridDim.x * S::kRows * S::D * 4)};
}

// A CTA's share: numbers [first, last) of the `total` of all groups, which `ctas` CTAs divide.
struct Share {
    long long first, last, total;
    int ctas;
};
struct PlanSmem {
    long long sums[16], start;   // by warp
    int start_b;
};

// This CTA's share and where it begins (c.at >= last where it holds no tile); false if it has none.  All threads call it.
template <class S>
__device__ __forceinline__ bool my_share(const AttnParams& p, int row_blocks, PlanSmem& sm, Cursor& c, Share& sh) {
    grid_dependency_wait();   // launched as a programmatic dependent: nothing global is touched before the previous kernel is done
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_seq = p.Hkv * row_blocks;   // groups of a sequence
    const int per = (p.B + S::kAll - 1) / S::kAll;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    bool over;
    auto numbers_of = [&](int b) {   // of a sequence's groups
        return static_cast<long long>(tiles_of<S::kTile>(seq_keys(p, b, &over)) + S::kGroupCost) * per_seq;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += numbers_of(b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm.sums[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < S::kAll / 32; ++w) {
        if (w < warp) before += sm.sums[w];
        total += sm.sums[w];
    }
    before += incl - mine;
    sh.total = total;
    sh.ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
    if (static_cast<int>(blockIdx.x) >= sh.ctas) return false;
    sh.first = quot(total * blockIdx.x, sh.ctas);
    sh.last = quot(total * (blockIdx.x + 1), sh.ctas);
    if (sh.first >= before && sh.first < before + mine) {   // one thread: its sequences hold the first number
        long long at = before;
        int b = b0;
        for (; b < b1; ++b) {
            const long long n = numbers_of(b);
            if (sh.first < at + n) break;
            at += n;
        }
        sm.start_b = b;
        sm.start = at;
    }
    __syncthreads();
    grid_launch_dependents();
    c.b = sm.start_b;
    c.len = seq_keys(p, c.b, &over);
    c.tiles = tiles_of<S::kTile>(c.len);
    const int size = c.tiles + S::kGroupCost;
    const long long in_seq = sh.first - sm.start;
    const int group = static_cast<int>(quot(in_seq, size));
    c.tile = static_cast<int>(in_seq - static_cast<long long>(group) * size);
    c.hk = group / row_blocks;
    c.rb = group - c.hk * row_blocks;
    c.at = sh.first;
    if (c.tile >= c.tiles) {   // among the numbers without a tile: the next group is the first
        c.at += size - c.tile;
        next_group<S>(p, c, row_blocks);
    }
    return true;
}

// After this CTA's part of a split group is written: join what is complete.  The CTAs c0.. of the group hold its n parts;
// the first one's lies in either of that CTA's two places.  Up to kFanOne parts are joined by the CTA that arrives
// last; of more, `fan` neighbours each are joined that way into the first one's place, and the results of those
// again: few parts for one CTA to read, and no CTA waits.  What is joined with what, and in which order, does not
// depend on who arrives last.  `strays`: this CTA has found some, of this part or another.  *flag_s is then kFinished where this CTA
// has written the results, and kStrays besides where the CTA of any part has found some.
template <class S>
__device__ __forceinline__ void join_group(const AttnParams& p, bool out_bf16, const Split& sp, const Share& sh, const Cursor& cc,
                                           long long g_first, long long g_last, int rows, float* join_s, const int* strays, int* flag_s) {
    const int c0 = static_cast<int>(quot((g_first + 1) * sh.ctas - 1, sh.total)), c1 = static_cast<int>(quot(g_last * sh.ctas - 1, sh.total));
    const int n = c1 - c0 + 1, fan = n <= kFanOne ? kFanOne : n <= 64 ? 8 : 12;
    const int k0 = (static_cast<int>(blockIdx.x) - c0) / fan * fan;   // this CTA's neighbours are k0..
    const int part0 = 2 * c0 + (quot(sh.total * c0, sh.ctas) >= g_first - S::kGroupCost ? 0 : 1);   // no tile of the group before in that CTA
    auto place = [&](int k) { return k == 0 ? part0 : 2 * (c0 + k); };
    if (threadIdx.x == 0) *flag_s = *strays ? kStrays : 0;
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
        const int from = level == 0 ? k0 : 0, stride = level == 0 ? 1 : fan;
        const int count = level == 0 ? min(fan, n - k0) : (n + fan - 1) / fan;
        const bool final = level == 1 || n <= fan;
        if (level == 0 && count == 1) continue;   // already where level 1 reads it
        sync_computing<S>();   // this CTA's part is written
        if (threadIdx.x == 0) {
            int* const counter = level == 0 ? sp.counters + place(k0) : sp.counters + 2 * kMaxCtas + c0;
            // releases what the CTA wrote, acquires what the others did; counts the parts, and above them those with strays; the
            // last one leaves zero for the next call
            unsigned old;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(*flag_s & kStrays ? kStrayPart + 1 : 1) : "memory");
            const bool is_last = old % kStrayPart == static_cast<unsigned>(count - 1);
            if (is_last) *counter = 0;
            *flag_s = (*flag_s & kStrays) | (old >= kStrayPart ? kStrays : 0) | (is_last ? kFinished : 0);
        }
        sync_computing<S>();
        if (!(*flag_s & kFinished)) return;
        join_parts<S>(p, out_bf16, sp, rows, cc.b, cc.hk, cc.rb * S::kRows, join_s, count, final, place(k0),
                      [&](int k) { return static_cast<size_t>(place(from + k * stride)) * S::kRows; });
        if (final) return;
    }
}

// kTokens: more than one token a sequence, so that some rows may not see a key that others do.
template <class S, bool kTokens>
__global__ void __launch_bounds__(S::kAll, 1) attn_decode_kernel(const AttnParams p, const int out_bf16) {
    using Ta = typename S::Ta;
    constexpr int D = S::D, NT = S::NT, RG = S::RG, KG = S::KG, KT = S::KT, PW = S::PW, kTile = S::kTile;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const q_s = smem + KG * kStages * S::kStageBytes;
    float* const join_s = reinterpret_cast<float*>(q_s + S::kQBytes);
    float2* const ml_s = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(join_s) + S::kJoinBytes);   // [KG][kRows]
    uint64_t* const full_s = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ml_s) + S::kMlBytes);   // [KG][kStages]
    uint64_t* const empty_s = full_s + KG * kStages;
    uint64_t* const never_s = empty_s + KG * kStages;
    volatile uint32_t* const valid_s = reinterpret_cast<uint32_t*>(never_s + 1);   // [KG][kStages][PW]
    __shared__ PlanSmem plan_s;
    __shared__ int flag_s, stop_s, strays_s;   // stop: a computing warp has missed a stage, strays: some were found; never taken back
    __shared__ volatile int abort_s;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.G * p.K, row_blocks = (R + S::kRows - 1) / S::kRows;

    if (threadIdx.x < KG * kStages) {
        tc::mbar_init(full_s + threadIdx.x, PW * 33);   // each loading lane's copies, and one arrival a warp for the valid word
        tc::mbar_init(empty_s + threadIdx.x, RG);
    }
    if (threadIdx.x == 0) {
        tc::mbar_init(never_s, 1);
        abort_s = 0;
        stop_s = strays_s = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");   // the barriers are there before asynchronous arrivals on them
    Cursor cc;
    Share sh;
    if (!my_share<S>(p, row_blocks, plan_s, cc, sh)) return;   // (an exit lets the next kernel start, too)
    const long long last = sh.last;
    bool over;

    // ---------------------------------------------------------------- the loading warps
    if (warp >= RG * KG) {
        if constexpr (S::kMoveRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        constexpr int kKeys = KT / PW;   // keys of a stage that one warp loads; lane l knows key l's page
        const int kg = (warp - RG * KG) / PW, pw = (warp - RG * KG) % PW;
        const uint32_t ring = smem_u32(smem) + kg * kStages * S::kStageBytes;
        const int ps = p.cache.page_size;
        // pages are looked up two tiles ahead of their keys' loads: turn t looks up tile t and loads tile t - 2
        int page[2] = {0, 0}, in_page[2] = {0, 0}, head[2] = {0, 0}, seq[2] = {-1, -1};   // seq -1: no key
        int tiles = 0, slot = 0;   // tiles: looked up so far
        uint32_t round = 0;
#pragma unroll 1
        for (int t = 0;; ++t) {
            const int pg = page[0], pg_seq = seq[0];
            const bool pg_late = kTokens && (head[0] & kLate) != 0;
            const long long off = pg * p.cache.page_stride + in_page[0] * p.cache.token_stride + (kTokens ? head[0] & (kLate - 1) : head[0]) * p.cache.head_stride;
            page[0] = page[1];
            in_page[0] = in_page[1];
            head[0] = head[1];
            seq[0] = seq[1];
            seq[1] = -1;
            if (cc.at < last) {
                const int j = cc.tile * kTile + kg * KT + pw * kKeys + lane;
                if (lane < kKeys && j < cc.len) {
                    const int k = j / ps;
                    in_page[1] = j - k * ps;
                    head[1] = kTokens && j > cc.len - p.K ? cc.hk | kLate : cc.hk;
                    seq[1] = cc.b;
                    page[1] = p.block_table[static_cast<size_t>(cc.b) * p.max_pages + k];   // looked at when it is used
                }
                advance<S>(p, cc, row_blocks);
                ++tiles;
            }
            if (t < 2) continue;
            if (t - 2 >= tiles) break;
            if (round > 0 && !warp_wait(empty_s + kg * kStages + slot, (round - 1) & 1, &abort_s)) break;
            const bool in_cache = pg >= 0 && pg < p.cache.num_pages;
            const uint32_t ok = __ballot_sync(0xffffffffu, pg_seq >= 0 && in_cache);
            if (pg_seq >= 0 && !in_cache && p.status) atomicOr(p.status + pg_seq, kKvBadIndex);
            if (lane == 0) valid_s[(kg * kStages + slot) * PW + pw] = ok;
            constexpr int kChunks = S::kRowBytes / 16;   // of a row
            const uint32_t st = ring + slot * S::kStageBytes;
            const uint32_t late = kTokens ? __ballot_sync(0xffffffffu, pg_late) & ok : 0u;
            bool strays = false;
            if (kTokens && late) strays = find_strays<Ta, kChunks>(static_cast<const Ta*>(p.cache.v), off, late);
            // Copies unrolled in full, but for bf16 heads of 128 with several tokens, where the loading warps' registers do not suffice for
            // that: 64 ragged sequences, 3 tokens 110 us against 138, 2 tokens 97 against 110; heads of 256 108.8 in fours against 108.1,
            // of 64 139 against 137, one token 173 either way.
            constexpr int kUnroll = kTokens && S::kBf16 && D == 128 ? 4 : 16;
#pragma unroll kUnroll
            for (int it = 0; it < kKeys * kChunks / 32; ++it) {
                const int flat = it * 32 + lane;
                const int key = flat / kChunks, ch = flat % kChunks;
                const long long o = __shfl_sync(0xffffffffu, off, key) + ch * (16 / static_cast<int>(sizeof(Ta)));
                const int n = (ok >> key) & 1 ? 16 : 0;
                const int row = pw * kKeys + key;
                const uint32_t dst = st + row * S::kRowBytes + (S::kBf16 ? (ch ^ (row & 7)) : ch) * 16;
                tc::cp_async16_zfill(dst, static_cast<const Ta*>(p.cache.k) + (n ? o : 0), n);
                tc::cp_async16_zfill(dst + S::kHalfBytes, static_cast<const Ta*>(p.cache.v) + (n ? o : 0), n);
            }
            if (kTokens && strays) {
                tc::cp_async_wait_all();
#pragma unroll 1
                for (int it = 0; it < kKeys * kChunks / 32; ++it) {
                    const int key = (it * 32 + lane) / kChunks, ch = (it * 32 + lane) % kChunks, row = pw * kKeys + key;
                    if ((late >> key) & 1)   // what this lane has copied
                        take_strays<Ta>(smem + (kg * kStages + slot) * S::kStageBytes + S::kHalfBytes + row * S::kRowBytes + (S::kBf16 ? (ch ^ (row & 7)) : ch) * 16);
                }
                strays_s = 1;
                __syncwarp();   // before lane 0's arrival
            }
            tc::cp_async_mbar_arrive(full_s + kg * kStages + slot);
            if (lane == 0) tc::mbar_arrive(full_s + kg * kStages + slot);
            if (++slot == kStages) {
                slot = 0;
                ++round;
            }
        }
        tc::cp_async_wait_all();   // nothing of a call that gives up is in flight when the CTA ends
        return;
    }

    // ---------------------------------------------------------------- the computing warps
    if constexpr (S::kMoveRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegs));
    const int kg = warp / RG, rg = warp % RG;
    const uint32_t ring = smem_u32(smem) + kg * kStages * S::kStageBytes;

    // ---------------------------------------------------------------- state of a row set
    // bf16: o[mt][nt] is the 16 x 8 fragment (channels 16 mt.., rows 8 nt..) of o transposed; this thread has rows
    // 8 nt + 2 (lane%4) + {0,1}.  fp32: lane l has all FR rows, the channels of qf.
    constexpr int FR = S::kWarpRows, kCols = S::kBf16 ? NT * 2 : FR;
    constexpr int kC = D / 32;
    float o[S::kBf16 ? D / 16 * NT : FR][S::kBf16 ? 4 : kC];
    float m[kCols], l[kCols];
    float qf[S::kBf16 ? 1 : FR][kC];
    // keys that row i of this warp's rows sees
    auto limit = [&](int i) {
        const int row = cc.rb * S::kRows + rg * S::kWarpRows + i;
        return row < R ? cc.len - p.K + token_of(p, row) + 1 : 0;
    };
    // the fp32 kernel's channels of a lane: kV consecutive ones every 32 kV
    constexpr int kV = kC < 4 ? kC : 4;

    auto begin_segment = [&]() {
        auto stall = [&]() {   // here, where few registers are in use
            if (p.test_stall && warp == RG * KG - 1 && !stage_wait(never_s, 0, &abort_s, 256)) stop_s = 1;
        };
        const Ta* q = static_cast<const Ta*>(p.q) + static_cast<long long>(cc.b) * p.K * p.ldq + static_cast<long long>(cc.hk) * p.G * D;
        const int row0 = cc.rb * S::kRows;
        if constexpr (S::kBf16) {
            constexpr int kChunks = S::kRowBytes / 16;
            for (int i = threadIdx.x; i < S::kRows * kChunks; i += S::kThreads) {
                const int r = i / kChunks, ch = i % kChunks, row = row0 + r;
                uint4 v = make_uint4(0, 0, 0, 0);
                const int tok = token_of(p, row);
                if (row < R) v = *reinterpret_cast<const uint4*>(q + tok * p.ldq + (row - tok * p.G) * D + ch * 8);
                *reinterpret_cast<uint4*>(q_s + r * S::kRowBytes + (ch ^ (r & 7)) * 16) = v;
            }
            sync_computing<S>();
            stall();
        } else {
            stall();
#pragma unroll
            for (int r = 0; r < FR; ++r) {
                const int row = row0 + rg * FR + r, tok = token_of(p, row);
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    qf[r][c] = row < R ? q[tok * p.ldq + (row - tok * p.G) * D + (c / kV) * 32 * kV + lane * kV + c % kV] *
                                             (p.scale * kLog2e)
                                       : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (auto& x : o)
#pragma unroll
            for (float& y : x) y = 0.f;
    };

    // ---------------------------------------------------------------- one stage
    int slot = 0;
    auto compute = [&]() {
        const uint32_t st = ring + slot * S::kStageBytes;
        const int j0 = cc.tile * kTile + kg * KT;   // the stage's first key
        uint32_t ok = 0;
#pragma unroll
        for (int w = 0; w < PW; ++w) ok |= valid_s[(kg * kStages + slot) * PW + w] << (w * (KT / PW));
        constexpr uint32_t kFull = KT == 32 ? 0xffffffffu : (1u << (KT & 31)) - 1;
        if (ok == 0) return;
        const bool masked = ok != kFull || j0 + KT > cc.len - p.K + 1;
        if constexpr (S::kBf16) {
            constexpr int SUB = KT / 16;
            float s[SUB][NT][4];
            // s transposed: keys x rows = K . Q^T.  A 16-byte chunk c of row r lies at c ^ (r % 8): with c = c0 + c1, c0 a
            // constant whose bits c1 (of the lane) lacks, that is the lane's (c1 ^ r%8) with c0's low bits flipped, so four
            // addresses and constant offsets reach all chunks.
            const int key = lane & 15;
            const uint32_t qa = smem_u32(q_s) + (rg * 8 * NT + (lane & 7)) * S::kRowBytes + ((lane >> 3) ^ (lane & 7)) * 16;
            const uint32_t ka = st + key * S::kRowBytes + ((lane >> 4) ^ (key & 7)) * 16;
            constexpr int kSplit = SUB * NT >= 4 ? 1 : 2;   // independent sums, for the latency of a product
            float s2[kSplit][SUB][NT][4] = {};
            constexpr int kKs = SUB == 1 ? 4 : 2;   // steps whose operands are loaded together
#pragma unroll
            for (int k0 = 0; k0 < D / 16; k0 += kKs) {
                uint32_t qb[kKs / 2][NT][4], a[kKs][SUB][4];
#pragma unroll
                for (int i = 0; i < kKs; ++i) {
                    const int ks = k0 + i;
                    if (i % 2 == 0)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            ldsm4((qa ^ ((2 * ks & 4) * 16)) + (2 * ks & ~7) * 16 + n * 8 * S::kRowBytes, qb[i / 2][n]);
#pragma unroll
                    for (int u = 0; u < SUB; ++u) ldsm4((ka ^ ((2 * ks & 6) * 16)) + (2 * ks & ~7) * 16 + u * 16 * S::kRowBytes, a[i][u]);
                }
#pragma unroll
                for (int i = 0; i < kKs; ++i)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(s2[i % kSplit][u][n], a[i][u], qb[i / 2][n][i % 2 * 2], qb[i / 2][n][i % 2 * 2 + 1]);
            }
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][n][e] = kSplit == 2 ? s2[0][u][n][e] + s2[kSplit - 1][u][n][e] : s2[0][u][n][e];
            const float c = p.scale * kLog2e;
            float mx[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mx[n][0] = mx[n][1] = -INFINITY;
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[u][n][e] * c;
                        if (masked) {
                            const int k = u * 16 + (lane >> 2) + (e & 2) * 4;
                            if (!((ok >> k) & 1) || j0 + k >= limit(n * 8 + (lane & 3) * 2 + (e & 1))) x = -INFINITY;
                        }
                        s[u][n][e] = x;
                        mx[n][e & 1] = fmaxf(mx[n][e & 1], x);
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], d));
            }
            bool up = false;
            float f[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float m2 = fmaxf(m[n * 2 + e], mx[n][e]);
                    up |= m2 > m[n * 2 + e];
                    const float base = m2 == -INFINITY ? 0.f : m2;   // a row that has seen no key
                    f[n][e] = ex2(m[n * 2 + e] - base);
                    m[n * 2 + e] = m2;
                    mx[n][e] = base;
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    l[n * 2] *= f[n][0];
                    l[n * 2 + 1] *= f[n][1];
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt * NT + n][e] *= f[n][e & 1];
                }
            }
            // The weights go to the tensor cores as PIECES bf16 parts, each the rounding of what the ones before
            // leave: two give 2^-17, below a bf16 result's own rounding; three all of an fp32 weight's bits.
            uint32_t pb[SUB][NT][S::PIECES][2];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = ex2(s[u][n][e] - mx[n][e & 1]);
                        l[n * 2 + (e & 1)] += w[e];
                    }
#pragma unroll
                    for (int i = 0; i < S::PIECES; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = StateIO<__nv_bfloat16>::pack(w[2 * h], w[2 * h + 1]);
                            if (i + 1 < S::PIECES) {
                                w[2 * h] -= __uint_as_float(x << 16);
                                w[2 * h + 1] -= __uint_as_float(x & 0xffff0000u);
                            }
                            pb[u][n][i][h] = movm(x);
                        }
                }
            // o transposed: channels x rows += V^T . P^T
            const uint32_t va = st + S::kHalfBytes + ((lane & 7) + (lane >> 4) * 8) * S::kRowBytes + (((lane >> 3) & 1) ^ (lane & 7)) * 16;
            // The tensor cores' sums drop what is below the last bit, always downwards in magnitude: over a long sequence that
            // adds up (16,000 keys: 1.3e-5 of the result, and 0.29% of bf16 results not the nearest ones, against 0.19% with sums
            // apart and 0.11% in fp32 throughout; 64 sequences of up to 16,384 keys).  So a stage is summed by itself and then
            // added with a rounding that goes both ways, where the result is fp32, and where up to 8 rows make it free (heads of
            // 256, 64 ragged sequences, 91.1 us against 91.3).  bf16 results of more rows keep the one running sum, whose drift
            // is a hundredth of their own rounding: 16 rows took 94.8 us against 94.6 (heads of 64 118 against 114), 24
            // rows 110.8 against 105.6, 32 rows 144 against 124.
            constexpr bool kApart = S::PIECES == 3 || RG * NT == 1;
            constexpr int kMt = SUB == 1 && !kApart ? 4 : 2;   // as kKs above
#pragma unroll
            for (int m0 = 0; m0 < D / 16; m0 += kMt) {
                uint32_t a[kMt][SUB][4];
                float sum[kMt][NT][4];
#pragma unroll
                for (int i = 0; i < kMt; ++i)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
                        ldsm4t((va ^ ((2 * (m0 + i) & 6) * 16)) + (2 * (m0 + i) & ~7) * 16 + u * 16 * S::kRowBytes, a[i][u]);
                if constexpr (kApart) {
#pragma unroll
                    for (int i = 0; i < kMt; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[i][n][e] = 0.f;
                }
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int q = 0; q < S::PIECES; ++q)
#pragma unroll
                        for (int i = 0; i < kMt; ++i)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma16816(kApart ? sum[i][n] : o[(m0 + i) * NT + n], a[i][u], pb[u][n][q][0], pb[u][n][q][1]);
                if constexpr (kApart) {
#pragma unroll
                    for (int i = 0; i < kMt; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[(m0 + i) * NT + n][e] += sum[i][n][e];
                }
            }
        } else {
            // fp32 products and sums on the CUDA cores: 4 keys x 8 rows (8 x 4, 16 x 2) at a time, the channels over the lanes; two such sets
            // side by side where the registers allow, since a warp has its scheduler to itself
            constexpr int SK = 32 / FR, U = D <= 128 && KT >= 2 * SK ? 2 : 1;   // keys of a set, sets
            const float* ks = reinterpret_cast<const float*>(smem + (kg * kStages + slot) * S::kStageBytes) + lane * kV;
            const float* vs = ks + S::kHalfBytes / 4;
            const int r = lane % FR;
#pragma unroll 1
            for (int k0 = 0; k0 < KT; k0 += SK * U) {
                float s[U], mx = -INFINITY;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float part[32];
#pragma unroll
                    for (int k = 0; k < SK; ++k) {
                        float kv[kC];
#pragma unroll
                        for (int c = 0; c < kC; c += kV)
#pragma unroll
                            for (int i = 0; i < kV; ++i) kv[c + i] = ks[(k0 + SK * u + k) * D + c / kV * 32 * kV + i];
#pragma unroll
                        for (int rr = 0; rr < FR; ++rr) {
                            float2 x = mul2(make_float2(kv[0], kv[1]), make_float2(qf[rr][0], qf[rr][1]));
#pragma unroll
                            for (int c = 2; c < kC; c += 2)
                                x = fma2(make_float2(kv[c], kv[c + 1]), make_float2(qf[rr][c], qf[rr][c + 1]), x);
                            part[k * FR + rr] = x.x + x.y;   // (two sums a row, of even and odd channels)
                        }
                    }
                    s[u] = reduce32_transposed(part);   // key k0 + SK u + lane / FR, row lane % FR
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int kk = k0 + SK * u + lane / FR;
                    if (masked && (!((ok >> kk) & 1) || j0 + kk >= limit(r))) s[u] = -INFINITY;
                    mx = fmaxf(mx, s[u]);
                }
#pragma unroll
                for (int d = FR; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                float mine_m = m[0];
#pragma unroll
                for (int i = 1; i < FR; ++i) mine_m = r == i ? m[i] : mine_m;
                const float m2 = fmaxf(mine_m, mx), base = m2 == -INFINITY ? 0.f : m2;
                float w[U], lsum = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    w[u] = ex2(s[u] - base);
                    lsum += w[u];
                }
#pragma unroll
                for (int d = FR; d < 32; d <<= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, d);
                if (__any_sync(0xffffffffu, m2 > mine_m)) {
                    const float f = ex2(mine_m - base);
#pragma unroll
                    for (int i = 0; i < FR; ++i) {
                        m[i] = __shfl_sync(0xffffffffu, m2, i);
                        const float fi = __shfl_sync(0xffffffffu, f, i);
                        l[i] *= fi;
#pragma unroll
                        for (int c = 0; c < kC; ++c) o[i][c] *= fi;
                    }
                }
#pragma unroll
                for (int i = 0; i < FR; ++i) l[i] += __shfl_sync(0xffffffffu, lsum, i);
#pragma unroll
                for (int k = 0; k < SK * U; ++k) {
                    float kv[kC];
#pragma unroll
                    for (int c = 0; c < kC; c += kV)
#pragma unroll
                        for (int i = 0; i < kV; ++i) kv[c + i] = vs[(k0 + k) * D + c / kV * 32 * kV + i];
#pragma unroll
                    for (int rr = 0; rr < FR; ++rr) {
                        const float wr = __shfl_sync(0xffffffffu, w[k / SK], k % SK * FR + rr);
#pragma unroll
                        for (int c = 0; c < kC; c += 2) {
                            const float2 x = fma2(make_float2(wr, wr), make_float2(kv[c], kv[c + 1]), make_float2(o[rr][c], o[rr][c + 1]));
                            o[rr][c] = x.x;
                            o[rr][c + 1] = x.y;
                        }
                    }
                }
            }
        }
    };

    // ---------------------------------------------------------------- the end of a group, or of this CTA's part of it
    const Split sp = split_of<S>(p);
    long long seg_first = cc.at;   // this CTA's first tile of the group
    bool first_seg = true;         // of this CTA
    auto end_segment = [&]() {     // the tiles from seg_first up to and with cc's are done
        const long long g_first = cc.at - cc.tile, g_last = g_first + cc.tiles;   // the group's tiles
        const bool whole = seg_first == g_first && cc.at + 1 == g_last;
        const int part = 2 * blockIdx.x + (first_seg ? 0 : 1);
        if constexpr (S::kBf16) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        }
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            if constexpr (S::kBf16) {
                if (lane < 4) ml_s[kg * S::kRows + rg * 8 * NT + (i / 2) * 8 + lane * 2 + (i & 1)] = make_float2(m[i], l[i]);
            } else {
                if (lane == i) ml_s[kg * S::kRows + rg * FR + i] = make_float2(m[i], l[i]);
            }
        }
        const int rows = min(S::kRows, R - cc.rb * S::kRows);
        constexpr int kHalves = D / S::JC, PR = S::kPassRows;
#pragma unroll 1
        for (int pass = 0; pass < RG * NT * kHalves; ++pass) {
            const int ch0 = pass % kHalves * S::JC, r0 = pass / kHalves * PR;
            if (r0 >= rows) break;
            if (pass / (NT * kHalves) == rg) {
                const int mine_pass = pass % (NT * kHalves);
                if constexpr (S::kBf16) {
                    float* w = join_s + (kg * 8 + (lane & 3) * 2) * S::kJPitch + (lane >> 2);
#pragma unroll
                    for (int q = 0; q < NT * kHalves; ++q)   // every index of o is a constant
                        if (q == mine_pass)
#pragma unroll
                            for (int mt = 0; mt < S::JC / 16; ++mt) {
                                const float(&x)[4] = o[(q % kHalves * (S::JC / 16) + mt) * NT + q / kHalves];
                                w[mt * 16] = x[0];
                                w[mt * 16 + S::kJPitch] = x[1];
                                w[mt * 16 + 8] = x[2];
                                w[mt * 16 + 8 + S::kJPitch] = x[3];
                            }
                } else {
#pragma unroll
                    for (int r = 0; r < PR; ++r)
#pragma unroll
                        for (int c = 0; c < kC; ++c)
                            if (c / kV * 32 * kV / S::JC == mine_pass)
                                join_s[(kg * PR + r) * S::kJPitch + c / kV * 32 * kV % S::JC + lane * kV + c % kV] = o[r][c];
                }
            }
            sync_computing<S>();
            if (stop_s) {   // a wait gave up: nothing of this group is written
                if (threadIdx.x == 0 && p.status) atomicOr(p.status + cc.b, 16);
                return;
            }
#pragma unroll 1   // code that runs once costs its fetch
            for (int i = threadIdx.x; i < PR * S::JC / 4; i += S::kThreads) {
                const int r = i / (S::JC / 4), ch = i % (S::JC / 4) * 4, row = r0 + r;
                if (row >= rows) break;
                float mm = -INFINITY, ll = 0.f;
#pragma unroll
                for (int k = 0; k < KG; ++k) mm = fmaxf(mm, ml_s[k * S::kRows + row].x);
                const float base = mm == -INFINITY ? 0.f : mm;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < KG; ++k) {
                    const float2 t = ml_s[k * S::kRows + row];
                    const float f = ex2(t.x - base);
                    const float4 x = *reinterpret_cast<const float4*>(join_s + (k * PR + r) * S::kJPitch + ch);
                    ll = fmaf(f, t.y, ll);
                    y.x = fmaf(f, x.x, y.x);
                    y.y = fmaf(f, x.y, y.y);
                    y.z = fmaf(f, x.z, y.z);
                    y.w = fmaf(f, x.w, y.w);
                }
                if (whole) {
                    put<Ta, D>(p, out_bf16, cc.b, cc.hk, cc.rb * S::kRows + row, ch0 + ch, times(y, ll == 0.f ? 0.f : 1.0f / ll));
                } else {
                    *reinterpret_cast<float4*>(sp.o + (static_cast<size_t>(part) * S::kRows + row) * D + ch0 + ch) = y;
                    if (ch0 + ch == 0) sp.ml[static_cast<size_t>(part) * S::kRows + row] = make_float2(mm, ll);
                }
            }
            sync_computing<S>();
        }
        if (!whole) join_group<S>(p, out_bf16, sp, sh, cc, g_first, g_last, rows, join_s, &strays_s, &flag_s);
        if (kTokens && (whole ? strays_s : flag_s == (kFinished | kStrays))) {   // of this group, or of another in one of its CTAs
#pragma unroll 1
            for (int i = threadIdx.x; i < rows * (D / 4); i += S::kThreads) {
                const int row = i / (D / 4), c = i % (D / 4) * 4;
                const float4 x = strays_of<Ta>(p, cc.b, cc.hk, cc.len, cc.rb * S::kRows + row, c);
                if (x.x == 0.f && x.y == 0.f && x.z == 0.f && x.w == 0.f) continue;
                put<Ta, D, true>(p, out_bf16, cc.b, cc.hk, cc.rb * S::kRows + row, c, x);
            }
        }
    };

    // ---------------------------------------------------------------- the walk (one copy of each part: the code is fetched
    // anew by every launch)
    bool fresh = true, new_seq = cc.tile == 0 && cc.hk == 0 && cc.rb == 0;
    uint32_t phase = 0;
#pragma unroll 1
    while (cc.at < last) {
        if (fresh) {
            begin_segment();
            if (new_seq && threadIdx.x == 0 && p.status) {
                seq_keys(p, cc.b, &over);
                if (over) atomicOr(p.status + cc.b, kKvBadIndex);
            }
            fresh = false;
        }
        if (warp_wait(full_s + kg * kStages + slot, phase, &abort_s)) compute();
        else stop_s = 1;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty_s + kg * kStages + slot);
        if (++slot == kStages) {
            slot = 0;
            phase ^= 1;
        }
        const bool group_done = cc.tile + 1 == cc.tiles;
        if (group_done || cc.at + 1 == last) {
            end_segment();
            first_seg = false;
        }
        const int b = cc.b;
        advance<S>(p, cc, row_blocks);
        if (group_done) {
            new_seq = cc.b != b;
            fresh = true;
            seg_first = cc.at;
        }
    }
}

template <class S, bool kTokens>
cudaError_t launch_as(const AttnParams& p, bool out_bf16, int sms, cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<S, kTokens>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_decode_kernel<S, kTokens>, dim3(sms), dim3(S::kAll), S::kSmem, stream, p, out_bf16 ? 1 : 0);
}

template <class S>
cudaError_t launch(const AttnParams& p, bool out_bf16, int sms, cudaStream_t stream) {
    if constexpr (S::kRows <= 16)   // more rows have several tokens: a kv head has at most 16 query heads
        if (p.K == 1) return launch_as<S, false>(p, out_bf16, sms, stream);
    return launch_as<S, true>(p, out_bf16, sms, stream);
}

// CTAs of a launch: one per SM (0 if the device cannot be asked).
inline int grid_ctas() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms < kMaxCtas ? sms : kMaxCtas;
}

cudaError_t launch_bf16(const AttnParams& p, int head_dim, bool out_bf16, int sms, cudaStream_t stream);
cudaError_t launch_tc(const AttnParams& p, int head_dim, int sms, cudaStream_t stream);
cudaError_t launch_f32(const AttnParams& p, int head_dim, bool out_bf16, int sms, cudaStream_t stream);

// Rows of a block for R rows a kv head.
inline int block_rows(int R, bool bf16) {
    const int most = bf16 ? 128 : 64;
    int n = 8;
    while (n < R && n < most) n *= 2;
    return n;
}

}  // namespace attn
}  // namespace gdn
