// gdn_chunk_simt.cu -- gdn_attn_chunk in fp32 on the CUDA cores: fp32 caches, and bf16 ones that have no tensor map (strides that
// none can have; with fp32 results pages of an odd number of tokens: 4 x 1,024 tokens behind 1,024, 16/2 heads of 256, 2,690
// us, on the tensor cores with pages of 16 422).
//
// Bound by the products: 2 d operations a row and key for the scores and as many for the result, of which an SM has 128 multiply-adds
// a cycle.  9 ragged sequences of up to 301 tokens behind 1,500, 6/3 heads of 64, take 77 us (23 TFLOP/s), 1,281 tokens with 32/4
// heads of 256 820 (33 TFLOP/s); ncu: warps wait for shared memory first, then for the fixed latency of the products.
#include "gdn_chunk.cuh"

namespace gdn {
namespace chunk {

namespace {

constexpr int kRt = 64, kKt = 64, kThreads = 256;   // rows of a unit, keys of a tile

// A CTA is a worker.  A thread has 4 rows (4 ty ..) and, of the scores, keys tx + 16 c, of the result channels 4 tx + 64 c; its
// 16 neighbours have the same rows.  Keys and values each have one buffer: a tile's keys are asked for while the products with
// the values before them run, and the values while the scores are computed.
template <typename Ta_, int D_>
struct Simt {
    using Ta = Ta_;
    static constexpr int D = D_, kEs = static_cast<int>(sizeof(Ta));
    static constexpr int kPitch = D * kEs + 16;        // bytes of a row of queries or keys: 16-byte accesses of 8 rows hit all banks
    static constexpr int kV = kKt * D * kEs, kPp = kKt + 4;
    static constexpr int kSmem = 2 * kRt * kPitch + kV + kRt * kPp * 4;
    static constexpr int kCtas = kSmem * 2 <= 224 * 1024 ? 2 : 1;   // an SM
    static constexpr int kCost = 64;   // of a unit, in keys (the first case above: 128 82 us, 32 81)
};

// n = 8 (bf16) or 4 elements of 16 bytes.
__device__ __forceinline__ void unpack16(const uint4& w, float (&v)[8], const __nv_bfloat16*) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(x[i] << 16);
        v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack16(const uint4& w, float (&v)[4], const float*) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
}

template <class S>
__global__ void __launch_bounds__(kThreads, S::kCtas) chunk_simt_kernel(const __grid_constant__ ChunkParams p, const bool out_bf16) {
    using Ta = typename S::Ta;
    constexpr int D = S::D, kE = 16 / S::kEs;   // elements of 16 bytes
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const q_s = smem;
    uint8_t* const k_s = q_s + kRt * S::kPitch;
    uint8_t* const v_s = k_s + kKt * S::kPitch;
    float* const p_s = reinterpret_cast<float*>(v_s + S::kV);
    __shared__ PlanSmem plan_s;
    __shared__ uint8_t there_s[2][kKt];
    __shared__ int last_s;
    const Line ln{kRt / p.G, 6, S::kCost};
    static_assert(kKt == 1 << 6, "keys of a tile");
    Share sh;
    Part c;
    const int worker = static_cast<int>(blockIdx.x);
    if (!my_share(p, ln, worker, static_cast<int>(gridDim.x), 2 * kKt, plan_s, sh, c)) return;
    const Parts<kRt, D> parts(p.workspace, static_cast<int>(gridDim.x));
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float scale = p.scale * kLog2e;
    // this thread's key of a tile, a quarter of its channels
    const int my_key = threadIdx.x >> 2, quarter = threadIdx.x & 3;
    auto load_rows = [&](const void* half, long long off, bool there, uint8_t* to) {
        const Ta* const src = static_cast<const Ta*>(half) + (there ? off : 0);
#pragma unroll
        for (int x = quarter; x < D / kE; x += 4) tc::cp_async16_zfill(to + x * 16, src + x * kE, there ? 16u : 0u);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    do {
        const int tok0 = c.i * ln.tokens, n_rows = tokens_of(ln, c) * p.G, off = c.r.len - c.r.n;
        const int end = c.seen;   // keys from here on are nobody's
        long long key_off = 0;
        bool there = false;
        auto look_up = [&](int t) {
            const int j = t * kKt + my_key;
            there = j < end;
            if (there) {
                const int k = j / p.cache.page_size, page = p.block_table[static_cast<size_t>(c.b) * p.max_pages + k];
                there = page >= 0 && page < p.cache.num_pages;
                if (!there && quarter == 0 && p.status) atomicOr(p.status + c.b, kKvBadIndex);
                key_off = page * p.cache.page_stride + (j - k * p.cache.page_size) * p.cache.token_stride + c.hk * p.cache.head_stride;
            }
            if (quarter == 0) there_s[t & 1][my_key] = there;
        };
        for (int x = threadIdx.x; x < kRt * (D / kE); x += kThreads) {
            const int r = x / (D / kE), ch = x % (D / kE) * kE, tok = r / p.G;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < n_rows)
                v = *reinterpret_cast<const uint4*>(static_cast<const Ta*>(p.q) + (c.r.row0 + tok0 + tok) * p.ldq +
                                                    static_cast<long long>(c.hk * p.G + r - tok * p.G) * D + ch);
            *reinterpret_cast<uint4*>(q_s + r * S::kPitch + ch * S::kEs) = v;
        }
        float m[4], l[4];
        int limit[4];   // the first key that a row does not see
        float2 o[4][D / 64][2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
            limit[r] = off + tok0 + (ty * 4 + r) / p.G + 1;
#pragma unroll
            for (int x = 0; x < D / 64; ++x) o[r][x][0] = o[r][x][1] = make_float2(0.f, 0.f);
        }
        if (c.t0 < c.t1) {
            look_up(c.t0);
            load_rows(p.cache.k, key_off, there, k_s + my_key * S::kPitch);
            load_rows(p.cache.v, key_off, there, v_s + my_key * D * S::kEs);
        }
#pragma unroll 1
        for (int t = c.t0; t < c.t1; ++t) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();   // keys are there
            float s[4][4];
            {
                float2 a[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k) a[r][k] = make_float2(0.f, 0.f);
#pragma unroll 4
                for (int x = 0; x < D / kE; ++x) {
                    float q[4][kE], kk[kE];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        unpack16(*reinterpret_cast<const uint4*>(q_s + (ty * 4 + r) * S::kPitch + x * 16), q[r], static_cast<const Ta*>(nullptr));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        unpack16(*reinterpret_cast<const uint4*>(k_s + (tx + 16 * k) * S::kPitch + x * 16), kk, static_cast<const Ta*>(nullptr));
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int e = 0; e < kE; e += 2)
                                a[r][k] = fma2(make_float2(q[r][e], q[r][e + 1]), make_float2(kk[e], kk[e + 1]), a[r][k]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[r][k] = (a[r][k].x + a[r][k].y) * scale;
            }
            __syncthreads();   // the keys have been read
            const bool late = (t + 1) * kKt > off + tok0 + 1;   // some rows do not see some keys
            if (t + 1 < c.t1) {
                look_up(t + 1);
                load_rows(p.cache.k, key_off, there, k_s + my_key * S::kPitch);
            } else {
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float mx = m[r];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = t * kKt + tx + 16 * k;
                    if (j >= limit[r] || !there_s[t & 1][tx + 16 * k]) s[r][k] = -INFINITY;
                    mx = fmaxf(mx, s[r][k]);
                }
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float base = mx == -INFINITY ? 0.f : mx, f = ex2(m[r] - base);
                m[r] = mx;
                l[r] *= f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float w = ex2(s[r][k] - base);
                    l[r] += w;
                    p_s[(ty * 4 + r) * S::kPp + tx + 16 * k] = w;
                }
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    o[r][x][0] = mul2(o[r][x][0], make_float2(f, f));
                    o[r][x][1] = mul2(o[r][x][1], make_float2(f, f));
                }
            }
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            bool stray = false;
            if (late) {   // values of keys that some rows do not see: are all of them finite?
#pragma unroll 1
                for (int x = quarter; x < D / kE; x += 4) stray |= attn::has_strays<Ta>(*reinterpret_cast<const uint4*>(v_s + my_key * D * S::kEs + x * 16));
            }
            stray = __syncthreads_or(stray);   // values and weights are there
            auto add = [&](int r, int x, const float (&v)[4], float w) {
                o[r][x][0] = fma2(make_float2(w, w), make_float2(v[0], v[1]), o[r][x][0]);
                o[r][x][1] = fma2(make_float2(w, w), make_float2(v[2], v[3]), o[r][x][1]);
            };
            auto value = [&](int j, int x, float (&v)[4]) {
                const Ta* const at = reinterpret_cast<const Ta*>(v_s) + j * D + 64 * x + 4 * tx;
                const float4 y = StateIO<Ta>::ld(at);
                v[0] = y.x;
                v[1] = y.y;
                v[2] = y.z;
                v[3] = y.w;
            };
            if (!stray) {
#pragma unroll 1
                for (int j = 0; j < kKt; j += 4) {
                    float4 w[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const float4*>(p_s + (ty * 4 + r) * S::kPp + j);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) {
                            float v[4];
                            value(j + e, x, v);
#pragma unroll
                            for (int r = 0; r < 4; ++r) add(r, x, v, e == 0 ? w[r].x : e == 1 ? w[r].y : e == 2 ? w[r].z : w[r].w);
                        }
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < kKt; ++j)
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        float v[4];
                        value(j, x, v);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (t * kKt + j < limit[r]) add(r, x, v, p_s[(ty * 4 + r) * S::kPp + j]);
                    }
            }
            __syncthreads();   // values and weights have been read
            if (t + 1 < c.t1) load_rows(p.cache.v, key_off, there, v_s + my_key * D * S::kEs);
            else asm volatile("cp.async.commit_group;" ::: "memory");
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        // ------------------------------------------------------------ the unit's end
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
        const bool whole = c.whole();
        const size_t place = parts.place(worker, c);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = ty * 4 + r;
            if (row >= n_rows) continue;
            const int tok = row / p.G, h = c.hk * p.G + row - tok * p.G;
            const float f = l[r] == 0.f ? 0.f : 1.0f / l[r];
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                const float4 y = make_float4(o[r][x][0].x, o[r][x][0].y, o[r][x][1].x, o[r][x][1].y);
                if (whole) put<Ta, D>(p, out_bf16, static_cast<long long>(c.r.row0) + tok0 + tok, h, 64 * x + 4 * tx, attn::times(y, f));
                else *reinterpret_cast<float4*>(parts.o + (place * kRt + row) * D + 64 * x + 4 * tx) = y;
            }
            if (!whole && tx == 0) parts.ml[place * kRt + row] = make_float2(m[r], l[r]);
        }
        if (!whole) {   // the worker that arrives last joins all parts, in their order
            const long long base = c.at + ln.cost;
            const int w0 = sh.owner(base), n = sh.owner(base + static_cast<long long>(kKt) * (c.tiles - 1)) - w0 + 1;
            __syncthreads();
            if (threadIdx.x == 0) {
                unsigned old;
                asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(parts.counters + w0), "r"(n - 1) : "memory");
                last_s = old == static_cast<unsigned>(n - 1);
            }
            __syncthreads();
            if (last_s) {
                auto at = [&](int k) { return (k == 0 ? 2 * static_cast<size_t>(w0) + 1 : 2 * static_cast<size_t>(w0 + k)) * kRt; };
                for (int i = threadIdx.x; i < n_rows * (D / 4); i += kThreads) {
                    const int row = i / (D / 4), ch = i % (D / 4) * 4, tok = row / p.G;
                    float mm = -INFINITY, ll = 0.f;
                    for (int k = 0; k < n; ++k) mm = fmaxf(mm, __ldcg(parts.ml + at(k) + row).x);
                    const float b0 = mm == -INFINITY ? 0.f : mm;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k = 0; k < n; ++k) {
                        const float2 z = __ldcg(parts.ml + at(k) + row);
                        const float f = ex2(z.x - b0);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(parts.o + (at(k) + row) * D + ch));
                        ll = fmaf(f, z.y, ll);
                        y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
                    }
                    const float f = ll == 0.f ? 0.f : 1.0f / ll;
                    put<Ta, D>(p, out_bf16, static_cast<long long>(c.r.row0) + tok0 + tok, c.hk * p.G + row - tok * p.G, ch, attn::times(y, f));
                }
            }
        }
        __syncthreads();
    } while (to_next_part(p, ln, sh, c));
}

template <typename Ta, int D>
cudaError_t launch(const ChunkParams& from, bool out_bf16, int sms, cudaStream_t stream) {
    using S = Simt<Ta, D>;
    ChunkParams p = from;
    p.heads = p.Hkv;
    const cudaError_t e = cudaFuncSetAttribute(chunk_simt_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = min(sms * S::kCtas, kMaxWorkers);
    return launch_dependent(chunk_simt_kernel<S>, dim3(ctas), dim3(kThreads), S::kSmem, stream, p, out_bf16);
}

template <typename Ta>
cudaError_t by_head(const ChunkParams& p, int head_dim, bool out_bf16, int sms, cudaStream_t stream) {
    if (head_dim == 64) return launch<Ta, 64>(p, out_bf16, sms, stream);
    if (head_dim == 128) return launch<Ta, 128>(p, out_bf16, sms, stream);
    return launch<Ta, 256>(p, out_bf16, sms, stream);
}

}  // namespace

}  // namespace chunk

size_t chunk_workspace_bytes(int head_dim, int act_dtype, int out_dtype) {
    const size_t n = head_dim == 64    ? chunk::parts_bytes<chunk::kRt, 64>(chunk::kMaxWorkers)
                     : head_dim == 128 ? chunk::parts_bytes<chunk::kRt, 128>(chunk::kMaxWorkers)
                                       : chunk::parts_bytes<chunk::kRt, 256>(chunk::kMaxWorkers);
    if (act_dtype != GDN_BF16) return n;
    const size_t n_tc = chunk::tc_workspace_bytes(head_dim, out_dtype == GDN_BF16);
    return n > n_tc ? n : n_tc;
}

cudaError_t launch_attn_chunk(const ChunkParams& p, int head_dim, int act_dtype, int out_dtype, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    const bool out_bf16 = out_dtype == GDN_BF16;
    if (act_dtype == GDN_BF16) {
        bool done;
        const cudaError_t e = chunk::launch_tc(p, head_dim, out_bf16, sms, &done, stream);
        if (e != cudaSuccess || done) return e;
    }
    if (act_dtype == GDN_BF16) return chunk::by_head<__nv_bfloat16>(p, head_dim, out_bf16, sms, stream);
    return chunk::by_head<float>(p, head_dim, out_bf16, sms, stream);
}

}  // namespace gdn
