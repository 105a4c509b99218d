// gdn_attn_api.cu -- the C ABI of include/gdn_attn.h, include/gdn_pages.h and
// include/gdn_norm.h: argument validation and dispatch.  Host code only; the
// work is in gdn_kv.cu, gdn_pages.cu, gdn_attn.cuh (gdn_attn_bf16.cu, gdn_attn_f32.cu, gdn_attn_tc.cu), gdn_chunk.cuh and gdn_norm.cu.
#include "gdn_attn.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "gdn_attn_internal.h"
#include "gdn_norm.h"
#include "gdn_pages.h"

namespace {

constexpr int64_t kMaxPitch = int64_t{1} << 40;   // elements
constexpr int64_t kMaxSpan = int64_t{1} << 60;    // elements: more than any address space has, and sums of a few stay in 64 bits

// a * b where that is under kMaxSpan, else kMaxSpan (a, b >= 0).
int64_t times(int64_t a, int64_t b) { return a != 0 && b > kMaxSpan / a ? kMaxSpan : a * b; }

constexpr int64_t kMaxEntries = int64_t{1} << 30;   // of block tables that share pages, and of what is numbered with them

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t elem_size(int32_t dt) { return dt == GDN_BF16 ? 2 : 4; }

bool is_dtype(int32_t dt) { return dt == GDN_F32 || dt == GDN_BF16; }

struct Range {
    const void* p;
    size_t bytes;
};

bool overlap(Range a, Range b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Every written range must be disjoint from every read-only range and from
// every other written range.
bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Range& i : ins)
            if (overlap(*o, i)) return true;
        for (auto o2 = o + 1; o2 != outs.end(); ++o2)
            if (overlap(*o, *o2)) return true;
    }
    return false;
}

gdn_status check_ptrs(std::initializer_list<const void*> required, std::initializer_list<const void*> optional) {
    for (const void* p : required)
        if (!p) return GDN_E_INVALID_ARG;
    for (const void* p : required)
        if (!aligned16(p)) return GDN_E_ALIGNMENT;
    for (const void* p : optional)
        if (p && !aligned16(p)) return GDN_E_ALIGNMENT;
    return GDN_OK;
}

gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_E_CUDA; }

gdn_status check_attn_dims(const gdn_attn_dims* d) {
    if (!d) return GDN_E_INVALID_ARG;
    if (d->H_q < 1 || d->H_kv < 1 || d->H_q > 4096 || d->H_kv > 4096 || d->H_q % d->H_kv != 0)
        return GDN_E_INVALID_ARG;
    if (!is_dtype(d->act_dtype) || !is_dtype(d->out_dtype)) return GDN_E_INVALID_ARG;
    if (!std::isfinite(d->scale) || !(d->eps > 0.0f) || !std::isfinite(d->eps)) return GDN_E_INVALID_ARG;
    if (d->rope_dim < 0 || d->rope_dim > d->head_dim || (d->flags & ~GDN_FLAG_TEST_STALL)) return GDN_E_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return GDN_E_UNSUPPORTED;
    if (d->H_q / d->H_kv > 16 || d->rope_dim % 16 != 0) return GDN_E_UNSUPPORTED;
    return GDN_OK;
}

struct Dim {
    int64_t n, stride;
};

// Whether two sets of elements, each {sum of i_d stride_d, 0 <= i_d < n_d} and one `delta` >= 0 elements after the other, meet: delta
// is then a sum of j_d stride_d with |j_d| < n_d.  The strides fall, each past all that is inside it, so that j_d is
// the quotient of what is left or the next number.
bool meet(const Dim* m, int dims, int64_t delta) {
    if (dims == 0) return delta == 0;
    if (m->n == 1) return meet(m + 1, dims - 1, delta);
    const int64_t a = delta < 0 ? -delta : delta, j = a / m->stride;
    return (j < m->n && meet(m + 1, dims - 1, a - j * m->stride)) || (j + 1 < m->n && meet(m + 1, dims - 1, a - (j + 1) * m->stride));
}

// The cache's shape, with the strides of dimensions of one set to zero; *bytes = its
// bytes from the first to the last element, per half.
gdn_status check_cache(const gdn_attn_dims* d, const gdn_kv_cache* c, gdn::KvCache* out, size_t* bytes) {
    if (!c) return GDN_E_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1) return GDN_E_INVALID_ARG;
    if (static_cast<int64_t>(c->num_pages) * c->page_size > INT32_MAX) return GDN_E_INVALID_ARG;
    if (c->k == c->v) return GDN_E_INVALID_ARG;
    const gdn_status s = check_ptrs({c->k, c->v}, {});
    if (s != GDN_OK) return s;
    Dim m[4] = {{c->num_pages, c->page_stride}, {c->page_size, c->token_stride}, {d->H_kv, c->head_stride}, {d->head_dim, 1}};
    const int64_t vec = 16 / static_cast<int64_t>(elem_size(d->act_dtype));
    for (Dim* x = m; x != m + 3; ++x) {
        if (x->n == 1) x->stride = 0;
        if (x->stride < 0 || x->stride > kMaxPitch) return GDN_E_INVALID_ARG;
        if (x->stride % vec != 0) return GDN_E_ALIGNMENT;
    }
    *out = gdn::KvCache{c->k, c->v, c->num_pages, c->page_size, m[0].stride, m[1].stride, m[2].stride};
    // from the smallest stride up, each steps past all that is inside it: no two elements share an address
    std::sort(m, m + 3, [](const Dim& a, const Dim& b) { return a.stride > b.stride; });
    int64_t span = d->head_dim;
    for (const Dim* x = m + 2; x >= m; --x) {
        if (x->n == 1) continue;
        if (x->stride < span) return GDN_E_INVALID_ARG;
        span += times(x->n - 1, x->stride);
        if (span >= kMaxSpan) return GDN_E_INVALID_ARG;
    }
    *bytes = static_cast<size_t>(span) * elem_size(d->act_dtype);
    // the halves may lie page by page or row by row inside one another, but share no element
    const uintptr_t k = reinterpret_cast<uintptr_t>(c->k), v = reinterpret_cast<uintptr_t>(c->v);
    const uintptr_t apart = k < v ? v - k : k - v;
    if (apart < *bytes && meet(m, 4, static_cast<int64_t>(apart / elem_size(d->act_dtype)))) return GDN_E_INVALID_ARG;
    return GDN_OK;
}

// Bytes from the first to the last element of T rows of n elements at a pitch.
size_t rows_bytes(int64_t T, int64_t n, int64_t ld, size_t es) {
    return T > 0 ? static_cast<size_t>(times(T - 1, ld) + n) * es : 0;
}

gdn_status check_pitch(int64_t ld, int64_t n, size_t es) {
    if (ld < n || ld > kMaxPitch) return GDN_E_INVALID_ARG;
    return (ld * static_cast<int64_t>(es)) % 16 == 0 ? GDN_OK : GDN_E_ALIGNMENT;
}

gdn_status check_kv_sizes(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages) {
    if (page_size < 1 || num_pages < 1 || B < 0 || max_pages < 1) return GDN_E_INVALID_ARG;
    if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return GDN_E_INVALID_ARG;
    if (B > GDN_KV_MAX_SEQ) return GDN_E_UNSUPPORTED;
    return GDN_OK;
}

// `out` may be `in` itself but not otherwise share bytes with it.
bool partly(const void* out, const void* in, size_t bytes) { return out != in && overlap({out, bytes}, {in, bytes}); }

}  // namespace

extern "C" {

gdn_status gdn_kv_extend(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages, int32_t T,
                         const int32_t* n_new, const int32_t* seq_len, const int32_t* n_pages,
                         int32_t* block_table, const int32_t* free_list, const int32_t* free_count,
                         int32_t* seq_len_out, int32_t* n_pages_out, int32_t* free_count_out,
                         int32_t* slot_map, int32_t* positions, int32_t* cu_seqlens, int32_t* dev_status,
                         gdn_stream_t stream) {
    gdn_status s = check_kv_sizes(page_size, num_pages, B, max_pages);
    if (s != GDN_OK) return s;
    if (T < 0) return GDN_E_INVALID_ARG;
    if ((s = check_ptrs({free_list, free_count, free_count_out, cu_seqlens}, {dev_status})) != GDN_OK) return s;
    if (B > 0 && (s = check_ptrs({n_new, seq_len, n_pages, block_table, seq_len_out, n_pages_out}, {})) != GDN_OK)
        return s;
    if (T > 0 && (s = check_ptrs({slot_map, positions}, {})) != GDN_OK) return s;
    const size_t nb = static_cast<size_t>(B) * 4, nt = static_cast<size_t>(T) * 4;
    if (partly(seq_len_out, seq_len, nb) || partly(n_pages_out, n_pages, nb) || partly(free_count_out, free_count, 4))
        return GDN_E_INVALID_ARG;
    const Range sl{seq_len_out == seq_len ? nullptr : seq_len, nb}, np{n_pages_out == n_pages ? nullptr : n_pages, nb},
        fc{free_count_out == free_count ? nullptr : free_count, 4};
    if (any_overlap({{block_table, nb * max_pages}, {seq_len_out, nb}, {n_pages_out, nb}, {free_count_out, 4},
                     {slot_map, nt}, {positions, nt}, {cu_seqlens, nb + 4}, {dev_status, nb}},
                    {{n_new, nb}, sl, np, fc, {free_list, static_cast<size_t>(num_pages) * 4}}))
        return GDN_E_INVALID_ARG;
    gdn::KvExtendParams p{page_size, num_pages, B, max_pages, T, n_new, seq_len, n_pages, block_table, free_list,
                          free_count, seq_len_out, n_pages_out, free_count_out, slot_map, positions, cu_seqlens,
                          dev_status};
    return cuda_status(gdn::launch_kv_extend(p, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_truncate(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages,
                           const int32_t* new_len, const int32_t* seq_len, const int32_t* n_pages,
                           const int32_t* block_table, int32_t* free_list, const int32_t* free_count,
                           int32_t* seq_len_out, int32_t* n_pages_out, int32_t* free_count_out,
                           int32_t* dev_status, gdn_stream_t stream) {
    gdn_status s = check_kv_sizes(page_size, num_pages, B, max_pages);
    if (s != GDN_OK) return s;
    if ((s = check_ptrs({free_list, free_count, free_count_out}, {dev_status})) != GDN_OK) return s;
    if (B > 0 && (s = check_ptrs({new_len, seq_len, n_pages, block_table, seq_len_out, n_pages_out}, {})) != GDN_OK)
        return s;
    const size_t nb = static_cast<size_t>(B) * 4;
    if (partly(seq_len_out, seq_len, nb) || partly(n_pages_out, n_pages, nb) || partly(free_count_out, free_count, 4))
        return GDN_E_INVALID_ARG;
    const Range sl{seq_len_out == seq_len ? nullptr : seq_len, nb}, np{n_pages_out == n_pages ? nullptr : n_pages, nb},
        fc{free_count_out == free_count ? nullptr : free_count, 4};
    if (any_overlap({{free_list, static_cast<size_t>(num_pages) * 4}, {seq_len_out, nb}, {n_pages_out, nb},
                     {free_count_out, 4}, {dev_status, nb}},
                    {{new_len, nb}, sl, np, fc, {block_table, nb * max_pages}}))
        return GDN_E_INVALID_ARG;
    gdn::KvTruncateParams p{page_size, num_pages, B, max_pages, new_len, seq_len, n_pages, block_table, free_list,
                            free_count, seq_len_out, n_pages_out, free_count_out, dev_status};
    return cuda_status(gdn::launch_kv_truncate(p, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_append(const gdn_attn_dims* dims, const gdn_kv_cache* cache, int32_t T, const void* q, int64_t ldq,
                         const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* positions,
                         const int32_t* slot_map, const float* q_norm_w, const float* k_norm_w,
                         const float* rope_cos, const float* rope_sin, int32_t n_pos, void* q_out,
                         int32_t* dev_status, gdn_stream_t stream) {
    gdn_status s = check_attn_dims(dims);
    if (s != GDN_OK) return s;
    gdn::KvCache kc;
    size_t kv_bytes = 0;
    if ((s = check_cache(dims, cache, &kc, &kv_bytes)) != GDN_OK) return s;
    if (T < 0) return GDN_E_INVALID_ARG;
    const bool rope = dims->rope_dim > 0;
    if (rope && (n_pos < 1 || !rope_cos || !rope_sin)) return GDN_E_INVALID_ARG;
    if (T == 0) return GDN_OK;
    if ((s = check_ptrs({q, k, v, positions, slot_map, q_out}, {q_norm_w, k_norm_w, rope_cos, rope_sin, dev_status})) !=
        GDN_OK)
        return s;
    const size_t es = elem_size(dims->act_dtype);
    const int64_t nq = static_cast<int64_t>(dims->H_q) * dims->head_dim;
    const int64_t nk = static_cast<int64_t>(dims->H_kv) * dims->head_dim;
    if ((s = check_pitch(ldq, nq, es)) != GDN_OK || (s = check_pitch(ldk, nk, es)) != GDN_OK ||
        (s = check_pitch(ldv, nk, es)) != GDN_OK)
        return s;
    const size_t tab = rope ? static_cast<size_t>(n_pos) * (dims->rope_dim / 2) * 4 : 0;
    const size_t nt = static_cast<size_t>(T) * 4, nw = static_cast<size_t>(dims->head_dim) * 4;
    const std::initializer_list<Range> ins = {{q, rows_bytes(T, nq, ldq, es)}, {k, rows_bytes(T, nk, ldk, es)},
                                              {v, rows_bytes(T, nk, ldv, es)}, {positions, nt}, {slot_map, nt},
                                              {q_norm_w, nw}, {k_norm_w, nw}, {rope_cos, tab}, {rope_sin, tab}};
    const Range qo{q_out, rows_bytes(T, nq, nq, es)}, st{dev_status, 4}, ck{kc.k, kv_bytes}, cv{kc.v, kv_bytes};
    // (the two halves of a cache may lie inside one another: check_cache)
    if (any_overlap({qo, st, ck}, ins) || any_overlap({qo, st, cv}, ins)) return GDN_E_INVALID_ARG;
    gdn::KvAppendParams p{kc, T, dims->H_q, dims->H_kv, dims->rope_dim, n_pos, dims->eps, q, k, v, ldq, ldk, ldv,
                          positions, slot_map, q_norm_w, k_norm_w, rope_cos, rope_sin, q_out, dev_status};
    return cuda_status(
        gdn::launch_kv_append(p, dims->head_dim, dims->act_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_decode_workspace_bytes(const gdn_attn_dims* dims, int32_t B, int32_t K) {
    if (check_attn_dims(dims) != GDN_OK || B < 1 || K < 1 || K > GDN_MAX_VERIFY_K) return 0;
    return gdn::attn_workspace_bytes(B, K, dims->H_q, dims->H_kv, dims->head_dim, dims->act_dtype);
}

gdn_status gdn_attn_decode(const gdn_attn_dims* dims, const gdn_kv_cache* cache, int32_t B, int32_t K,
                           int32_t max_pages, const void* q, int64_t ldq, const void* gate, int64_t ldg,
                           const int32_t* block_table, const int32_t* seq_len, void* out, void* workspace,
                           size_t workspace_bytes, int32_t* dev_status, gdn_stream_t stream) {
    gdn_status s = check_attn_dims(dims);
    if (s != GDN_OK) return s;
    gdn::KvCache kc;
    size_t kv_bytes = 0;
    if ((s = check_cache(dims, cache, &kc, &kv_bytes)) != GDN_OK) return s;
    if (B < 0 || K < 1 || K > GDN_MAX_VERIFY_K || max_pages < 1) return GDN_E_INVALID_ARG;
    // a row of the output has one index of 31 bits
    if (static_cast<int64_t>(B) * K * dims->H_q > INT32_MAX) return GDN_E_INVALID_ARG;
    if (B == 0) return GDN_OK;
    if ((s = check_ptrs({q, block_table, seq_len, out}, {gate, workspace, dev_status})) != GDN_OK) return s;
    const size_t es = elem_size(dims->act_dtype), eo = elem_size(dims->out_dtype);
    const int64_t T = static_cast<int64_t>(B) * K, n = static_cast<int64_t>(dims->H_q) * dims->head_dim;
    if ((s = check_pitch(ldq, n, es)) != GDN_OK) return s;
    if (gate && (s = check_pitch(ldg, n, es)) != GDN_OK) return s;
    const size_t need = gdn_attn_decode_workspace_bytes(dims, B, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_E_WORKSPACE;
    const size_t nb = static_cast<size_t>(B) * 4;
    if (any_overlap({{out, rows_bytes(T, n, n, eo)}, {workspace, need}, {dev_status, nb}},
                    {{kc.k, kv_bytes}, {kc.v, kv_bytes}, {q, rows_bytes(T, n, ldq, es)},
                     {gate, rows_bytes(T, n, ldg, es)}, {block_table, nb * max_pages}, {seq_len, nb}}))
        return GDN_E_INVALID_ARG;
    const int G = dims->H_q / dims->H_kv;
    gdn::AttnParams p{kc, B, K, dims->H_q, dims->H_kv, G, max_pages, (65536u + G - 1) / G, dims->scale, q, gate, ldq,
                      ldg, block_table, seq_len, out, workspace, dev_status,
                      (dims->flags & GDN_FLAG_TEST_STALL) ? 1 : 0};
    return cuda_status(gdn::launch_attn_decode(p, dims->head_dim, dims->act_dtype, dims->out_dtype,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_chunk_workspace_bytes(const gdn_attn_dims* dims, int32_t B, int32_t T) {
    if (check_attn_dims(dims) != GDN_OK || B < 1 || T < 1) return 0;
    return gdn::chunk_workspace_bytes(dims->head_dim, dims->act_dtype, dims->out_dtype);
}

gdn_status gdn_attn_chunk(const gdn_attn_dims* dims, const gdn_kv_cache* cache, int32_t B, int32_t T,
                          int32_t max_pages, const void* q, int64_t ldq, const void* gate, int64_t ldg,
                          const int32_t* cu_seqlens, const int32_t* block_table, const int32_t* seq_len, void* out,
                          void* workspace, size_t workspace_bytes, int32_t* dev_status, gdn_stream_t stream) {
    gdn_status s = check_attn_dims(dims);
    if (s != GDN_OK) return s;
    gdn::KvCache kc;
    size_t kv_bytes = 0;
    if ((s = check_cache(dims, cache, &kc, &kv_bytes)) != GDN_OK) return s;
    if (B < 0 || T < 0 || max_pages < 1) return GDN_E_INVALID_ARG;
    if (static_cast<int64_t>(T) * dims->H_q > INT32_MAX) return GDN_E_INVALID_ARG;   // a row of the output has one index of 31 bits
    if (B == 0 || T == 0) return GDN_OK;
    if ((s = check_ptrs({q, cu_seqlens, block_table, seq_len, out}, {gate, workspace, dev_status})) != GDN_OK) return s;
    const size_t es = elem_size(dims->act_dtype), eo = elem_size(dims->out_dtype);
    const int64_t n = static_cast<int64_t>(dims->H_q) * dims->head_dim;
    if (T == 1) ldq = ldg = n;   // one row's pitch is of no account
    if ((s = check_pitch(ldq, n, es)) != GDN_OK) return s;
    if (gate && (s = check_pitch(ldg, n, es)) != GDN_OK) return s;
    const size_t need = gdn_attn_chunk_workspace_bytes(dims, B, T);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_E_WORKSPACE;
    const size_t nb = static_cast<size_t>(B) * 4;
    if (any_overlap({{out, rows_bytes(T, n, n, eo)}, {workspace, need}, {dev_status, nb}},
                    {{kc.k, kv_bytes}, {kc.v, kv_bytes}, {q, rows_bytes(T, n, ldq, es)},
                     {gate, rows_bytes(T, n, ldg, es)}, {cu_seqlens, nb + 4}, {block_table, nb * max_pages},
                     {seq_len, nb}}))
        return GDN_E_INVALID_ARG;
    gdn::ChunkParams p{kc, B, T, dims->H_q, dims->H_kv, dims->H_q / dims->H_kv, max_pages, dims->scale, q, gate, ldq, ldg,
                       block_table, seq_len, cu_seqlens, out, workspace, dev_status,
                       (dims->flags & GDN_FLAG_TEST_STALL) ? 1 : 0};
    return cuda_status(gdn::launch_attn_chunk(p, dims->head_dim, dims->act_dtype, dims->out_dtype,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_fork(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages, int32_t N,
                       const int32_t* src, const int32_t* dst, const int32_t* len, int32_t* seq_len,
                       int32_t* n_pages, int32_t* block_table, int32_t* page_refs, const int32_t* free_list,
                       int32_t* free_count, int32_t* copy_src, int32_t* copy_dst, int32_t* dev_status,
                       gdn_stream_t stream) {
    gdn_status s = check_kv_sizes(page_size, num_pages, B, max_pages);
    if (s != GDN_OK) return s;
    if (N < 0) return GDN_E_INVALID_ARG;
    if (N > GDN_KV_MAX_SEQ || static_cast<int64_t>(B) * max_pages > kMaxEntries) return GDN_E_UNSUPPORTED;
    if (N == 0) return GDN_OK;
    if ((s = check_ptrs({src, dst, len, page_refs, free_list, free_count, copy_src, copy_dst}, {dev_status})) != GDN_OK)
        return s;
    if (B > 0 && (s = check_ptrs({seq_len, n_pages, block_table}, {})) != GDN_OK) return s;
    const size_t nb = static_cast<size_t>(B) * 4, nn = static_cast<size_t>(N) * 4, np = static_cast<size_t>(num_pages) * 4;
    if (any_overlap({{seq_len, nb}, {n_pages, nb}, {block_table, nb * max_pages}, {page_refs, np}, {free_count, 4},
                     {copy_src, nn}, {copy_dst, nn}, {dev_status, nn}},
                    {{src, nn}, {dst, nn}, {len, nn}, {free_list, np}}))
        return GDN_E_INVALID_ARG;
    gdn::KvForkParams p{page_size, num_pages, B, max_pages, N, src, dst, len, seq_len, n_pages, block_table, page_refs,
                        free_list, free_count, copy_src, copy_dst, dev_status, 0};
    return cuda_status(gdn::launch_kv_fork(p, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_release(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages,
                          const int32_t* new_len, int32_t* seq_len, int32_t* n_pages, int32_t* block_table,
                          int32_t* page_refs, int32_t* free_list, int32_t* free_count, int32_t* copy_src,
                          int32_t* copy_dst, int32_t* dev_status, gdn_stream_t stream) {
    gdn_status s = check_kv_sizes(page_size, num_pages, B, max_pages);
    if (s != GDN_OK) return s;
    if (static_cast<int64_t>(B) * max_pages > kMaxEntries) return GDN_E_UNSUPPORTED;
    if (B == 0) return GDN_OK;
    if ((s = check_ptrs({new_len, seq_len, n_pages, block_table, page_refs, free_list, free_count, copy_src, copy_dst},
                        {dev_status})) != GDN_OK)
        return s;
    const size_t nb = static_cast<size_t>(B) * 4, np = static_cast<size_t>(num_pages) * 4;
    if (any_overlap({{seq_len, nb}, {n_pages, nb}, {block_table, nb * max_pages}, {page_refs, np}, {free_list, np},
                     {free_count, 4}, {copy_src, nb}, {copy_dst, nb}, {dev_status, nb}},
                    {{new_len, nb}}))
        return GDN_E_INVALID_ARG;
    gdn::KvReleaseParams p{page_size, num_pages, B, max_pages, new_len, seq_len, n_pages, block_table, page_refs,
                           free_list, free_count, copy_src, copy_dst, dev_status, 0};
    return cuda_status(gdn::launch_kv_release(p, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_compact(int32_t num_pages, int32_t B, int32_t max_pages, const int32_t* n_pages,
                          const int32_t* block_table, int32_t* block_table_out, int32_t* page_refs,
                          int32_t* free_list, int32_t* free_count, int32_t* page_map, int32_t n_copy_max,
                          int32_t* copy_src, int32_t* copy_dst, int32_t* n_copy, int32_t* dev_status,
                          gdn_stream_t stream) {
    gdn_status s = check_kv_sizes(1, num_pages, B, max_pages);
    if (s != GDN_OK) return s;
    if (n_copy_max < num_pages / 2) return GDN_E_INVALID_ARG;
    if (num_pages > kMaxEntries || n_copy_max > kMaxEntries || static_cast<int64_t>(B) * max_pages > kMaxEntries)
        return GDN_E_UNSUPPORTED;
    if ((s = check_ptrs({page_refs, free_list, free_count, page_map, n_copy}, {dev_status})) != GDN_OK) return s;
    if (n_copy_max > 0 && (s = check_ptrs({copy_src, copy_dst}, {})) != GDN_OK) return s;
    if (B > 0 && (s = check_ptrs({n_pages, block_table, block_table_out}, {})) != GDN_OK) return s;
    const size_t nb = static_cast<size_t>(B) * 4, np = static_cast<size_t>(num_pages) * 4;
    const size_t nc = static_cast<size_t>(n_copy_max) * 4;
    if (partly(block_table_out, block_table, nb * max_pages)) return GDN_E_INVALID_ARG;
    const Range table{block_table_out == block_table ? nullptr : block_table, nb * max_pages};
    if (any_overlap({{block_table_out, nb * max_pages}, {page_refs, np}, {free_list, np}, {free_count, 4}, {page_map, np},
                     {copy_src, nc}, {copy_dst, nc}, {n_copy, 4}, {dev_status, nb}},
                    {{n_pages, nb}, table}))
        return GDN_E_INVALID_ARG;
    gdn::KvCompactParams p{num_pages, B, max_pages, n_pages, block_table, block_table_out, page_refs, free_list, free_count,
                           page_map, n_copy_max, copy_src, copy_dst, n_copy, dev_status};
    return cuda_status(gdn::launch_kv_compact(p, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_copy_pages(const gdn_attn_dims* dims, const gdn_kv_cache* cache, int32_t n,
                             const int32_t* copy_src, const int32_t* copy_dst, int32_t* dev_status,
                             gdn_stream_t stream) {
    gdn_status s = check_attn_dims(dims);
    if (s != GDN_OK) return s;
    gdn::KvCache kc;
    size_t kv_bytes = 0;
    if ((s = check_cache(dims, cache, &kc, &kv_bytes)) != GDN_OK) return s;
    if (n < 0) return GDN_E_INVALID_ARG;
    if (n == 0) return GDN_OK;
    if ((s = check_ptrs({copy_src, copy_dst}, {dev_status})) != GDN_OK) return s;
    const size_t nn = static_cast<size_t>(n) * 4;
    const Range a{copy_src, nn}, b{copy_dst, nn}, st{dev_status, 4};
    // (the two halves of a cache may lie inside one another: check_cache)
    if (any_overlap({{kc.k, kv_bytes}, st}, {a, b}) || any_overlap({{kc.v, kv_bytes}, st}, {a, b})) return GDN_E_INVALID_ARG;
    const int64_t vec = 16 / static_cast<int64_t>(elem_size(dims->act_dtype));
    const int64_t vectors = times(times(kc.page_size, dims->H_kv), dims->head_dim / vec);
    if (vectors > kMaxEntries) return GDN_E_UNSUPPORTED;
    // rows of consecutive vectors, the smaller stride inside; dimensions that follow on one another are one
    Dim in{dims->H_kv, kc.head_stride / vec}, out{kc.page_size, kc.token_stride / vec};
    if (out.n > 1 && (in.n == 1 || out.stride < in.stride)) std::swap(in, out);
    int64_t run = dims->head_dim / vec;
    for (int i = 0; i < 2 && (in.n == 1 || in.stride == run); ++i) {
        run *= in.n;
        in = out;
        out = Dim{1, 0};
    }
    gdn::KvCopyParams p{kc, n, copy_src, copy_dst, dev_status, static_cast<int>(vectors), static_cast<int>(run),
                        static_cast<int>(in.n), 0, kc.page_stride / vec, in.stride, out.stride};
    return cuda_status(gdn::launch_kv_copy(p, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_norm_residual(const gdn_norm_dims* dims, int32_t T, const void* y, int64_t ldy, const void* gate,
                             int64_t ldg, int32_t gate_cols, const void* h, const float* post_w,
                             const float* chan_scale, const float* pre_w, void* h_out, void* x, gdn_stream_t stream) {
    if (!dims) return GDN_E_INVALID_ARG;
    if (dims->H < 1 || T < 0 || !is_dtype(dims->act_dtype) || !is_dtype(dims->res_dtype)) return GDN_E_INVALID_ARG;
    if (!(dims->eps > 0.0f) || !std::isfinite(dims->eps) || !std::isfinite(dims->alpha)) return GDN_E_INVALID_ARG;
    if (gate_cols != 0 && gate_cols != 1 && gate_cols != dims->H) return GDN_E_INVALID_ARG;
    if (dims->H > GDN_NORM_MAX_H) return GDN_E_UNSUPPORTED;
    if (dims->act_dtype == GDN_F32 && dims->res_dtype == GDN_BF16) return GDN_E_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    if (!h || (!h_out && !x) || (x != nullptr) != (pre_w != nullptr)) return GDN_E_INVALID_ARG;
    if ((gate_cols != 0) != (gate != nullptr)) return GDN_E_INVALID_ARG;
    if (!y && (gate || post_w || chan_scale)) return GDN_E_INVALID_ARG;
    const gdn_status s = check_ptrs({h}, {y, gate, post_w, chan_scale, pre_w, h_out, x});
    if (s != GDN_OK) return s;
    if (y && (ldy < dims->H || ldy > kMaxPitch)) return GDN_E_INVALID_ARG;
    if (gate && (ldg < gate_cols || ldg > kMaxPitch)) return GDN_E_INVALID_ARG;
    const size_t es = elem_size(dims->act_dtype), er = elem_size(dims->res_dtype);
    const size_t n = static_cast<size_t>(T) * dims->H, nw = static_cast<size_t>(dims->H) * 4;
    const Range hr{h_out == h ? nullptr : h, n * er};
    if (any_overlap({{h_out, n * er}, {x, n * es}},
                    {{y, rows_bytes(T, dims->H, ldy, es)}, {gate, rows_bytes(T, gate_cols, ldg, es)}, hr,
                     {post_w, nw}, {chan_scale, nw}, {pre_w, nw}}))
        return GDN_E_INVALID_ARG;
    gdn::NormParams p{T, dims->H, gate_cols, dims->eps, dims->alpha, y, gate, h, post_w, chan_scale, pre_w, h_out, x,
                      ldy, ldg};
    return cuda_status(gdn::launch_norm_residual(p, dims->act_dtype, dims->res_dtype,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
