// gdn_attn_internal.h -- launch parameter blocks of the paged-attention, page
// and norm kernels (not installed; the public surface is include/gdn_attn.h,
// include/gdn_pages.h and include/gdn_norm.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

constexpr int kKvRefused = 32;    // GDN_KV_REFUSED
constexpr int kKvBadIndex = 64;   // GDN_KV_BAD_INDEX
constexpr int kKvMaxSeq = 16384;  // GDN_KV_MAX_SEQ

struct KvExtendParams {
    int page_size, num_pages, B, max_pages, T;
    const int* n_new;
    const int* seq_len;
    const int* n_pages;
    int* block_table;
    const int* free_list;
    const int* free_count;
    int* seq_len_out;
    int* n_pages_out;
    int* free_count_out;
    int* slot_map;
    int* positions;
    int* cu_seqlens;
    int* status;          // optional [B]
};

struct KvTruncateParams {
    int page_size, num_pages, B, max_pages;
    const int* new_len;
    const int* seq_len;
    const int* n_pages;
    const int* block_table;
    int* free_list;
    const int* free_count;
    int* seq_len_out;
    int* n_pages_out;
    int* free_count_out;
    int* status;          // optional [B]
};

// A layer's cache; strides in elements (0 for a dimension of one).
struct KvCache {
    void* k;
    void* v;
    int num_pages, page_size;
    long long page_stride, token_stride, head_stride;
};

struct KvAppendParams {
    KvCache cache;
    int T, Hq, Hkv, rope_dim, n_pos;
    float eps;
    const void* q;
    const void* k;
    const void* v;
    long long ldq, ldk, ldv;
    const int* positions;
    const int* slot_map;
    const float* q_norm_w;
    const float* k_norm_w;
    const float* rope_cos;
    const float* rope_sin;
    void* q_out;
    int* status;          // optional [1]
};

struct AttnParams {
    KvCache cache;
    int B, K, Hq, Hkv, G, max_pages;
    unsigned g_inv;       // 65536 / G rounded up
    float scale;
    const void* q;
    const void* gate;     // optional
    long long ldq, ldg;
    const int* block_table;
    const int* seq_len;
    void* out;
    void* workspace;
    int* status;          // optional [B]
    int test_stall;       // GDN_FLAG_TEST_STALL
};

// Attention of packed new tokens; a unit is up to `tokens` tokens (tokens * G rows) of one sequence and kv head.
struct ChunkParams {
    KvCache cache;
    int B, T, Hq, Hkv, G, max_pages;
    float scale;
    const void* q;
    const void* gate;     // optional
    long long ldq, ldg;
    const int* block_table;
    const int* seq_len;
    const int* cu_seqlens;
    void* out;
    void* workspace;
    int* status;          // optional [B]
    int test_stall;       // GDN_FLAG_TEST_STALL
    int heads;            // filled in at the launch: Hkv, times what a head's units are divided in by channels
};

struct KvForkParams {
    int page_size, num_pages, B, max_pages, N;
    const int* src;
    const int* dst;
    const int* len;
    int* seq_len;
    int* n_pages;
    int* block_table;
    int* page_refs;
    const int* free_list;
    int* free_count;
    int* copy_src;
    int* copy_dst;
    int* status;          // optional [N]
    int room;             // filled in at the launch, as in KvReleaseParams
};

struct KvReleaseParams {
    int page_size, num_pages, B, max_pages;
    const int* new_len;
    int* seq_len;
    int* n_pages;
    int* block_table;
    int* page_refs;
    int* free_list;
    int* free_count;
    int* copy_src;
    int* copy_dst;
    int* status;          // optional [B]
    int room;             // filled in at the launch: words for the pages' counts in shared memory, or 0
};

struct KvCompactParams {
    int num_pages, B, max_pages;
    const int* n_pages;
    const int* block_table;
    int* table_out;
    int* page_refs;
    int* free_list;
    int* free_count;
    int* page_map;
    int n_copy_max;
    int* copy_src;
    int* copy_dst;
    int* n_copy;
    int* status;          // optional [B]
};

// A page is `vectors` of 16 bytes: rows of `run` consecutive ones, row r at (r / inner) * outer_stride + r % inner * inner_stride
// (strides in vectors); `chunks` pieces that a CTA copies at a time.
struct KvCopyParams {
    KvCache cache;
    int n;
    const int* copy_src;
    const int* copy_dst;
    int* status;          // optional [1]
    int vectors, run, inner, chunks;
    long long page_stride, inner_stride, outer_stride;
};

struct NormParams {
    int T, H, gate_cols;
    float eps, alpha;
    const void* y;        // optional
    const void* gate;
    const void* h;
    const float* post_w;
    const float* chan_scale;
    const float* pre_w;
    void* h_out;          // optional
    void* x;              // optional
    long long ldy, ldg;
};

cudaError_t launch_kv_extend(const KvExtendParams& p, cudaStream_t stream);
cudaError_t launch_kv_truncate(const KvTruncateParams& p, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendParams& p, int head_dim, int act_dtype, cudaStream_t stream);
size_t attn_workspace_bytes(int B, int K, int Hq, int Hkv, int head_dim, int act_dtype);
cudaError_t launch_attn_decode(const AttnParams& p, int head_dim, int act_dtype, int out_dtype, cudaStream_t stream);
size_t chunk_workspace_bytes(int head_dim, int act_dtype, int out_dtype);
cudaError_t launch_attn_chunk(const ChunkParams& p, int head_dim, int act_dtype, int out_dtype, cudaStream_t stream);
cudaError_t launch_kv_fork(KvForkParams p, cudaStream_t stream);         // these two fill in room
cudaError_t launch_kv_release(KvReleaseParams p, cudaStream_t stream);
cudaError_t launch_kv_compact(const KvCompactParams& p, cudaStream_t stream);
cudaError_t launch_kv_copy(KvCopyParams p, cudaStream_t stream);   // fills in chunks
cudaError_t launch_norm_residual(const NormParams& p, int act_dtype, int res_dtype, cudaStream_t stream);

}  // namespace gdn
