/*
 * gdn_attn.h -- the full-attention side of a hybrid layer stack in libgdn.so:
 * a paged key-value cache (its page bookkeeping and the append of new tokens)
 * and the attention of new tokens over it, for a caller that decodes the
 * gated DeltaNet layers of include/gdn.h and also has the full-attention
 * layers between them.
 *
 * Source of the layer: xwen CLAUDE.md page, "Architecture cheat sheet (Qwen
 * 3.6, ggml-org GGUF)": full attention at every fourth layer, with RMSNorm of
 * the q and k heads, partial NeoX rotary embedding, scaled dot-product
 * attention and a sigmoid output gate.  The pages do not define a cache
 * layout; the paged form here is this library's.
 *
 * Per layer and token, from the q, k and v rows of the layer's projection:
 *   1. per head of q and k: u = x / sqrt(mean(x^2) + eps) * w;
 *   2. the first rope_dim channels of u in NeoX pairs (i, i + rope_dim/2):
 *        u'_i = u_i cos - u_{i+r/2} sin,   u'_{i+r/2} = u_{i+r/2} cos + u_i sin
 *      with the cos and sin of the token's position and pair;
 *   3. k and v are stored in the cache at the token's slot;
 *   4. query head h reads kv head h / (H_q/H_kv) (grouped order):
 *        s_j = scale * (q . k_j),  o = sum_j softmax(s)_j v_j   over the keys
 *      the query sees; a query that sees no key gives o = 0;
 *   5. out = o * sigmoid(gate).
 *
 * Conventions as in gdn.h: caller-owned device buffers, 16-byte aligned
 * (GDN_E_ALIGNMENT), asynchronous on `stream`, errors returned, written ranges
 * disjoint from read ranges unless said otherwise, no memory allocated.
 * What only the device can see (page indices, lengths, slots) is checked in
 * the kernels: it never leads to an access outside the buffers given, and is
 * reported in the optional dev_status words (the caller zeroes them and reads
 * them after synchronising):
 *   GDN_KV_REFUSED   the page bookkeeping left the sequence as it was
 *   GDN_KV_BAD_INDEX a length, page, slot or position outside its range; the
 *                    keys or tokens concerned were left out
 *   16 (bit 4)       a bounded wait inside gdn_attn_decode gave up: outputs of
 *                    the sequence were not (fully) written, and the workspace
 *                    has to be zeroed before its next use
 */
#ifndef GDN_ATTN_H
#define GDN_ATTN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_KV_REFUSED 32
#define GDN_KV_BAD_INDEX 64
/* Most sequences of one gdn_kv_extend / gdn_kv_truncate call. */
#define GDN_KV_MAX_SEQ 16384

typedef struct {
    int32_t H_q;        /* query heads                                          */
    int32_t H_kv;       /* key/value heads, H_q % H_kv == 0, H_q/H_kv <= 16     */
    int32_t head_dim;   /* 64, 128 or 256 (else GDN_E_UNSUPPORTED)              */
    int32_t rope_dim;   /* rotated channels, 0 or a multiple of 16 <= head_dim  */
    float scale;        /* of the scores, usually 1/sqrt(head_dim)              */
    float eps;          /* RMSNorm eps                                          */
    int32_t act_dtype;  /* gdn_dtype of q, k, v, gate and the cache             */
    int32_t out_dtype;  /* gdn_dtype of the attention's out                     */
    uint32_t flags;     /* 0, or GDN_FLAG_TEST_STALL (gdn.h; in gdn_attn_decode
                           one warp of a CTA waits while the others go on)      */
} gdn_attn_dims;

/*
 * The cache of one layer: token t of page g, head h, channel i is element
 *   g*page_stride + t*token_stride + h*head_stride + i
 * of k and of v (strides in elements, the same for both; multiples of 16
 * bytes; any order of pages, tokens and heads that does not overlap itself; k
 * and v may lie inside one another, but share no element).
 * num_pages * page_size <= INT32_MAX; a slot is g*page_size + t.
 */
typedef struct {
    void* k;
    void* v;
    int32_t num_pages;
    int32_t page_size;   /* tokens in a page, >= 1 */
    int64_t page_stride;
    int64_t token_stride;
    int64_t head_stride;
} gdn_kv_cache;

/*
 * gdn_kv_extend -- give B sequences room for their next tokens: block tables,
 * slots and positions formed on the device from the lengths, with no host
 * round trip (so a decode loop can be captured in a graph).
 *   n_new [B]        tokens to add to each sequence (0: none)
 *   seq_len [B]      current lengths;  n_pages [B]  pages held
 *   block_table [B][max_pages]   page of each page_size tokens; the entries
 *                    n_pages.. of an accepted sequence are filled, the others
 *                    are left (entries past the pages held mean nothing)
 *   free_list [num_pages], free_count [1]   stack of free pages, top last
 *   seq_len_out, n_pages_out [B], free_count_out [1]   the new values; each
 *                    may be the input itself (in place)
 *   slot_map, positions [T]  of the new tokens, sequence after sequence; rows
 *                    past the last one get slot -1 and position 0
 *   cu_seqlens [B+1] first row of each sequence
 *   dev_status [B] or NULL
 * The rows are packed: row b*K + p of gdn_attn_decode is row cu_seqlens[b] + p
 * here, the same only while every sequence is given exactly K tokens.  Where one
 * may be refused or idle the caller maps the one to the other (slot -1 for rows
 * that a sequence does not have; examples/hybrid_decode.py does).
 * Sequences are served in order: sequence b takes its pages from the top of
 * the stack, after those of the sequences before it.  It is refused -- keeps
 * its length and pages, gets no rows -- when its new length needs more than
 * max_pages or num_pages pages, when the pages that it and those before it
 * ask for exceed free_count, when their rows exceed T, or when n_new, seq_len
 * or n_pages is negative or n_pages exceeds max_pages or num_pages.  (What a sequence asks for counts for the ones
 * after it even where it was refused for want of pages or rows.)
 * A token whose page -- from the block table or the stack -- lies outside
 * 0..num_pages-1 gets slot -1, and its sequence GDN_KV_BAD_INDEX.
 * B <= GDN_KV_MAX_SEQ (else GDN_E_UNSUPPORTED).  B == 0 only pads the rows.
 */
gdn_status gdn_kv_extend(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages, int32_t T,
                         const int32_t* n_new, const int32_t* seq_len, const int32_t* n_pages,
                         int32_t* block_table, const int32_t* free_list, const int32_t* free_count,
                         int32_t* seq_len_out, int32_t* n_pages_out, int32_t* free_count_out,
                         int32_t* slot_map, int32_t* positions, int32_t* cu_seqlens, int32_t* dev_status,
                         gdn_stream_t stream);

/*
 * gdn_kv_truncate -- shorten sequences to new_len[b] tokens (0: finished) and
 * put the pages past them back on the stack: the rejected tail of a
 * speculative verify, or finished requests.  The pages go back in the order
 * that undoes a gdn_kv_extend of the same sequences exactly.  Arguments as in
 * gdn_kv_extend; block_table is only read.  A sequence with new_len outside
 * 0..seq_len, or n_pages outside 0..max_pages, or whose pages would not fit
 * the stack, is refused.  Pages go back as the block table has them; one that
 * lies outside 0..num_pages-1 gives its sequence GDN_KV_BAD_INDEX.
 */
gdn_status gdn_kv_truncate(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages,
                           const int32_t* new_len, const int32_t* seq_len, const int32_t* n_pages,
                           const int32_t* block_table, int32_t* free_list, const int32_t* free_count,
                           int32_t* seq_len_out, int32_t* n_pages_out, int32_t* free_count_out,
                           int32_t* dev_status, gdn_stream_t stream);

/*
 * gdn_kv_append -- steps 1-3 for T tokens.
 *   q [T] rows of H_q*head_dim, k, v [T] rows of H_kv*head_dim elements, row
 *     pitches ldq, ldk, ldv in elements (multiples of 16 bytes; slices of one
 *     fused projection row)
 *   positions, slot_map [T]   as gdn_kv_extend forms them; a token with a
 *     negative slot is not stored (its q_out row is still formed)
 *   q_norm_w, k_norm_w [head_dim] fp32, or NULL for no norm
 *   rope_cos, rope_sin [n_pos][rope_dim/2] fp32 (NULL when rope_dim == 0)
 *   q_out [T][H_q*head_dim] act dtype
 *   dev_status [1] or NULL: GDN_KV_BAD_INDEX when a position is outside
 *     0..n_pos-1 (rope_dim > 0) or a slot past the cache; that token is skipped
 * Two tokens with one slot: either may be the one that stays.
 */
gdn_status gdn_kv_append(const gdn_attn_dims* dims, const gdn_kv_cache* cache, int32_t T, const void* q, int64_t ldq,
                         const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* positions,
                         const int32_t* slot_map, const float* q_norm_w, const float* k_norm_w,
                         const float* rope_cos, const float* rope_sin, int32_t n_pos, void* q_out,
                         int32_t* dev_status, gdn_stream_t stream);

/*
 * gdn_attn_decode_workspace_bytes -- device scratch that gdn_attn_decode needs
 * for B sequences of K tokens (0 for arguments that it refuses).
 */
size_t gdn_attn_decode_workspace_bytes(const gdn_attn_dims* dims, int32_t B, int32_t K);

/*
 * gdn_attn_decode -- steps 4-5 for the last K tokens of each of B sequences
 * (K = 1: a decode step; K <= GDN_MAX_VERIFY_K: the tokens of a speculative
 * verify), already in the cache.  Token p of sequence b is row b*K + p and
 * sees keys 0 .. seq_len[b] - K + p; none when that is negative.
 *   q    [B*K][H_q*head_dim], row pitch ldq elements (a multiple of 16 bytes)
 *   gate as q, row pitch ldg, or NULL for no gate
 *   block_table [B][max_pages], seq_len [B]   on the device, as gdn_kv_extend
 *        leaves them (page and length values are not needed on the host)
 *   out  [B*K][H_q*head_dim]
 *   workspace of at least gdn_attn_decode_workspace_bytes() bytes, which the
 *        caller zeroes once, before its first use; every call leaves it ready
 *        for the next call, of any shape that it is large enough for.  Calls
 *        that may run at the same time need a workspace each.
 *   dev_status [B] or NULL: GDN_KV_BAD_INDEX when seq_len[b] exceeds
 *        max_pages*page_size (taken as that) or a page index lies outside the
 *        cache (its keys are left out)
 * No memory beyond a sequence's length is read, so what lies there (NaN
 * included) does not matter; nor does a token's key or value to the rows that do
 * not see it.  An infinite or NaN value element makes that channel of the rows
 * that see it infinite or NaN.  Results do not depend on what runs beside the
 * call, and are the same from run to run.
 */
gdn_status gdn_attn_decode(const gdn_attn_dims* dims, const gdn_kv_cache* cache, int32_t B, int32_t K,
                           int32_t max_pages, const void* q, int64_t ldq, const void* gate, int64_t ldg,
                           const int32_t* block_table, const int32_t* seq_len, void* out, void* workspace,
                           size_t workspace_bytes, int32_t* dev_status, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H */
