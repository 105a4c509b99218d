/*
 * gdn_pages.h -- pages of a paged key-value cache (include/gdn_attn.h) that
 * several sequences share: forking a sequence, releasing shared pages, moving
 * the pages in use together, and the copies of pages that these ask for.
 *
 * Source: the paged cache is this library's form (gdn_attn.h); the xwen
 * CLAUDE.md page serves several answers and cached prefixes from one server
 * and defines no cache layout.
 *
 * page_refs [num_pages] counts the holders of a page beyond its first: 0 for a
 * page that one sequence holds, or none.  The caller zeroes it once; only the
 * calls here change it, and gdn_kv_extend / gdn_kv_append / gdn_attn_decode /
 * gdn_attn_chunk need not know of it: a page is shared only where it is full
 * for all of its holders, so nobody writes into it.  (A page that is not full
 * belongs to one sequence: a fork copies it, and a release that ends inside a
 * shared page replaces it by a copy.)  gdn_kv_truncate does not look at
 * page_refs: sequences that share pages are shortened by gdn_kv_release.
 *
 * The calls that change tables only name the pages to copy, in copy_src and
 * copy_dst (entries of -1: nothing to copy); gdn_kv_copy_pages makes the
 * copies, once for every layer's cache, before the next call that writes keys.
 *
 * Conventions as in gdn_attn.h: caller-owned device buffers, 16-byte aligned,
 * asynchronous on `stream`, no host round trip, no memory allocated, written
 * ranges disjoint from read ranges unless said otherwise.  Arrays called
 * "in place" are read and updated.  B and N up to GDN_KV_MAX_SEQ and
 * B * max_pages up to 2^30 (else GDN_E_UNSUPPORTED).  Results do not depend on
 * the order in which threads run.
 */
#ifndef GDN_PAGES_H
#define GDN_PAGES_H

#include "gdn_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdn_kv_fork -- for i = 0..N-1: sequence dst[i], which is empty, gets the
 * first len[i] tokens of sequence src[i]: the full pages of them are shared
 * (entries copied, page_refs raised), and a last page that is not full becomes
 * a page from the top of the free stack and a pair copy_src[i] -> copy_dst[i].
 *   src, dst, len [N];  seq_len, n_pages [B], block_table [B][max_pages],
 *   page_refs [num_pages], free_count [1]  in place;  free_list [num_pages] read
 *   copy_src, copy_dst [N]   pages, -1 where fork i needs no copy
 *   dev_status [N] or NULL
 * Forks are served in order.  One is refused -- nothing of it happens, and
 * GDN_KV_REFUSED -- when src or dst is outside 0..B-1 or they are equal, when
 * len is negative or more than src's length or than its pages hold, when dst
 * holds tokens or pages or is the dst of an earlier fork that these rules let
 * pass, or when the pages that it and those before it ask for exceed
 * free_count (what a fork asks for counts for the ones after it even where it
 * was refused for want of pages).  A page outside 0..num_pages-1 is handed on
 * as it is, without a count; where a copy would read or write such a page its
 * pair is -1 (the fork's last page then holds nothing of use); either gives
 * the fork GDN_KV_BAD_INDEX.
 */
gdn_status gdn_kv_fork(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages, int32_t N,
                       const int32_t* src, const int32_t* dst, const int32_t* len, int32_t* seq_len,
                       int32_t* n_pages, int32_t* block_table, int32_t* page_refs, const int32_t* free_list,
                       int32_t* free_count, int32_t* copy_src, int32_t* copy_dst, int32_t* dev_status,
                       gdn_stream_t stream);

/*
 * gdn_kv_release -- shorten sequences to new_len[b] tokens (0: finished), as
 * gdn_kv_truncate does, where pages may be shared.  Every page past the new
 * length loses a holder, and goes back to the stack when that was its last.
 * Where the last kept page is not full and had other holders when the call
 * began, it loses a holder too, and the sequence gets a page from the top of
 * the stack in its place and a pair copy_src[b] -> copy_dst[b].
 *   new_len [B];  seq_len, n_pages, block_table, page_refs, free_list,
 *   free_count  in place;  copy_src, copy_dst [B], -1 where there is no copy
 *   dev_status [B] or NULL
 * The pages for copies are taken first, in sequence order; then the pages that
 * nobody holds go back so that the first one given up (by sequence, then by
 * place in it; of a page that several give up, its first place) is on top:
 * without shared pages the stack is the one that gdn_kv_truncate leaves, and a
 * fork of sequences in rising order is undone exactly.
 * Refused, as in gdn_kv_truncate: new_len outside 0..seq_len, n_pages outside
 * 0..max_pages; and a sequence that needs a page for a copy when those before
 * it have asked for all.  A page outside 0..num_pages-1 goes nowhere, and one
 * that the stack has no room for (its caller's books are wrong) is dropped;
 * either gives GDN_KV_BAD_INDEX.
 */
gdn_status gdn_kv_release(int32_t page_size, int32_t num_pages, int32_t B, int32_t max_pages,
                          const int32_t* new_len, int32_t* seq_len, int32_t* n_pages, int32_t* block_table,
                          int32_t* page_refs, int32_t* free_list, int32_t* free_count, int32_t* copy_src,
                          int32_t* copy_dst, int32_t* dev_status, gdn_stream_t stream);

/*
 * gdn_kv_compact -- move the pages that sequences hold to the lowest indices:
 * with `used` such pages, the ones at `used` and above go to the places below
 * that nobody holds, the highest page to the lowest place.
 *   n_pages [B], block_table [B][max_pages]  read (the first n_pages entries
 *     of each sequence)
 *   block_table_out  the same entries with the new indices; may be block_table
 *     itself; entries past a sequence's pages are left
 *   page_refs [num_pages]  formed anew from the tables
 *   free_list [num_pages], free_count [1]  formed anew: all pages that no
 *     sequence holds, the lowest on top (entries past free_count are left)
 *   page_map [num_pages]  new index of each page in use, -1 for the others
 *   copy_src, copy_dst [n_copy_max], n_copy [1]  the moves, then -1; no page
 *     is in both.  n_copy_max >= num_pages / 2 (else GDN_E_INVALID_ARG)
 *   dev_status [B] or NULL: GDN_KV_BAD_INDEX for a page outside
 *     0..num_pages-1 (its entry stays as it is) or n_pages outside
 *     0..max_pages (its pages are not counted as held, its entries left)
 */
gdn_status gdn_kv_compact(int32_t num_pages, int32_t B, int32_t max_pages, const int32_t* n_pages,
                          const int32_t* block_table, int32_t* block_table_out, int32_t* page_refs,
                          int32_t* free_list, int32_t* free_count, int32_t* page_map, int32_t n_copy_max,
                          int32_t* copy_src, int32_t* copy_dst, int32_t* n_copy, int32_t* dev_status,
                          gdn_stream_t stream);

/*
 * gdn_kv_copy_pages -- for i = 0..n-1: page copy_dst[i] := page copy_src[i],
 * keys and values of one layer's cache, all page_size tokens.  Of dims,
 * H_kv, head_dim and act_dtype count (the others have to be valid).  A pair
 * with a negative index is skipped; one with an index past the cache too, and
 * gives GDN_KV_BAD_INDEX in dev_status [1] (or NULL).  A page that is the dst
 * of two pairs, or src of one and dst of another, has no defined result.
 */
gdn_status gdn_kv_copy_pages(const gdn_attn_dims* dims, const gdn_kv_cache* cache, int32_t n,
                             const int32_t* copy_src, const int32_t* copy_dst, int32_t* dev_status,
                             gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_PAGES_H */
