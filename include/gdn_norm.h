/*
 * gdn_norm.h -- the norms either side of a block of libgdn.so's layers, fused
 * with the block's gate and its residual connection.
 *
 * Source: xwen CLAUDE.md page, "Architecture cheat sheet (Qwen 3.6, ggml-org
 * GGUF)": RMSNorm, eps 1e-6, multiply-ready weights (no +1).  The gate, the
 * norm after the block and the residual scale are the general form of the
 * connection; each is optional.
 *
 * For a row y of a block's output (H channels) and a row h of the residual
 * stream:
 *   u  = y / sqrt(mean(y^2) + eps) * post_w      (y itself without post_w)
 *   u  = u * sigmoid(gate)                       (with a gate)
 *   h' = h + alpha * chan_scale * u
 *   x  = h' / sqrt(mean(h'^2) + eps) * pre_w     (the next block's input)
 * all in fp32; h' is rounded once to res_dtype, and x is formed from the
 * unrounded h'.
 */
#ifndef GDN_NORM_H
#define GDN_NORM_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t H;          /* channels, 1 .. GDN_NORM_MAX_H                        */
    float eps;          /* RMSNorm eps                                          */
    float alpha;        /* residual scale                                       */
    int32_t act_dtype;  /* gdn_dtype of y, gate and x                           */
    int32_t res_dtype;  /* gdn_dtype of h and h_out (GDN_F32 where act is GDN_F32) */
} gdn_norm_dims;

#define GDN_NORM_MAX_H 16384

/*
 * gdn_norm_residual -- T rows.
 *   y [T][H] row pitch ldy, or NULL (h' = h: the norm before the first block)
 *   gate_cols 0: no gate; 1: one gate a row; H: one a channel.  gate has row
 *     pitch ldg.  Needs y.
 *   h [T][H], h_out [T][H]  residual stream, dense; h_out may be h (in place),
 *     or NULL (h' is not stored)
 *   post_w, chan_scale, pre_w [H] fp32 or NULL;  x [T][H] dense or NULL (with pre_w)
 * At least one of h_out and x.  Pitches in elements, at least the row's width.
 * GDN_E_ALIGNMENT for a pointer off 16 bytes.  H and the pitches need no
 * alignment, but rows that start on 16 bytes are read and written faster.
 * GDN_E_UNSUPPORTED for H > GDN_NORM_MAX_H or fp32 activations on a bf16 residual stream.
 */
gdn_status gdn_norm_residual(const gdn_norm_dims* dims, int32_t T, const void* y, int64_t ldy, const void* gate,
                             int64_t ldg, int32_t gate_cols, const void* h, const float* post_w,
                             const float* chan_scale, const float* pre_w, void* h_out, void* x, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_NORM_H */
