/*
 * moe_train.h - C ABI of the training side of the MI355X (gfx950) MoE library
 * (libmoe_route.so): the top-k gate that makes the expert ids and weights of
 * moe_route.h, the embedding lookup, and the gradients of gate, dispatch,
 * combine and lookup.
 *
 * The conventions of moe_route.h hold for every entry point here: device
 * pointers, row-major layouts without gaps between rows, buffers owned by the
 * caller, work enqueued on `stream` without waiting, every argument checked on
 * the host before anything is enqueued, deterministic results (no sum depends
 * on timing: there are no floating-point atomics), no output that needs clearing
 * between calls.  Entries, rows and token ids outside their range never fault:
 * they are skipped as stated.  Sums, softmax statistics and products are held in
 * f32; a bf16 output is rounded once, to nearest even, when it is stored.
 * Input and output buffers must not overlap unless a call says so.
 *
 * Limits: 0 <= T, N; 1 <= K <= 16; 1 <= E <= 1024; T*K < 2^31; N < 2^31;
 * H > 0 with H % 8 == 0 (H % 128 == 0 for fp8 and fp4 rows) and H <= 2^24;
 * 1 <= V <= 2^31-1; row counts <= 2^31-1; row buffers 16-byte aligned.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Top-k gate: the K largest of each token's E logits and their softmax weights.
 *   logits  [T,E] l_dt (MOE_BF16 or MOE_F32), aligned to its element
 *   idx     out int32 [T,K]: expert ids by descending logit, equal logits by
 *           ascending id.  A NaN counts as the largest value.  -inf is "masked":
 *           such an expert is never chosen, and places that find no other get -1
 *           (which the dispatch skips silently).
 *   w       out f32 [T,K]: scale * p, 0 where idx is -1.  renormalize != 0: p is
 *           the softmax over the chosen logits; 0: over all E logits.  A NaN or
 *           +inf among the logits that the softmax runs over makes the token's
 *           weights NaN.  A weight is off by at most about (2.25 d + 2 n + 8) 2^-24
 *           of its value, d the distance from the lowest to the highest logit of the
 *           token (at most 104) and n the number of terms of the softmax; the
 *           gradient's p likewise.
 * K <= E. */
int moe_gate(const void* logits, moe_dtype l_dt, int64_t T, int E, int K, int renormalize,
             float scale, int32_t* idx, float* w, void* stream);

/* Gradient of moe_gate with respect to the logits, the choice held fixed.  With
 * p as above, d_k = scale * p[idx_k] * dw_k and D = sum_k d_k (k ascending):
 *   renormalize != 0:  dlogits[t,j] = sum over k with idx_k = j of (d_k - p_k*D);
 *                      0 for every expert that was not chosen
 *   renormalize == 0:  dlogits[t,j] = sum over k with idx_k = j of d_k, - p_j*D
 * Entries whose idx is outside [0,E), or whose expert's logit is -inf, are skipped
 * whatever their dw holds; a token whose softmax runs over nothing but -inf gets
 * zeros.  "The chosen" are the entries: an expert named twice, which moe_gate never
 * does, stands twice in the softmax of renormalize and gets both entries' gradients.
 *   logits  [T,E] l_dt, as given to moe_gate
 *   idx     int32 [T,K]; dw f32 [T,K]
 *   dlogits out [T,E] l_dt */
int moe_gate_backward(const void* logits, moe_dtype l_dt, int64_t T, int E, int K,
                      int renormalize, float scale, const int32_t* idx, const float* dw,
                      void* dlogits, void* stream);

/* Gradient of the combines (moe_combine, plain or dedup, moe_combine_fp8 and
 * moe_combine_fp4: they share one formula).  For every entry with
 * 0 <= r = tok_map[t,k] < y_rows:
 *   dy[r]   = w[t,k] * dout[t]                        (one f32 product, rounded to dy_dt)
 *   dw[t,k] = sum_h dout[t,h] * v[r,h] + dout_weights[t]
 * with v the expert output in f32, codes times their block scale for fp8 / fp4
 * (scale 1 if y_scales is NULL).  An entry without a row has dw = 0.
 *   dout          [T,H] dout_dt (MOE_BF16 or MOE_F32)
 *   dout_weights  f32 [T], the gradient of out_weights, or NULL for none
 *   y             [y_rows,H] y_dt (any of the four; fp4: [y_rows,H/2] bytes); may be
 *                 NULL when dw is NULL
 *   y_scales      f32 [y_rows,H/128] or NULL; only with MOE_FP8_E4M3 / MOE_FP4_E2M1
 *   tok_map       int64 [T,K]; each row at most once, as every dispatch writes it.
 *                 (The entries of a row named twice have their dw; each element of
 *                 its dy comes from one of them, which one is not fixed.)
 *   w             f32 [T,K]; may be NULL when dy is NULL
 *   dy            out [y_rows,H] dy_dt (MOE_BF16 or MOE_F32), or NULL: not computed
 *   packed_cnt, packed_off  int32 [E], [E+1] as the dispatch wrote them, or both NULL.
 *                 Given: the rows of dy that no entry owns (the tails of padded
 *                 segments, and the rows behind the last segment) are set to zero.
 *                 NULL: those rows are left as they were.
 *   dw            out f32 [T,K], or NULL: not computed */
int moe_combine_backward(const void* dout, moe_dtype dout_dt, const float* dout_weights,
                         int64_t T, int64_t H, const void* y, moe_dtype y_dt,
                         const float* y_scales, int64_t y_rows, const int64_t* tok_map,
                         const float* w, int K, void* dy, moe_dtype dy_dt,
                         const int32_t* packed_cnt, const int32_t* packed_off, int E, float* dw,
                         void* stream);

/* Gradient of the dispatches (moe_dispatch, its no-allocation, replay and dedup
 * forms) with respect to the token rows; a quantizing dispatch is passed straight
 * through.  For k ascending with 0 <= r = tok_map[t,k] < packed_rows:
 *   dx[t] = residual[t] + sum_k dpacked[r]      (f32; residual 0 if NULL)
 *   dpacked   [packed_rows,H] d_dt (MOE_BF16 or MOE_F32)
 *   tok_map   int64 [T,K]
 *   residual  [T,H] dx_dt, or NULL; may be dx itself (the sum is then added to it)
 *   dx        out [T,H] dx_dt (MOE_BF16 or MOE_F32) */
int moe_dispatch_backward(const void* dpacked, moe_dtype d_dt, int64_t packed_rows, int64_t H,
                          const int64_t* tok_map, int64_t T, int K, const void* residual,
                          void* dx, moe_dtype dx_dt, void* stream);

/* Embedding lookup with scaling: out[n] = scale * table[ids[n]].  A token id
 * outside [0,V) gives a zero row; -1 is "no token", any other is counted.
 *   table   [V,H] table_dt (MOE_BF16 or MOE_F32)
 *   ids     [N] integers of id_bytes (4: int32, 8: int64)
 *   out     out [N,H] out_dt (MOE_BF16 or MOE_F32)
 *   stats   int32 [1] out, may be NULL: ids outside [0,V) other than -1 */
int moe_embedding(const void* table, moe_dtype table_dt, int64_t V, int64_t H, const void* ids,
                  int id_bytes, int64_t N, float scale, void* out, moe_dtype out_dt,
                  int32_t* stats, void* stream);

/* Bytes of device workspace that moe_embedding_backward needs for these sizes (0
 * for sizes outside the limits).  For one H it does not shrink when N or V grows, so a
 * workspace for the longest batch and the largest table serves every smaller call.  It
 * needs no initialisation, may be reused by consecutive calls on one stream, of any
 * sizes it is large enough for, also from a captured graph.  Calls that may run
 * at the same time, or that several host threads enqueue at the same time, need
 * workspaces of their own. */
size_t moe_embedding_workspace_size(int64_t N, int64_t V, int64_t H);

/* Gradient of the embedding lookup with respect to the table:
 *   dtable[v] = base[v] + scale * sum over n with ids[n] = v of dout[n]
 * The sum runs over n ascending, in f32; a token that occurs often is summed in
 * runs of consecutive occurrences whose sums are then added in order.
 *   dout        [N,H] dout_dt (MOE_BF16 or MOE_F32)
 *   ids         as for moe_embedding; ids outside [0,V) are skipped
 *   accumulate  0: base is 0 and every row of dtable is written (zeros for tokens
 *               that do not occur).  Otherwise: base is dtable itself, and rows of
 *               tokens that do not occur are neither read nor written.
 *   dtable      [V,H] dtable_dt (MOE_BF16 or MOE_F32)
 *   ws          at least moe_embedding_workspace_size(N, V, H) bytes, 256-byte aligned */
int moe_embedding_backward(const void* dout, moe_dtype dout_dt, const void* ids, int id_bytes,
                           int64_t N, int64_t V, int64_t H, float scale, int accumulate,
                           void* dtable, moe_dtype dtable_dt, void* ws, size_t ws_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */
