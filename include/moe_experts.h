/*
 * moe_experts.h - C ABI of the experts' step of the MI355X (gfx950) MoE library
 * (libmoe_route.so): what lies between the dispatch and the combine of
 * moe_route.h, and what its gradient keeps.
 *
 * The conventions of moe_route.h hold for every entry point here: device
 * pointers, row-major layouts without gaps between rows, buffers owned by the
 * caller, work enqueued on `stream` without waiting, every argument checked on
 * the host before anything is enqueued, deterministic results, no output that
 * needs clearing between calls.  Sums and products are held in f32; a bf16 output
 * is rounded once, to nearest even, when it is stored.  Input and output buffers
 * must not overlap.
 *
 * MXFP4: a row of H elements (H % 32 == 0) is H/2 bytes of OCP e2m1 codes (element
 * 2i in the low nibble of byte i) and, in an array of its own, H/32 e8m0 scale
 * bytes, one per block of 32 elements: byte s stands for 2^(s-127), 255 for NaN.
 *
 * Segments: packed_cnt [E] and packed_off [E+1] as a dispatch wrote them: expert e
 * owns rows packed_off[e] .. packed_off[e] + packed_cnt[e] - 1.  The offsets ascend.
 * Rows outside every segment (the tails of padded segments, rows behind the last
 * one) are neither read nor written; parts of a segment outside the buffer are
 * skipped.
 *
 * Limits: row counts in [0, 2^31-1]; 1 <= E <= 1024; row lengths in (0, 2^24]; row
 * buffers 16-byte aligned.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows to MXFP4.  Per block, with amax the largest finite magnitude: the scale is
 * the power of two 2^e with amax / 2^e in [3.5, 7), at least 2^-127 (1 for a block
 * without a finite value other than 0), and a code is x / 2^e rounded to nearest
 * even and saturated at +-6 (infinities too; zeros keep their sign).  A block with a
 * NaN gets zero codes and the NaN scale.
 *   x       [rows,H] x_dt (MOE_BF16 or MOE_F32), H % 32 == 0
 *   codes   out [rows,H/2] bytes, 16-byte aligned
 *   scales  out [rows,H/32] bytes */
int moe_mxfp4_quantize(const void* x, moe_dtype x_dt, int64_t rows, int64_t H, void* codes,
                       void* scales, void* stream);

/* The values of MXFP4 rows: y = code * 2^(s-127), in f32, rounded to y_dt (which
 * changes only values outside y_dt's normal range).
 *   codes, scales  as moe_mxfp4_quantize writes them
 *   y       out [rows,H] y_dt (MOE_BF16 or MOE_F32) */
int moe_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t H, void* y,
                         moe_dtype y_dt, void* stream);

/* The product of packed rows with their experts' weights, both in MXFP4 (sums in f32):
 *   y[r,n] = sum_h a[r,h] * w[e,n,h]     for every row r of expert e's segment
 * or, with swiglu != 0, where a weight matrix is I gate rows and then I up rows, N = 2I:
 *   y[r,i] = silu(sum_h a[r,h] * w[e,i,h]) * sum_h a[r,h] * w[e,I+i,h]
 * E = 1 with one segment is an ordinary product.  Segments must not overlap (no dispatch
 * makes such): rows of those that do may be left as they were, or hold the result of
 * either expert.
 *   a, a_scales  [rows,H/2] codes (16-byte aligned), [rows,H/32] scales, H % 32 == 0
 *   w, w_scales  [E,N,H/2] codes (16-byte aligned), [E,N,H/32] scales,
 *           N % 8 == 0 (N % 16 == 0 with swiglu), N <= 2^24
 *   packed_cnt, packed_off  the segments
 *   y       out [rows,N] (swiglu: [rows,N/2]) y_dt (MOE_BF16 or MOE_F32) */
int moe_expert_product_mxfp4(const void* a, const void* a_scales, int64_t rows, int64_t H,
                             const void* w, const void* w_scales, int64_t N,
                             const int32_t* packed_cnt, const int32_t* packed_off, int E,
                             int swiglu, void* y, moe_dtype y_dt, void* stream);

/* Bytes of device workspace that moe_experts_decode needs for these sizes (0 for sizes
 * outside its limits).  It does not shrink when T, K, H or I grows, so one for the largest
 * sizes serves all; it needs no initialisation and may be reused by consecutive calls on
 * one stream, also from a captured graph.
 * Calls that may run at the same time, or that several host threads enqueue at the same time,
 * need workspaces of their own. */
size_t moe_experts_decode_workspace_size(int64_t T, int K, int64_t H, int64_t I);

/* The whole experts' step of a few tokens (T*K <= 1024; H, I <= 2^20), from token rows to
 * token rows, without a dispatch or a combine:
 *   out[t] = sum over k of w[t,k] * W2[e] h,  h = silu(W1[e] x[t]) * (W3[e] x[t]),  e = idx[t,k]
 * The sum over k ascends, in f32; entries whose idx is outside [0,E) are skipped whatever
 * their w holds, and a token without any other gets zeros.  h is held between the
 * products with at least 16 bits of significand (24 for an f32 result), small ones to within
 * 2^-134, and finite if it is finite in f32.
 *   x       [T,H] MOE_BF16
 *   idx     int32 [T,K]; w f32 [T,K]
 *   w13     [E,2I,H], I rows of W1 and then I of W3 per expert: wt_dt MOE_BF16
 *           (H % 8 == 0, I % 8 == 0), or MOE_FP4_E2M1: MXFP4 codes with w13_scales
 *           [E,2I,H/32] (H % 32 == 0, I % 32 == 0); a value past bf16's largest is
 *           infinite (infinite weights give infinities as in the formula, 0 times one NaN)
 *   w2      [E,H,I], likewise, with w2_scales [E,H,I/32]; both scales NULL for bf16
 *   out     out [T,H] out_dt (MOE_BF16 or MOE_F32)
 *   ws      at least moe_experts_decode_workspace_size(T, K, H, I) bytes, 256-byte aligned */
int moe_experts_decode(const void* x, int64_t T, int64_t H, const int32_t* idx, const float* w,
                       int K, int E, int64_t I, const void* w13, const void* w13_scales,
                       const void* w2, const void* w2_scales, moe_dtype wt_dt, void* out,
                       moe_dtype out_dt, void* ws, size_t ws_bytes, void* stream);

/* SwiGLU of packed rows, h[r,i] = silu(gu[r,i]) * gu[r,I+i], silu(g) = g / (1 + exp(-g))
 * (here and in the products an exp(-|g|) below 2^-126 counts as 0), and on request the
 * 8-bit checkpoint of gu that moe_swiglu_backward takes.
 *   gu      [rows,2I] gu_dt (MOE_BF16 or MOE_F32), I % 8 == 0
 *   packed_cnt, packed_off  the segments (E experts), or both NULL: every row
 *   h       out [rows,I] h_dt (MOE_BF16 or MOE_F32)
 *   codes   out [rows,2I] e4m3 codes, or NULL: no checkpoint.  Needs I % 128 == 0.
 *   scales  out f32 [rows,2I/128], with codes: per block of 128 elements the smallest
 *           power of two s >= 2^-126 with amax <= 448 s over the block's finite values
 *           (1 if they are all 0).  A code is x / s rounded to nearest even;
 *           infinities saturate at +-448 and a NaN gets the NaN code with its sign.
 *           moe_fp8_dequant gives the kept values. */
int moe_swiglu(const void* gu, moe_dtype gu_dt, int64_t rows, int64_t I,
               const int32_t* packed_cnt, const int32_t* packed_off, int E, void* h,
               moe_dtype h_dt, void* codes, float* scales, void* stream);

/* Gradient of moe_swiglu.  With s = 1 / (1 + exp(-g)):
 *   dgu[r,i]   = dh[r,i] * u * s * (1 + g * (1 - s)),   dgu[r,I+i] = dh[r,i] * g * s
 * for g = gu[r,i], u = gu[r,I+i], and on request h again (which the gradient of the
 * second product needs), so that a training step keeps nothing of this layer but the
 * checkpoint.
 *   dh      [rows,I] dh_dt (MOE_BF16 or MOE_F32)
 *   gu      [rows,2I] gu_dt: MOE_BF16, MOE_F32 (I % 8 == 0), or MOE_FP8_E4M3 codes
 *           (I % 128 == 0), whose values are code * scale
 *   gu_scales  f32 [rows,2I/128] with MOE_FP8_E4M3, else NULL
 *   packed_cnt, packed_off  the segments (E experts), or both NULL: every row
 *   dgu     out [rows,2I] out_dt (MOE_BF16 or MOE_F32)
 *   h       out [rows,I] out_dt, or NULL: not computed */
int moe_swiglu_backward(const void* dh, moe_dtype dh_dt, const void* gu, moe_dtype gu_dt,
                        const float* gu_scales, int64_t rows, int64_t I,
                        const int32_t* packed_cnt, const int32_t* packed_off, int E, void* dgu,
                        void* h, moe_dtype out_dt, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
