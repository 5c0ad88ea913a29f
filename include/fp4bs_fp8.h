/*
 * fp4bs_fp8.h - 8-bit (E4M3) products with one scale to each block of 128, their quantizers, and
 * the gated feed-forward projections built on them, in the same library (libfp4bs.so) and with the
 * conventions of fp4bs.h: caller-owned device buffers, stream order, no host synchronisation,
 * arguments validated before anything is enqueued, fp4_last_error() for the message.
 *
 *   fp8_quantize       bf16 / float32 -> E4M3 operands (row, transposed, both, 128 x 128 tiles)
 *   fp8_dequantize     their values
 *   fp8_gemm           y = a . b^T: forward, gradient of the input, gradient of the weight
 *   fp8_expert_gemm    the same for rows in expert order, each with its expert's weight
 *   fp8_gated          h = act(x . Wg^T) * (x . Wu^T) in one product, also over experts
 *   gated_grad         gradient of the two projections, plain
 *   fp8_gated_grad     the same as the operands of the next two products
 *
 * An operand [rows x k] is
 *   q   E4M3 codes (bias 7, 0x7F / 0xFF NaN), one byte each, rows of kp = k rounded up to whole
 *       blocks of 128 bytes, packed; the bytes past k are zero codes (fp8_quantize writes them; NaN
 *       codes where the block is NaN throughout)
 *   s   scales: E8M0 codes (value 2^(c - 127)) or float32, packed, by layout:
 *         FP4_SCALES_1D    [rows x kp / 128]                 a block is 128 of a row
 *         FP4_SCALES_2D    [ceil(rows / 128) x kp / 128]     a block is 128 x 128
 *         FP4_SCALES_2D_T  [kp / 128 x ceil(rows / 128)]     the same grid for the transposed operand
 * q is 16-byte aligned, s aligned to its elements. fp4_mxfp4_to_fp8 (not transposed) writes such an
 * operand with E8M0 scales.
 */
#ifndef FP4BS_FP8_H
#define FP4BS_FP8_H

#include "fp4bs.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { FP8_SCALE_E8M0 = 0, FP8_SCALE_F32 = 1 };
enum { FP8_VIEW_ROWCOL = 3 };                     /* beside FP4_VIEW_ROW, _COL and _TILE2D */
enum { FP8_ACT_SILU = 0, FP8_ACT_GELU = 1, FP8_ACT_GELU_TANH = 2 };
enum { FP8_OUT_E4M3 = 2 };                        /* beside FP4_IN_BF16 and FP4_IN_FP32 */

typedef struct {
  const uint8_t* q;
  const void* s;
  int32_t scale;    /* FP8_SCALE_* */
  int32_t layout;   /* FP4_SCALES_* */
  int64_t rows, k;
} fp8_operand;

/*
 * fp8_quantize - x [rows x cols] as E4M3 operands.
 *   x         device, bf16 or float32, row stride ld elements (>= cols; element aligned)
 *   view      FP4_VIEW_ROW     q, s: x with 1D scales
 *             FP4_VIEW_COL     qt, st: x^T [cols x rows] with 1D scales
 *             FP8_VIEW_ROWCOL  both from one read
 *             FP4_VIEW_TILE2D  q, qt: x and x^T, s: their one grid of 128 x 128 tiles' scales
 *                              (2D for q, 2D_T for qt)
 * With a = max |x| of a block: E8M0 S = 2^ceil(log2(a / 448)), at least 2^-127; float32
 * S = a' / 448 with a' = max(a, 2^-100); S = 1 for a block of zeros. The codes are
 * E4M3(x * 2^-e) or E4M3(x * (448 / a')), float32 arithmetic, nearest-even. A block that holds an
 * infinity or NaN gets NaN codes throughout and S = 1.
 * rows below 2^31, ld at most 2^22, fewer than 2^24 tiles of 128 x 128. Rows need only be aligned to their
 * elements; base addresses and strides that are multiples of 16 bytes take a faster form. Pointers a view
 * does not write may be NULL.
 */
fp4_status fp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld, int32_t view,
                        int32_t scale, uint8_t* q, void* s, uint8_t* qt, void* st, void* stream);

/* fp8_dequantize - y [rows x k] = code * S (float32 product), row stride ldy, rounded to y_dtype. Rows and k below 2^31. */
fp4_status fp8_dequantize(const fp8_operand* a, void* y, int32_t y_dtype, int64_t ldy, void* stream);

/*
 * fp8_gemm - y[m][n] = sum over blocks c of Sa(m, c) Sb(n, c) sum_{k in c} a[m][k] b[n][k].
 *   a    1D scales; b any layout; both of one scale type and the same k
 *   y    device, [a->rows x b->rows] of y_dtype (FP4_IN_BF16 / FP4_IN_FP32), row stride ldy
 *        (>= b->rows; element aligned)
 *   ws   device workspace of at least the bytes fp8_gemm_workspace gives (16-byte aligned; may be
 *        NULL when that is 0)
 * Blocks' sums are added in float32 over all of k and rounded once to y_dtype; their order depends on the sizes
 * and the device only, so equal calls give equal bits. For a bf16 y the E4M3 matrix core adds a block's products
 * in a window narrower than float32: a block's sum is off by about 1.5e-5 of its norm, the root of the sum of its
 * products' squares. That does not add up over k (128 to 131072 measured, products of one sign too). It is below 1% of
 * y's rounding where y is as large as its products' norm; a y that cancels below that keeps the error. For a
 * float32 y the codes are widened to bf16, exactly, and the sums are those of the bf16 matrix core, at less than
 * half the rate. Float32 scales, and for a float32 y also E8M0 ones, multiply as the float32 product of a block's
 * two scales (infinite from 2^128 on). k = 0 gives zeros. k at most 2^22, rows below 2^31, one weight below 2^37
 * bytes.
 *
 * fp8_expert_gemm - rows of x in expert order: row p with offsets[e] <= p < offsets[e + 1] uses
 * expert e's weight; rows from offsets[n_experts] on are written as zeros.
 *   w        expert 0's weight; expert e's codes and scales follow at e times one expert's bytes
 *   offsets  device int32 [n_experts + 1], ascending from 0, at most rows (fp4_expert_sort)
 * n_experts in [1, 1024].
 *
 * fp8_gated - h[m][j] = act(g) * u with g = (x . w^T)[m][j], u = (x . w^T)[m][f + j]: w stacks the
 * gate's f rows and the up projection's (w->rows = 2 f). n_experts 0: one weight, offsets NULL.
 *   h        [x->rows x f] of h_kind: FP4_IN_BF16, FP4_IN_FP32 (row stride ldh), or FP8_OUT_E4M3: the
 *            operand of the next product, codes [rows x f in whole blocks] (ldh ignored, 16-byte
 *            aligned) and 1D scales hs of x's scale type, from the float32 h as fp8_quantize would
 *   gu       NULL, or the projections [x->rows x 2 f] of gu_dtype, row stride ldgu, for the gradient
 * act and the product are taken in float32 on the unrounded projections, whose sums are those of a
 * float32 y above where h or gu is float32, and those of a bf16 y otherwise (codes of h that stand at a
 * rounding boundary, and the scale of a block whose maximum stands at one, then differ from those of exact
 * sums; a float32 gu gives the latter). The sigmoid takes the hardware's exponential and reciprocal, the
 * normal distribution in GELU an approximation within 1.5e-7: act(g) is off by at most 1.3e-7 (1 + |g|) and
 * act'(g) by 3.4e-7 (1 + |g|) before any rounding, measured over |g| <= 30.
 *
 * A launch holds fewer than 2^32 threads: calls of 2^23 or more tiles of 128 or 256 rows, or of 2^24 or more lower
 * ones, return FP4_EUNSUPPORTED (fp8_gemm_form gives the tiles; an expert counts one more row of them). Fewer than
 * 2^22 tiles of 32 x 128 are always accepted.
 */
fp4_status fp8_gemm(const fp8_operand* a, const fp8_operand* b, void* y, int32_t y_dtype, int64_t ldy, void* ws,
                    size_t ws_bytes, void* stream);
fp4_status fp8_expert_gemm(const fp8_operand* x, const fp8_operand* w, int32_t n_experts, const int32_t* offsets,
                           void* y, int32_t y_dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream);
fp4_status fp8_gated(const fp8_operand* x, const fp8_operand* w, int32_t n_experts, const int32_t* offsets,
                     int32_t act, void* h, int32_t h_kind, int64_t ldh, void* hs, void* gu, int32_t gu_dtype,
                     int64_t ldgu, void* ws, size_t ws_bytes, void* stream);
/* Bytes of ws for the three calls (n_experts 0: one weight; gated 0, 1, or 2 for h as codes; f32 1 where y, h
 * or gu is float32), from rows of x and w's sizes: w's pointers are not looked at. */
fp4_status fp8_gemm_workspace(int64_t rows, const fp8_operand* w, int32_t n_experts, int32_t gated, int32_t f32,
                              size_t* ws_bytes);
/* How those calls run on the current device, from the same sizes, for tests and profiles: form[0] rows of an
 * output tile (0: the form for few rows, or nothing to do), form[1] its columns, form[2] the parts that K is split
 * into, form[3] whose scales are copied turned first (1: x's, 2: w's, 3: both). */
fp4_status fp8_gemm_form(int64_t rows, const fp8_operand* w, int32_t n_experts, int32_t gated, int32_t f32,
                         int32_t* form);

/*
 * gated_grad - dgu[m][j] = dh u act'(g), dgu[m][f + j] = dh act(g) in float32, rounded once.
 *   dh   [rows x f], gu and dgu [rows x 2 f], all of dtype (bf16 or float32), row strides lddh, ldgu, lddgu;
 *        dgu may be gu itself (same stride)
 * fp8_gated_grad - the same as operands of the next products: q, s the row view [rows x 2 f] with 1D
 * scales (dx = dgu . W), qt, st the transposed one [2 f x rows] (dW = dgu^T . x). Either pair may be
 * NULL. f must be a multiple of 128 (pad gate and up each with zero rows), lddh and ldgu at most 2^22; fewer
 * than 2^24 tiles of 128 x 128 of dh, 2^23 for float32.
 */
fp4_status gated_grad(const void* dh, int32_t dtype, int64_t rows, int64_t f, int64_t lddh, const void* gu,
                      int64_t ldgu, int32_t act, void* dgu, int64_t lddgu, void* stream);
fp4_status fp8_gated_grad(const void* dh, int32_t dtype, int64_t rows, int64_t f, int64_t lddh, const void* gu,
                          int64_t ldgu, int32_t act, int32_t scale, uint8_t* q, void* s, uint8_t* qt, void* st,
                          void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4BS_FP8_H */
