/*
 * fp4bs_experts.h - the operators around FP4 weights that a mixture-of-experts layer needs, in
 * the same library (libfp4bs.so) and with the conventions of fp4bs.h: caller-owned device
 * buffers, stream order, no host synchronisation, arguments validated before anything is
 * enqueued, fp4_last_error() for the message.
 *
 *   fp4_expert_sort          slots sorted by expert
 *   fp4_expert_gather        token rows -> expert order          (+ fp4_expert_gather_grad)
 *   fp4_linear               y = x . W^T, bf16 / float32 x and an FP4 weight
 *   fp4_expert_linear        the same for rows in expert order, each with its expert's weight
 *   fp4_expert_combine       expert rows -> weighted sum per token (+ fp4_expert_combine_grad)
 *
 * A slot is one (token, choice) pair, s = token * topk + choice; n = tokens * topk slots in all
 * (n < 2^31). A position is a row of the expert-ordered tensors, which have n rows: the kept
 * slots first, by expert and then by slot, then the dropped ones by slot. Rows of dropped slots
 * are written as zeros wherever an entry point writes expert-ordered rows, and never read.
 */
#ifndef FP4BS_EXPERTS_H
#define FP4BS_EXPERTS_H

#include "fp4bs.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp4_expert_sort - stable counting sort of the slots by expert.
 *   ids      device int32 (ids_int64 0) or int64 (1), [tokens x topk], row stride ld_ids. An id
 *            outside [0, n_experts) drops its slot.
 *   order    device int32 [n]: order[position] = slot
 *   pos      device int32 [n]: pos[slot] = position of a kept slot, ~position (negative) of a
 *            dropped one
 *   offsets  device int32 [n_experts + 1]: expert e holds positions offsets[e] .. offsets[e+1];
 *            offsets[n_experts] is the number of kept slots
 *   ws       device workspace of at least the bytes fp4_expert_sort_workspace gives (4-byte
 *            aligned; may be NULL when that is 0)
 * n_experts in [1, 1024]. tokens = 0 writes the offsets only.
 */
fp4_status fp4_expert_sort(const void* ids, int32_t ids_int64, int64_t tokens, int32_t topk, int64_t ld_ids,
                           int32_t n_experts, int32_t* order, int32_t* pos, int32_t* offsets, void* ws,
                           size_t ws_bytes, void* stream);
fp4_status fp4_expert_sort_workspace(int64_t tokens, int32_t topk, int32_t n_experts, size_t* ws_bytes);

/*
 * fp4_expert_gather - xs[pos[s]] = x[s / topk] for kept slots, zeros for dropped ones.
 * fp4_expert_gather_grad - dx[t] = the sum of dxs[pos[s]] over t's kept slots, in slot order in
 * float32, rounded once (zeros when t keeps none).
 *   x / dx   device, [tokens x hidden] of dtype (FP4_IN_BF16 or FP4_IN_FP32), row stride ldx
 *   xs / dxs device, [tokens * topk x hidden] of the same dtype, row stride ldxs
 *   pos      device int32 [tokens x topk] as fp4_expert_sort writes it; a value that is neither a
 *            position nor ~position below n is skipped
 * Rows need only be aligned to their elements; base addresses and strides that are multiples of
 * 16 bytes take the faster 16-byte form.
 */
fp4_status fp4_expert_gather(const void* x, int32_t dtype, int64_t tokens, int64_t hidden, int64_t ldx,
                             const int32_t* pos, int32_t topk, void* xs, int64_t ldxs, void* stream);
fp4_status fp4_expert_gather_grad(const void* dxs, int32_t dtype, int64_t tokens, int64_t hidden, int64_t ldxs,
                                  const int32_t* pos, int32_t topk, void* dx, int64_t ldx, void* stream);

/*
 * fp4_expert_combine - y[t] = sum over t's kept slots of w[s] * ys[pos[s]], in slot order in
 * float32, rounded once (zeros when t keeps none).
 * fp4_expert_combine_grad - its gradients: dys[pos[s]] = w[s] * dy[s / topk] (zeros for dropped
 * slots) and dw[s] = <dy[s / topk], ys[pos[s]]> in float32 (0 for dropped slots). Either of dys
 * and dw may be NULL; ys may be NULL without dw, and w without dys.
 *   w, dw    device float32 [tokens x topk], row strides ldw, lddw
 *   the rest as in fp4_expert_gather
 */
fp4_status fp4_expert_combine(const void* ys, int32_t dtype, int64_t tokens, int64_t hidden, int64_t ldys,
                              const float* w, int64_t ldw, const int32_t* pos, int32_t topk, void* y, int64_t ldy,
                              void* stream);
fp4_status fp4_expert_combine_grad(const void* dy, int32_t dtype, int64_t tokens, int64_t hidden, int64_t lddy,
                                   const void* ys, int64_t ldys, const float* w, int64_t ldw, const int32_t* pos,
                                   int32_t topk, void* dys, int64_t lddys, float* dw, int64_t lddw, void* stream);

/*
 * fp4_linear - y[m][n] = g * sum_k x[m][k] E2M1(q[n][k]) S(n, k): activations that are not
 * quantized times an FP4 weight.
 *   x        device, [rows x K] of x_dtype, row stride ldx elements (16-byte aligned rows)
 *   w        the weight: any format, block, scale layout and g (NULL, one float or stripes) that
 *            the GEMMs take; N = w->rows, K = w->k. The forward view of a weight gives X . W^T,
 *            the transposed view (FP4_SCALES_2D_T) of the same weight dX = dY . W; with 1D scales
 *            dX takes the weight's COL view (FP4_VIEW_COL), quantized for itself. Scale
 *            codes 4-byte aligned; K and ldx at most 2^22, rows and N below 2^31.
 *   y        device, [rows x N] of y_dtype, row stride ldy elements (>= N; element aligned)
 *   ws       device workspace of at least the bytes fp4_linear_workspace gives (16-byte aligned;
 *            may be NULL when that is 0)
 * Arithmetic: E2M1 * S is exact in bfloat16. (E8M0 codes 253 and 254, which fp4_quantize writes for no
 * finite weight, make products from 2^128 on: they are infinite, as in float32.) bf16 x: bf16 matrix
 * products accumulated in float32. float32 x: each element is split into three bf16 parts, whose
 * products accumulate in the same float32 sums; the parts add up to x exactly from magnitude 2^-110
 * on, below it bits under 2^-133 (bfloat16's least subnormal) are dropped; an infinite product with
 * a weight that is itself infinite is NaN. The sum, over all of K, is multiplied by g in float32 and
 * rounded once to y_dtype. The order of the sums depends on the sizes and the device only: equal
 * calls give equal bits. K = 0 gives zeros.
 *
 * fp4_expert_linear - rows in expert order: row p with offsets[e] <= p < offsets[e+1] uses
 * expert e's weight; rows from offsets[n_experts] on are written as zeros.
 *   w        expert 0's weight; expert e's payload, scale codes and g follow at e times the bytes of
 *            one expert's (N * K / 2; N * K / block or N * K / 256; 1 or ceil(N / g_stripe) floats)
 *   offsets  device int32 [n_experts + 1], ascending from 0, at most rows (fp4_expert_sort)
 * n_experts in [1, 1024]. Weights of experts without rows are not read.
 *
 * Either call returns FP4_EUNSUPPORTED where its output tiles (of at least 32 x 256, and one more row of
 * tiles to an expert) are 2^23 or more: rows * N or n_experts * N above 2^31 may be so many.
 */
fp4_status fp4_linear(const void* x, int32_t x_dtype, int64_t rows, int64_t ldx, const fp4_operand* w, void* y,
                      int32_t y_dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream);
fp4_status fp4_expert_linear(const void* x, int32_t x_dtype, int64_t rows, int64_t ldx, const fp4_operand* w,
                             int32_t n_experts, const int32_t* offsets, void* y, int32_t y_dtype, int64_t ldy,
                             void* ws, size_t ws_bytes, void* stream);
/* Bytes of ws for either call (n_experts 0: fp4_linear), from the sizes alone: w's pointers are not looked at. */
fp4_status fp4_linear_workspace(int64_t rows, int32_t x_dtype, const fp4_operand* w, int32_t n_experts,
                                size_t* ws_bytes);

#ifdef __cplusplus
}
#endif
#endif /* FP4BS_EXPERTS_H */
