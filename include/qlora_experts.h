/*
 * qlora_experts.h -- C ABI of the expert-grouped NF4 linear layer with LoRA
 * adapters (gfx950).
 * The conventions of qlora_nf4.h (pointers, streams, ownership, errors) hold.
 */
#ifndef QLORA_EXPERTS_H
#define QLORA_EXPERTS_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The linear layer of a mixture of experts: `experts` frozen NF4 weights of
 * one shape with a LoRA adapter each, applied to rows sorted by expert,
 *   U_t = X_t A_e^T,   Y_t = X_t dequant(W_e)^T + s U_t B_e^T,   s = alpha / r
 * for the rows t of expert e, offsets[e] <= t < offsets[e + 1].
 *   w        the experts' weights stacked along the rows: [experts * rows,
 *            cols], expert e's rows e * rows .. (e + 1) * rows - 1 (one
 *            qlora_nf4_quantize of the stack); w->rows % (16 * experts) == 0.
 *   offsets  [experts + 1] int32 in DEVICE memory, 16-byte aligned, read by
 *            the kernels (the host never sees the counts): not decreasing,
 *            within 0 .. T.  Experts may have no rows.  Rows before
 *            offsets[0] and from offsets[experts] on belong to no expert:
 *            they are not read, and their rows of Y, U_save and dX keep what
 *            they held.  Offsets outside 0 .. T are taken as the nearest
 *            bound and a group that ends before it starts as empty; with
 *            offsets that decrease the outputs are unspecified, but nothing
 *            outside the given buffers is touched.
 *   X        [T, cols], A [experts, r, cols], B [experts, rows, r],
 *   Y        [T, rows] (written), U_save [T, r] (written, or NULL): 16-bit in
 *            the weight's compute dtype.
 * 1 <= experts <= 1024; T, rows, cols and r as in qlora_linear_fwd, and T * r
 * below 2^28, rows and cols at most 2^20.  The weights are the values
 * qlora_nf4_dequantize gives; sums are float32.  s U meets B as the sum of
 * two 16-bit terms (16 bits of s U in bf16; 22 in fp16, but no closer than
 * 2^-25 and only up to 65504), so the rounding of Y is the largest
 * (qlora_linear_fwd rounds s U to one 16-bit number).
 * T = 0 writes nothing; X, Y, U_save and ws may be NULL.
 * Few rows an expert on average (at most 24; 32 with up to 8 experts, 64 with
 * up to 2^26 weights in all) take kernels that stream the touched experts'
 * weights, more take the tiled GEMM.
 */
qlora_status qlora_grouped_linear_fwd(const qlora_nf4_weight *w, int32_t experts,
                                      const uint16_t *X, int64_t T, const int32_t *offsets,
                                      const uint16_t *A, const uint16_t *B, int32_t r,
                                      float alpha, uint16_t *Y, uint16_t *U_save, void *ws,
                                      size_t ws_bytes, void *stream);

/*
 * Backward of the same (no gradient for the frozen weights):
 *   G_t = dY_t B_e,  dX_t = dY_t dequant(W_e) + s G_t A_e   [T, cols] 16-bit
 *   dA_e = s G_e^T X_e   [experts, r, cols] float32
 *   dB_e = s dY_e^T U_e  [experts, rows, r] float32
 * all written; experts without rows get zeros in dA and dB.  U_saved is the
 * forward's U_save (required).
 * G is split into 16-bit terms whose products add up in float32: on its way
 * to dX two (16 bits of G in bf16, 22 in fp16), on its way to dA three in bf16
 * (24 bits of G) and two in fp16 (22 bits).  The fp16 terms are those of G
 * times a power of two, one for each 128 rows of an expert, that brings their
 * largest G below 2^15, so dX and dA keep their bits whatever the size of dY
 * and B: a G far below the largest of its 128 rows is off by at most 2^-38 S
 * of their largest float32 partial sum, where G is summed in S <= 128 parts.
 * Where X or G is not finite, the entries of dA that it meets are infinite or
 * NaN.  T = 0 zeroes dA and dB; X, dY, U_saved, dX and ws may then be NULL.
 */
qlora_status qlora_grouped_linear_bwd(const qlora_nf4_weight *w, int32_t experts,
                                      const uint16_t *X, const uint16_t *dY, int64_t T,
                                      const int32_t *offsets, const uint16_t *A,
                                      const uint16_t *B, int32_t r, float alpha,
                                      const uint16_t *U_saved, uint16_t *dX, float *dA, float *dB,
                                      void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes for qlora_grouped_linear_fwd (is_bwd = 0) or _bwd (1) with
 * T rows, `experts` experts of [rows, cols] each, rank r and the weight's
 * compute_dtype (0 on bad arguments, and for T = 0). */
size_t qlora_grouped_linear_workspace(int64_t T, int32_t experts, int64_t rows, int64_t cols,
                                      int32_t r, int compute_dtype, int is_bwd);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_EXPERTS_H */
