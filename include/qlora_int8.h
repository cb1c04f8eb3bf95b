/*
 * qlora_int8.h -- C ABI of the linear layer in 8-bit integers (gfx950).
 * The conventions of qlora_nf4.h (pointers, streams, ownership, errors) hold.
 */
#ifndef QLORA_INT8_H
#define QLORA_INT8_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* type of a matrix that qlora_int8_quantize reads */
#define QLORA_TYPE_BF16 QLORA_COMPUTE_BF16
#define QLORA_TYPE_FP16 QLORA_COMPUTE_FP16
#define QLORA_TYPE_FP32 2

/*
 * The linear layer in 8-bit integers: a weight whose adapter is merged
 * (qlora_nf4_merge) served with one scale a channel, the activations with one
 * scale a token,
 *   Y_tn = round16( x_scale_t * w_scale_n * sum_k xq_tk wq_nk ).
 * The sum is exact (32-bit integers; cols at most 2^17 - 16, so it cannot
 * overflow); it is converted to float32 and multiplied by w_scale_n and then
 * by x_scale_t, and rounded once to the 16-bit type.
 *
 * qlora_int8_quantize: rows of X [rows, cols] (x_type QLORA_TYPE_*) to codes
 * [rows, cols] and scale [rows], both written:
 *   scale_i = RN32(max_k |x_ik| / 127),
 *   code_ik = the integer nearest to the real quotient x_ik / scale_i, ties
 *             to even, within -127 .. 127; a row whose scale is 0 (all zeros,
 *             or a maximum that rounds to it) gets codes 0.  A row that holds
 *             an infinity or a NaN gets codes 0 and an infinite or NaN scale,
 *             so every output of that channel or token is NaN.
 * Rows are output channels of a weight or tokens of the activations.
 * rows >= 0 (0: nothing is done, X, codes and scale may be NULL), at most
 * 2^22 - 1; cols a multiple of 16, 16 .. 2^17 - 16.
 */
qlora_status qlora_int8_quantize(const void *X, int x_type, int64_t rows, int64_t cols,
                                 int8_t *codes, float *scale, void *stream);

/* Workspace bytes of qlora_int8_matmul (x_given = 1: the tokens' codes are
 * given) or qlora_int8_linear_fwd (x_given = 0); 0 on bad arguments, for
 * T = 0, and where none is needed (ws may then be NULL). */
size_t qlora_int8_workspace(int64_t T, int64_t rows, int64_t cols, int x_given);

/*
 * Y [T, rows] of codes: W [rows, cols] int8 with w_scale [rows], X [T, cols]
 * int8 with x_scale [T]; Y is bf16 or fp16 by compute_dtype (QLORA_COMPUTE_*).
 * T >= 0 (0 writes nothing; X, x_scale, Y and ws may be NULL), at most
 * 2^22 - 1; rows >= 1, at most 2^22 - 1; cols a multiple of 16, 16 .. 2^17 -
 * 16; T * rows below 2^36 (QLORA_ERR_SHAPE otherwise).  QLORA_ERR_FORMAT for another
 * compute_dtype.  Codes of -128 are taken as they are.
 */
qlora_status qlora_int8_matmul(const int8_t *W, const float *w_scale, int64_t rows, int64_t cols,
                               const int8_t *X, const float *x_scale, int64_t T,
                               int compute_dtype, uint16_t *Y, void *ws, size_t ws_bytes,
                               void *stream);

/*
 * The same with 16-bit tokens X [T, cols] (bf16 or fp16 by compute_dtype),
 * quantised by token within the call; same result as qlora_int8_quantize
 * followed by qlora_int8_matmul, bit for bit.
 */
qlora_status qlora_int8_linear_fwd(const int8_t *W, const float *w_scale, int64_t rows,
                                   int64_t cols, const uint16_t *X, int64_t T, int compute_dtype,
                                   uint16_t *Y, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_INT8_H */
