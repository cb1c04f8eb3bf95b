/*
 * qlora_gated.h -- C ABI of the gated feed-forward block over frozen NF4
 * weights with LoRA adapters (gfx950).
 * The conventions of qlora_nf4.h (pointers, streams, ownership, errors) hold.
 */
#ifndef QLORA_GATED_H
#define QLORA_GATED_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* activation of a gated block: act(g) = g sigmoid(z), z = g (SiLU) or
 * z = 2 sqrt(2 / pi) (g + 0.044715 g^3) (the tanh form of GELU) */
#define QLORA_ACT_SILU 0
#define QLORA_ACT_GELU_TANH 1

/*
 * The first half of a gated feed-forward block: two linear layers of the same
 * shape over the same tokens (qlora_linear_fwd's P = X dequant(W)^T + (alpha /
 * r) (X A^T) B^T, the gate's and the up projection's), the activation and the
 * product,
 *   H = round16( act(P_gate) * P_up ),
 * with P in float32.  U = X A^T meets B in float32 for few tokens (up to 48; 64
 * on weights of at most 2^23), beyond as the sum of two 16-bit terms (16 bits of U
 * in bf16, 22 in fp16); s enters afterwards, in float32.  The fp16 terms are those
 * of U times a power of two, one for each 128 tokens, that brings their largest U
 * below 2^15, so P keeps its bits whatever the size of U: a U far below the largest
 * of its 128 tokens is off by at most 2^-38 S of their largest float32 partial
 * sum, where U is summed in S <= 64 parts.  What follows is a linear layer of its
 * own (qlora_linear_fwd with H as its X).
 *
 * gate and up: [rows, cols], NF4, the same shape and the same format
 * (QLORA_ERR_SHAPE, QLORA_ERR_FORMAT otherwise); A [r, cols], B [rows, r], X
 * [T, cols], H [T, rows] in the weights' compute dtype.  Limits of T, rows,
 * cols and r as for qlora_linear_fwd, and T * r below 2^28.  act: QLORA_ACT_*
 * (QLORA_ERR_FORMAT otherwise).  There is no lora_dropout here: a block trained
 * with it takes two qlora_linear_fwd_dropout calls.
 *
 * For the backward pass: P_gate, P_up [T, rows], P rounded to 16 bits, and
 * U_gate, U_up [T, r], U rounded to 16 bits (fp16: infinite past 65504).  All
 * four are written, or all four NULL (inference); QLORA_ERR_NULL otherwise.
 * T = 0 writes nothing (X, H, these four and ws may be NULL).
 *
 * The workspace of two calls that may run at the same time (two streams, two
 * captured graphs) must not be shared.
 */
size_t qlora_gated_linear_workspace(int64_t T, int64_t rows, int64_t cols, int32_t r, int is_bwd);

qlora_status qlora_gated_linear_fwd(const qlora_nf4_weight *gate, const qlora_nf4_weight *up,
                                    const uint16_t *X, int64_t T, const uint16_t *A_gate,
                                    const uint16_t *B_gate, const uint16_t *A_up,
                                    const uint16_t *B_up, int32_t r, float alpha, int act,
                                    uint16_t *H, uint16_t *P_gate, uint16_t *P_up,
                                    uint16_t *U_gate, uint16_t *U_up, void *ws, size_t ws_bytes,
                                    void *stream);

/*
 * Backward of the same, from dH [T, rows] and what the forward kept:
 *   dG = dH P_up act'(P_gate),   dU = dH act(P_gate),   s = alpha / r,
 *   dX [T, cols] = dG dequant(W_gate) + dU dequant(W_up)
 *                  + s (dG B_gate) A_gate + s (dU B_up) A_up,
 *   dA = s (dG B)^T X [r, cols],   dB = s dG^T U [rows, r]   (float32),
 * the latter two of either adapter (with dU for the up projection); no
 * gradient for the frozen weights.  dX is in the compute dtype.  dG and dU
 * meet the weights rounded to 16 bits, and B and U as 16-bit terms (24 bits in
 * bf16; 22 in fp16, but no closer than 2^-36; fp16: dG or dU past 65504 gives
 * gradients that are not finite).  dG B and dU B meet A as U meets B in the
 * forward, and X in dA with 24 bits in bf16 and 22 in fp16, the power of two of 128
 * tokens that of the larger of the two.  T = 0 writes zeros to the four adapter
 * gradients (the token tensors, dX and ws may be NULL).
 */
qlora_status qlora_gated_linear_bwd(const qlora_nf4_weight *gate, const qlora_nf4_weight *up,
                                    const uint16_t *X, const uint16_t *dH, int64_t T,
                                    const uint16_t *A_gate, const uint16_t *B_gate,
                                    const uint16_t *A_up, const uint16_t *B_up, int32_t r,
                                    float alpha, int act, const uint16_t *P_gate,
                                    const uint16_t *P_up, const uint16_t *U_gate,
                                    const uint16_t *U_up, uint16_t *dX, float *dA_gate,
                                    float *dB_gate, float *dA_up, float *dB_up, void *ws,
                                    size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_GATED_H */
