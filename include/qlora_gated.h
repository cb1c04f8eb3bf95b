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

#ifdef __cplusplus
}
#endif

#endif /* QLORA_GATED_H */
