// Launchers of the expert-grouped linear layer's kernels (gemm.hip, gemv.hip,
// lora.hip).  The layouts are those of the dense launchers in kernels.h with
// a leading expert index on weights and adapters; g.rows is one expert's.
#pragma once

#include "grouped.h"
#include "kernels.h"

namespace qlora {

// out = act * Wop_e + lora_l lora_r_e^T for the rows of each expert e (see
// launch_qlora_fwd_gemm / launch_qlora_dx_gemm; keep, wdq and split_from are
// not used; part: kGroupPartBytes, cnt: kGroupCounters zeroed counters).
// lora_l: planes [kSeedTerms][T][r] whose sum is the operand; the backward
// multiplies the product by seed.scale, and with f16 by its tile's seed.down
// (TermScale).
// lora_r: [experts, out_len, r], in the backward [experts, r, out_len].
// MI: 4 or 2, tiles of 64 MI rows by 64 MI outputs.
struct GroupSeed {   // backward
  float scale;
  const float* down;   // f16
};
hipError_t launch_grouped_gemm(const GemmArgs& a, const GroupArgs& ga, const GroupSeed& seed,
                               bool bwd, int MI, hipStream_t stream);

// The streaming forward over tiles of H rows (16 or 32).
hipError_t launch_grouped_gemv(const GemvArgs& a, const GroupArgs& ga, int H, hipStream_t stream);

// P[s][t][p] as launch_lora_proj_partial with R_e of t's expert.  ts: with
// f16 and r_by_rows its `largest` is written, else it is empty.
hipError_t launch_grouped_proj(const uint16_t* L, const uint16_t* R, bool r_by_rows,
                               const GroupArgs& ga, int64_t red, int32_t r, int splits, float* P,
                               const TermScale& ts, bool f16, hipStream_t stream);

// v = sum_s P[s] (fixed order) for the rows some expert owns: out = 16-bit v
// (may be NULL), terms: planes [n_terms][T][r] of 16-bit numbers whose sum is
// scale v (ts given: times its tile's term_scale, whose inverse goes into ts.down).
struct GroupedReduce {
  const float* P;
  int32_t r;
  int splits;
  float scale;
  uint16_t* out;
  uint16_t* terms;
  int n_terms;
  bool f16;
  uint32_t* zero_cnt;      // kGroupCounters arrival counters of the GEMM that follows, zeroed
  TermScale ts;            // with fp16 terms, as launch_grouped_proj left it; else empty
};
hipError_t launch_grouped_reduce(const GroupedReduce& a, const GroupArgs& ga, hipStream_t stream);

// dA [experts, r, cols] = scale G_e^T X_e with G given in n_terms planes (in
// fp16 scaled by tile, see TermScale), and
// dB [experts, rows, r] = scale dY_e^T U_e; experts without rows get zeros.
// splits > 1: partials in Pa, Pb ([splits] copies of dA, dB), then summed.
struct GroupedGrads {
  const uint16_t* G;
  int n_terms;
  const uint16_t* X;
  const uint16_t* U;
  const uint16_t* dY;
  int64_t rows, cols;
  int32_t r;
  float scale;
  float* dA;
  float* dB;
  float* Pa;
  float* Pb;
  int splits;
  const float* down;       // fp16: what the terms' products are multiplied by (TermScale)
  bool f16;
};
hipError_t launch_grouped_grads(const GroupedGrads& a, const GroupArgs& ga, hipStream_t stream);

}  // namespace qlora
