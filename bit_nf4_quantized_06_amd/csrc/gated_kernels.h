// Launchers of the gated feed-forward block over NF4 weights (gemm.hip,
// gemv.hip, lora.hip, gated.hip).  [0] is the gate, [1] the up projection.
#pragma once

#include "grouped.h"
#include "kernels.h"

namespace qlora {

// Work units of the gated GEMM that decodes its weights in LDS: tiles of 64 MI
// tokens by 64 MI outputs (forward: outputs of both projections), the last
// round's in parts of the reduction.
inline GroupSplit gated_split(int64_t T, int64_t rows, int64_t cols, bool bwd, int MI) {
  const int64_t side = 64 * MI, out = bwd ? cols : 2 * rows;
  const int64_t steps = bwd ? 2 * ((rows + 63) / 64) : (cols + 63) / 64;
  return group_split((int)(((T + side - 1) / side) * ((out + side - 1) / side)), (int)steps,
                     group_slots(MI));
}

// How a gated forward or backward runs and where its workspace lies; offsets
// of pairs: [0] the gate, [1] the up projection.
struct GatedWs {
  int s_gemv;        // splits of the streaming forward, 0: the tiled GEMM
  int s_proj;        // splits of U_i = X A_i^T or d_i B_i
  int s_grad;        // splits of the adapters' gradients over the tokens
  int mi;            // tiled GEMM: 4 (256 x 256 tiles) or 2 (128 x 128)
  int gemm_split;    // once-dequantised weights: first split tile
  int n_split;       // split tiles
  bool pre_dq;
  size_t proj_off[2], gemv_off[2], gemv_u_off[2], wdq_off[2];
  size_t largest_off[2], down_off[2];   // scale of the terms (TermScale)
  size_t at_off[2], d_off[2], terms_off[2], grad_a_off[2], grad_b_off[2];
  size_t split_part_off, split_cnt_off;
  size_t total;
};
// d: the dimensions of either weight.
GatedWs gated_ws_layout(int64_t T, const WeightDims& d, int32_t r, bool bwd);

// What the up projection of a gated GEMM has of its own (the gate's are in
// GemmArgs; shapes, r and formats are shared).
struct GateArgs {
  const uint8_t* codes;
  const uint8_t* code8;
  const float* s2;
  const float* mu;
  const uint16_t* wdq;
  const uint16_t* act;      // backward: dU [T, rows] (GemmArgs::act: dG)
  const uint16_t* lora_l;   // planes [kSeedTerms][T][r], as GemmArgs::lora_l here
  const uint16_t* lora_r;   // forward B_up [rows, r], backward A_up^T [cols, r]
  float scale;              // of the adapters' products
  const float* down[2];     // f16: by 128-row tile, what they are multiplied by too (TermScale;
                            // backward: [0] of both)
  uint16_t* p_gate;         // forward: both projections [T, rows] or NULL
  uint16_t* p_up;
  int act_fn;               // forward: QLORA_ACT_*
};
// H [T, rows] (GemmArgs::out).  wdq given: 256-row tiles, split_from counts tiles
// of 128 outputs; else MI 4 or 2, tiles of 64 MI, split as gated_split says (part:
// a float32 tile for each part, cnt: a zeroed counter for each split tile).
hipError_t launch_gated_fwd_gemm(const GemmArgs& a, const GateArgs& gate, int MI,
                                 hipStream_t stream);
// dX [T, cols], one reduction over the rows of both weights.
hipError_t launch_gated_dx_gemm(const GemmArgs& a, const GateArgs& gate, int MI,
                                hipStream_t stream);

// Split partials of U_i = X A_i^T, as launch_lora_proj_partial, of both; with f16
// also the largest of each (TermScale::largest, [splits][slots][4], a number for
// each 32 rows).
hipError_t launch_gated_proj(const uint16_t* X, const uint16_t* const A[2], int64_t T, int64_t red,
                             int32_t r, int splits, float* const P[2], const TermScale (&ts)[2],
                             bool f16, hipStream_t stream);

constexpr int64_t gated_slots(int64_t T) { return (T + 127) / 128; }

// launch_lora_proj_reduce of both projections in one launch.  terms: planes
// [n_terms][T][r] of 16-bit numbers whose sum is v (f16: times its tile's
// term_scale, whose inverse goes into ts.down; common: one for both).
struct GatedReduce {
  ProjReduce part[2];
  TransposeJobs tj[2];
  uint16_t* terms[2];
  int n_terms;
  TermScale ts[2];         // f16
  bool common;
};
hipError_t launch_gated_reduce(const GatedReduce& a, hipStream_t stream);

// Few tokens: launch_qlora_gemv's first kernel for both weights.
hipError_t launch_gated_gemv_partial(const GemvArgs& gate, const GemvArgs& up, hipStream_t stream);
// U_i = sum_s PU_i (stored in 16 bits when U_save is given), P_i = sum_s P_i +
// scale U_i B_i^T in float32, H = act(P_gate) P_up, and both P in 16 bits.
struct GatedFinish {
  const float* P[2];       // [splits][T][rows]
  const float* PU[2];      // [splits][T][r]
  const uint16_t* B[2];    // [rows, r]
  uint16_t* U_save[2];     // [T, r] or NULL
  uint16_t* P_save[2];     // [T, rows] or NULL
  uint16_t* H;             // [T, rows]
  int64_t T, rows;
  int32_t r;
  int splits;
  float scale;
  int act_fn;
  bool f16;
};
hipError_t launch_gated_finish(const GatedFinish& a, hipStream_t stream);

// dG = dH P_up act'(P_gate), dU = dH act(P_gate): both in 16 bits, and the split
// partials of dG B_gate and dU B_up from their values in terms.
struct GatedBwd {
  const uint16_t* dH;      // [T, rows]
  const uint16_t* Pg;
  const uint16_t* Pu;
  const uint16_t* B[2];    // [rows, r]
  uint16_t* d[2];          // dG, dU [T, rows]
  float* P[2];             // [splits][T][r]
  TermScale ts[2];         // f16: `largest` is written, as by launch_gated_proj
  int64_t T, rows;
  int32_t r;
  int splits;
  int act_fn;
  bool f16;
};
int gated_bwd_splits(int64_t T, int64_t rows);
hipError_t launch_gated_bwd(const GatedBwd& a, hipStream_t stream);

// Split partials of dB_i = d_i^T U_i with d formed again from dH and both
// projections, and of dA_i = (d_i B_i)^T X with d_i B_i given in terms.
struct GatedGrads {
  const uint16_t* dH;
  const uint16_t* Pg;
  const uint16_t* Pu;
  const uint16_t* X;
  const uint16_t* U[2];      // [T, r]
  const uint16_t* terms[2];  // planes [grad_terms][T][r] (GatedReduce)
  const float* down[2];      // f16: by 128-row tile, what the terms' products are multiplied by
  float* part_a[2];          // [splits][r][cols]
  float* part_b[2];          // [splits][rows][r]
  int64_t T, rows, cols;
  int32_t r;
  int splits;
  int act_fn;
  bool f16;
};
int gated_grad_splits(int64_t T, int64_t rows, int64_t cols, int32_t r);
hipError_t launch_gated_grads(const GatedGrads& a, hipStream_t stream);

// out = scale sum_s part for four gradients of n float32 each, in one launch.
struct GatedSum {
  const float* part[4];
  float* out[4];
  int64_t n[4];
  int splits;
  float scale;
};
hipError_t launch_gated_sum(const GatedSum& a, hipStream_t stream);

}  // namespace qlora
