// Host-side shapes, plan and workspace of the expert-grouped linear layer.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "abi_internal.h"

namespace qlora {

constexpr int32_t kMaxExperts = 1024;
constexpr int64_t kGroupSmallWeights = int64_t(1) << 26;   // of all experts (see grouped_ws_layout)

struct GroupArgs {
  const int32_t* offsets;   // [experts + 1], device
  int32_t experts;
  int64_t T;                // rows of X
};

// Rows [start, end) of a group whose offsets are s and t: taken into 0 .. T,
// an end before its start counts as empty.
constexpr int group_start(int s, int T) { return s < 0 ? 0 : (s > T ? T : s); }
constexpr int group_end(int s, int t, int T) {
  return t < group_start(s, T) ? group_start(s, T) : (t > T ? T : t);
}

// Largest number of tiles of H rows that T rows in `experts` groups can make:
// each group wastes at most one partial tile.
inline int64_t group_tile_bound(int64_t T, int32_t experts, int64_t H) {
  const int64_t b = T / H + (T < experts ? T : experts);
  return b < T ? b : T;
}

// The fp16 terms of G are scaled by 128-row tile (term_scale).  Slot of the
// tile of expert e that starts at row row0: later tiles have later slots, as
// the next tile of an expert starts 128 rows on and the next expert's adds one.
constexpr int term_slot(int e, int row0) { return row0 / 128 + e; }
constexpr int64_t term_slots(int64_t T, int32_t experts) { return T / 128 + experts; }
struct TermScale {
  float* largest;   // [projection splits][slots]: largest finite partial in size
  float* down;      // [slots]: what the terms' products are multiplied by
  int64_t slots;
};

// Tiles the chip holds at a time: one of 256 x 256 (MI = 4) a CU, two of
// 128 x 128 (MI = 2).
constexpr int group_slots(int MI) { return MI == 4 ? kGemmCUs : 2 * kGemmCUs; }

// Work units of the tiled GEMM: `tiles` tiles on `slots` places.  The tiles of
// the last round (all of them where there are fewer than slots) are split into
// `parts` parts of the reduction, as many as fit the round, at most 8 and at
// least 4 of its 64-wide steps long.  The float32 tiles of the parts, at most
// `slots` of them, take at most kGroupPartBytes.  8 experts of 4096 x 11008,
// 8192 rows, the backward's 576 tiles of 172 steps: 850 us in 3 rounds without
// the split, 750 us with it.
struct GroupSplit {
  int full;     // whole tiles, units 0 .. full - 1
  int parts;    // of each later tile
  int units;    // all units
};
constexpr int kGroupMaxParts = 8;
constexpr GroupSplit group_split(int tiles, int steps, int slots) {
  const int rem = tiles % slots;
  int parts = rem > 0 ? slots / rem : 1;
  parts = parts > kGroupMaxParts ? kGroupMaxParts : parts;
  parts = parts > steps / 4 ? steps / 4 : parts;
  parts = parts < 1 ? 1 : parts;
  return GroupSplit{tiles - rem, parts, tiles - rem + rem * parts};
}
constexpr size_t kGroupPartBytes = size_t(kGemmCUs) * 65536 * sizeof(float);
constexpr int kGroupCounters = 2 * kGemmCUs;   // arrival counters, one a split tile

// How a grouped forward or backward runs and where its workspace lies.
struct GroupedWs {
  int mi;            // tiled GEMM: 4 (256 x 256 tiles) or 2 (128 x 128)
  int skinny;        // forward: rows per tile of the streaming kernels, 0: the tiled GEMM
  int s_gemv;        // splits of the streaming kernels
  int s_proj;        // splits of U = X A^T or G = dY B
  int s_grad;        // splits of dA and dB over an expert's rows
  size_t proj_off, terms_off, grad_a_off, grad_b_off, gemv_off, gemv_u_off;
  size_t part_off, cnt_off;   // the GEMM's split: float32 parts and arrival counters
  size_t largest_off, down_off;   // fp16 backward: scale of G's terms (TermScale)
  size_t total;
};
// d: the expert's dimensions (rows = rows of one expert).
GroupedWs grouped_ws_layout(int64_t T, int32_t experts, const WeightDims& d, int32_t r, bool bwd);

// s U and G meet B and A as two 16-bit terms each (16 bits in bf16, 22 in fp16).
constexpr int kSeedTerms = 2;
// 16-bit terms that G = dY B is split into for dA (their sum has 24 bits in
// bf16, 22 in fp16); the first kSeedTerms of them are dX's.
inline int grad_terms(bool f16) { return f16 ? 2 : 3; }

}  // namespace qlora
