// Row groups of the expert-grouped linear layer: which rows belong to which
// expert is known on the device only (offsets [experts + 1]), so every
// workgroup finds its own tile of rows from its index.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grouped.h"

namespace qlora {

// Expert e's rows [start, end): whatever the offsets hold, every row named
// here lies inside the tensors (group_start, group_end).
__device__ __forceinline__ void group_range(const GroupArgs& a, int e, int& start, int& end) {
  const int T = (int)a.T;
  const int s = a.offsets[e], t = a.offsets[e + 1];
  start = group_start(s, T);
  end = group_end(s, t, T);
}

// Inclusive sum over the lanes of a full wave by DPP: shifts by 1, 2, 4 and 8
// within each row of 16, then the row totals handed on (row_bcast:15 to rows
// 1 and 3, row_bcast:31 to rows 2 and 3).
__device__ __forceinline__ int wave_inclusive_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// Tiles of H rows of this lane's expert (base + lane), 0 past the last.
template <int H>
__device__ __forceinline__ int group_lane_tiles(const GroupArgs& a, int base, int lane, int& start,
                                                int& end) {
  start = end = 0;
  const int e = base + lane;
  if (e < a.experts) group_range(a, e, start, end);
  return (end - start + H - 1) / H;
}

// Number of tiles of H rows over all experts (every lane of a full wave
// calls it; the result is uniform).
template <int H>
__device__ __forceinline__ int group_tiles(const GroupArgs& a) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int base = 0; base < a.experts; base += 64) {
    int s, t;
    const int inc = wave_inclusive_scan(group_lane_tiles<H>(a, base, lane, s, t));
    total += __builtin_amdgcn_readlane(inc, 63);
  }
  return total;
}

// Expert of row t, which lies in some expert's range (for offsets that
// decrease: some expert).  offsets: of `experts` experts, in LDS.
__device__ __forceinline__ int group_of_row(const int* offsets, int experts, int t) {
  int lo = 0, hi = experts - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The power of two that the G of a 128-row tile is multiplied by before it is
// split into fp16 terms, and its inverse.  `largest`: the tile's largest
// finite partial sum of G in size, of `splits` of them; so |G| is at most
// splits times that, and the product lies below 2^15.  A term below fp16's
// normal range is then off by at most 2^-39 of that bound's power of two.
// (Sums of fp16 products lie between 2^-48 and 2^52, inside the clamps.)
__device__ __forceinline__ void term_scale(float largest, int splits, float& up, float& down) {
  int ex = (int)(__float_as_uint(largest) >> 23) +
           (splits > 1 ? 32 - __builtin_clz(splits - 1) : 0);
  ex = ex < 64 ? 64 : (ex > 190 ? 190 : ex);
  up = __uint_as_float((uint32_t)(268 - ex) << 23);
  down = __uint_as_float((uint32_t)(ex - 14) << 23);
}

// The larger of m and |v|, unless v is not finite.
__device__ __forceinline__ float larger_finite(float m, float v) {
  v = fabsf(v);
  return v > m && v < __builtin_inff() ? v : m;   // not for NaN
}

struct GroupTile {
  int expert;    // -1: the index is past the last tile
  int row0;      // first row of the tile
  int rows;      // rows in it, 1 .. H
};

// Tile `want` in expert order (uniform).
template <int H>
__device__ __forceinline__ GroupTile group_tile(const GroupArgs& a, int want) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < a.experts; base += 64) {
    int s, t;
    const int mine = group_lane_tiles<H>(a, base, lane, s, t);
    const int inc = wave_inclusive_scan(mine);
    const int total = __builtin_amdgcn_readlane(inc, 63);
    if (want < before + total) {
      // first lane whose inclusive count passes the index
      const uint64_t past = __ballot(before + inc > want);
      const int l = __builtin_ctzll(past);
      const int start = __builtin_amdgcn_readlane(s, l);
      const int end = __builtin_amdgcn_readlane(t, l);
      const int first = before + __builtin_amdgcn_readlane(inc - mine, l);
      GroupTile g;
      g.expert = base + l;
      g.row0 = start + (want - first) * H;
      g.rows = end - g.row0 < H ? end - g.row0 : H;
      return g;
    }
    before += total;
  }
  return GroupTile{-1, 0, 0};
}

}  // namespace qlora
