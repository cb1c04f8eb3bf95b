// Byte offsets of the tiled GEMMs' loads, which run up to two steps ahead of the
// reduction and so past its end.  A load's address is the 32-bit sum of a scalar
// offset (the step, the rows) and a lane's, and it reads 0 where that sum lies past
// the descriptor's range: one of the two may be out of range, not both, as 2 * 2^31
// is 0.
#pragma once

#include <stdint.h>

namespace qlora {

constexpr uint32_t kOOB = 0x80000000u;   // past every range (tensors stay below 2 GiB)
// A lane's offset into packed codes, of at most 2^30 bytes, where its row or column
// lies past the weight: with kOOB as the step's offset the sum does not wrap.
constexpr uint32_t kOOBCodes = 0x40000000u;

// Scalar offset of step `step` of a part of nsteps.
constexpr uint32_t step_soff(int step, int nsteps, uint32_t bytes) {
  return step < nsteps ? bytes : kOOB;
}

// The step of a part (first: its first step) in which lanes past the end of the
// reduction take kOOB: the reduction's last, or -1 where that is not the part's.  (A
// part that ends a step or two before it also loads it, as a step past its own end,
// which step_soff puts out of range.)
constexpr int tail_step(int last, int first, int nsteps) {
  return last >= first && last - first < nsteps ? last - first : -1;
}

}  // namespace qlora
