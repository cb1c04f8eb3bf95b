// Walks the steps that the tiled GEMMs load, those past a part's end included, and
// checks where each lane's address lies: the columns of the reduction in the tensor,
// everything else past every range, without the 32-bit sum wrapping.  Prints how many
// loads it looked at; exits 1 at the first wrong one.
#include <stdint.h>
#include <stdio.h>

#include "abi_internal.h"
#include "fp8.h"
#include "gated_kernels.h"
#include "step_offsets.h"

using namespace qlora;

static long long looked = 0, past_end_tails = 0;

// One part of a reduction of `bytes` bytes in steps of 128, which ends in step
// `last`; `again`: a second operand's steps follow (its step number `last2`).
static bool part(int first, int nsteps, int last, int last2, uint32_t bytes) {
  const int tail = tail_step(last, first, nsteps);
  const int tail2 = last2 < 0 ? -1 : tail_step(last2, first, nsteps);
  for (int step = 0; step < nsteps + 2; ++step) {
    int ks = first + step;
    if (step >= nsteps && (ks == last || ks == last2)) ++past_end_tails;
    if (last2 >= 0 && ks > last) ks -= last + 1;
    for (uint32_t chunk = 0; chunk < 128; chunk += 16) {
      const bool in_row = (uint32_t)ks * 128u + chunk < bytes;
      const uint32_t lane = (step == tail || step == tail2) && !in_row ? kOOB : chunk;
      const uint32_t scalar = step_soff(step, nsteps, (uint32_t)ks * 128u);
      const uint64_t sum = (uint64_t)scalar + lane;
      const bool reads = step < nsteps && in_row;
      ++looked;
      if (sum >> 32 || (reads ? sum >= bytes : sum < kOOB)) {
        printf("first %d nsteps %d last %d step %d chunk %u: %llx\n", first, nsteps, last, step,
               chunk, (unsigned long long)sum);
        return false;
      }
    }
  }
  return true;
}

int main() {
  // the gated backward: two operands of `rows` 16-bit columns, parts as group_split
  for (int64_t T : {65, 300, 509, 1100, 2187})
    for (int64_t rows = 16; rows <= 3000; rows += 16)
      for (int mi : {2, 4}) {
        const int half = (int)((rows + 63) / 64), all = 2 * half;
        for (int64_t cols : {64, 1024, 4096}) {
          const int parts = gated_split(T, rows, cols, true, mi).parts;
          for (int p = 0; p < parts; ++p) {
            const int first = all * p / parts, end = all * (p + 1) / parts;
            if (rows % 64 != 0 &&
                !part(first, end - first, half - 1, all - 1, (uint32_t)(rows * 2)))
              return 1;
          }
        }
      }
  // 8-bit products: `cols` codes in splits of whole steps
  for (int64_t cols = 16; cols <= 6000; cols += 16)
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      const int all = (int)fp8_blocks(cols), per = (all + splits - 1) / splits;
      for (int s = 0; s < splits; ++s) {
        const int first = s * per, end = first + per < all ? first + per : all;
        if (end > first && !part(first, end - first, all - 1, -1, (uint32_t)cols)) return 1;
      }
    }
  // packed codes: the largest weight, a lane past it, and a step past the end
  const int64_t most = 2 * ((int64_t(1) << 30) - 64);
  if (!linear_dims_ok(1, most / 2048, 2048) || linear_dims_ok(1, most / 2048 + 16, 2048)) return 1;
  if ((int64_t)kOOBCodes < most / 2) return 1;
  if (((uint64_t)kOOBCodes + (uint64_t)(most / 2)) >> 32) return 1;
  if (((uint64_t)kOOBCodes + kOOB) >> 32 || (((uint64_t)most / 2 + kOOB) >> 32)) return 1;
  printf("%lld %lld\n", looked, past_end_tails);
  return 0;
}
