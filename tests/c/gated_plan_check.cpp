// Prints how the 8-bit floating point and the gated entry points run given
// sizes: one line for each line read from the standard input.
//   fp8 T outs cols x16            ->  path splits
//   gated T rows cols r bwd        ->  s_gemv mi pre_dq split parts s_proj s_grad
//       (split: split tiles; parts: parts of each)
#include <stdio.h>
#include <string.h>

#include <sstream>
#include <string>

#include "fp8.h"
#include "gated_kernels.h"

int main() {
  char buf[256];
  while (fgets(buf, sizeof(buf), stdin)) {
    std::istringstream in(buf);
    std::string what;
    long long T, rows, cols;
    in >> what >> T >> rows >> cols;
    if (what == "fp8") {
      int x16;
      in >> x16;
      const qlora::Fp8Plan p = qlora::fp8_plan(T, rows, cols, x16 != 0);
      printf("%d %d\n", (int)p.path, p.splits);
    } else {
      int r, bwd;
      in >> r >> bwd;
      qlora::WeightDims d;
      memset(&d, 0, sizeof(d));
      d.rows = rows;
      d.cols = cols;
      d.n = rows * cols;
      const qlora::GatedWs L = qlora::gated_ws_layout(T, d, r, bwd != 0);
      int parts = L.n_split > 0 ? 2 : 1;
      if (!L.pre_dq && !L.s_gemv) parts = qlora::gated_split(T, rows, cols, bwd != 0, L.mi).parts;
      printf("%d %d %d %d %d %d %d\n", L.s_gemv, L.mi, (int)L.pre_dq, L.n_split, parts, L.s_proj,
             L.s_grad);
    }
  }
  return 0;
}
