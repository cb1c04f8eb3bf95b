// Prints how the 8-bit and the expert-grouped entry points run given sizes:
// one line for each line read from the standard input.
//   int8 T rows cols given             ->  path splits
//   group rows cols r dq f16 bwd T count count ...
//       ->  skinny mi s_gemv s_proj s_grad parts   (parts of a split tile, 1: none split)
#include <stdio.h>
#include <string.h>

#include <sstream>
#include <string>

#include "grouped.h"
#include "int8.h"

int main() {
  char buf[1 << 16];
  while (fgets(buf, sizeof(buf), stdin)) {
    std::istringstream in(buf);
    std::string what;
    in >> what;
    if (what == "int8") {
      long long T, rows, cols;
      int given;
      in >> T >> rows >> cols >> given;
      const qlora::Int8Plan p = qlora::int8_plan(T, rows, cols, !given);
      printf("%d %d\n", (int)p.path, p.splits);
    } else {
      long long rows, cols, T, c;
      int r, dq, f16, bwd;
      in >> rows >> cols >> r >> dq >> f16 >> bwd >> T;
      std::string counts;
      int experts = 0;
      std::getline(in, counts);
      std::istringstream all(counts);
      qlora::WeightDims d;
      memset(&d, 0, sizeof(d));
      d.rows = rows;
      d.cols = cols;
      d.dq = dq != 0;
      d.f16 = f16 != 0;
      while (all >> c) ++experts;
      const qlora::GroupedWs L = qlora::grouped_ws_layout(T, experts, d, r, bwd != 0);
      long tiles = 0;
      std::istringstream again(counts);
      const int side = 64 * L.mi;
      while (again >> c) tiles += (c + side - 1) / side;
      const long long out = bwd ? cols : rows, red = bwd ? rows : cols;
      const qlora::GroupSplit s = qlora::group_split((int)(tiles * ((out + side - 1) / side)),
                                                     (int)((red + 63) / 64), qlora::group_slots(L.mi));
      printf("%d %d %d %d %d %d\n", L.skinny, L.mi, L.s_gemv, L.s_proj, L.s_grad, s.parts);
    }
  }
  return 0;
}
