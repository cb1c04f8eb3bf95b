// Row groups of the expert-grouped layer on the host: whatever the offsets
// hold, every group's rows lie in 0 .. T, and for offsets that do not
// decrease the tiles never exceed the bound that sizes the grids.
#include <stdio.h>
#include <stdlib.h>

#include "grouped.h"

int main() {
  srand(1);
  for (int rep = 0; rep < 200000; ++rep) {
    const int T = rand() % 700, E = 1 + rand() % 40;
    const bool sorted = rep & 1;
    int off[41];
    int at = rand() % 5;
    for (int e = 0; e <= E; ++e) {
      if (sorted) {
        off[e] = at < T ? at : T;
        at += rand() % 3 ? rand() % 60 : 0;
      } else {
        off[e] = rand() % 4 ? rand() % (T + 1) : rand() - (1 << 30);
      }
    }
    const int H[4] = {16, 64, 128, 256};
    for (int h : H) {
      long tiles = 0;
      for (int e = 0; e < E; ++e) {
        const int s = qlora::group_start(off[e], T), t = qlora::group_end(off[e], off[e + 1], T);
        if (s < 0 || s > t || t > T) return printf("range %d %d of %d\n", s, t, T), 1;
        if (sorted && (s != off[e] || t != off[e + 1])) return printf("changed\n"), 1;
        tiles += (t - s + h - 1) / h;
      }
      if (sorted && tiles > qlora::group_tile_bound(T, E, h))
        return printf("tiles %ld over %ld\n", tiles, (long)qlora::group_tile_bound(T, E, h)), 1;
    }
  }
  puts("ok");
  return 0;
}
