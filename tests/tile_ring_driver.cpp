// Prints csrc/tile_ring.h's places: "split nst tiles value n stage fill last" a line.
#include <cstdio>

#include "tile_ring.h"

using namespace detattn;

int main() {
  const int rings[2][2] = {{3, 7}, {4, 8}};   // the kernels' rings
  for (int split = 0; split < 2; split++)
    for (int nst : rings[split])
      for (int tiles = 1; tiles <= 40; tiles++)
        for (int n = 0; n < tiles; n++) {
          const int k = split ? key_place<true>(n) : key_place<false>(n);
          const int v = split ? value_place<true>(n, tiles) : value_place<false>(n, tiles);
          std::printf("%d %d %d 0 %d %d %d %d\n", split, nst, tiles, n, k % nst, k / nst, (int)last_place(k, tiles, nst));
          std::printf("%d %d %d 1 %d %d %d %d\n", split, nst, tiles, n, v % nst, v / nst, (int)last_place(v, tiles, nst));
        }
}
