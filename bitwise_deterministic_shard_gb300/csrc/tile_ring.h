// Where the training attention's forward pass keeps its key and value tiles: a ring of `nst` stages, each with a full and an
// empty barrier whose phases are its fills.  The tile at place k takes fill k / nst of stage k % nst.
//
// A wait for a phase by its parity is met by the phase two before it too.  So who waits for a fill of a stage must know that
// the fill before it was complete: each group of softmax warps and its products may only wait for stages whose fill
// before was a tile that the group has taken.
//   Both groups take every tile (SPLIT false): places in the order of the copies, K0 K1 V0 K2 V1 K3 ...  A group
//   that takes a tile has taken every one before it that the ring could have replaced.
//   Each group takes every other tile (SPLIT true): in that order a value tile could follow a key tile of the
//   other group, perhaps still on its way (the second group then went ahead on the parity of the fill before and released
//   a stage that was being filled, whose barrier got an arrival too many: a launch failure).  So the places are K0 V0
//   K1 V1 ..., and with nst a multiple of 4 a stage's tiles are all of one kind and one group.
#pragma once

#if defined(__CUDACC__)
#define DA_RING_FN __host__ __device__ __forceinline__
#else
#define DA_RING_FN inline
#endif

namespace detattn {

template <bool SPLIT>
DA_RING_FN int key_place(int n) {
  return SPLIT ? 2 * n : n < 2 ? n : 2 * n - 1;
}
template <bool SPLIT>
DA_RING_FN int value_place(int n, int tiles) {
  const int keys = n + (SPLIT ? 1 : 2);   // before it
  return (tiles < keys ? tiles : keys) + n;
}
// whether no later tile takes its stage
DA_RING_FN bool last_place(int k, int tiles, int nst) { return k + nst >= 2 * tiles; }

}  // namespace detattn
