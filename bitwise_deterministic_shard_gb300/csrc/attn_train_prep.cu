// Document ids of each tile of 128 keys (and of 128 queries): their range and whether any is negative, from which the
// attention kernels find the tiles that can see each other.
#include "attn_train.h"

namespace detattn {
namespace {

__global__ void __launch_bounds__(128) ta_bounds_kernel(const int* docs, int Skv, int Sq, TaBounds* keys, TaBounds* queries) {
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;   // one warp a tile
  const int S = blockIdx.z ? Sq : Skv, tiles = (S + TA_TILE - 1) / TA_TILE;
  if (w >= tiles) return;
  const int* d = docs + (int64_t)blockIdx.y * Skv + (Skv - S);
  int lo = 0x7fffffff, hi = -1, neg = 0;
#pragma unroll
  for (int i = 0; i < TA_TILE; i += 32) {
    const int j = w * TA_TILE + i + lane, x = j < S ? d[j] : -1;
    neg |= x < 0;
    lo = min(lo, x < 0 ? 0x7fffffff : x);
    hi = max(hi, x);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  neg = __any_sync(0xffffffffu, neg);
  if (lane == 0) (blockIdx.z ? queries : keys)[(int64_t)blockIdx.y * tiles + w] = TaBounds{lo, max(hi, -1), neg};
}

}  // namespace

cudaError_t ta_bounds(const int* docs, int B, int Skv, int Sq, TaBounds* keys, TaBounds* queries, cudaStream_t st) {
  const int tiles = (Skv + TA_TILE - 1) / TA_TILE;
  if (B == 0 || tiles == 0) return cudaSuccess;
  ta_bounds_kernel<<<dim3((tiles + 3) / 4, B, queries ? 2 : 1), 128, 0, st>>>(docs, Skv, Sq, keys, queries);
  return cudaGetLastError();
}

}  // namespace detattn
