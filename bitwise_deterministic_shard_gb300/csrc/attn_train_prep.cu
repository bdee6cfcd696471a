// Small passes before the attention kernels.
//
// Document ids of each tile of 128 keys: their range and whether any is negative, from which the
// attention kernels find the key tiles that a tile of queries can see.
#include "attn_train.h"
#include "train_math.cuh"

namespace detattn {
namespace {

__global__ void __launch_bounds__(128) ta_bounds_kernel(const int* docs, int Skv, int S, int tiles, TaBounds* out) {
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;   // one warp a tile
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
  if (lane == 0) out[(int64_t)blockIdx.y * tiles + w] = TaBounds{lo, max(hi, -1), neg};
}

// What the backward passes take of a query row: minus its lse in log2 units and minus delta = sum out * grad.
// Eight threads a row, 16-byte loads; bound by reading out and grad once.
template <typename T>
__global__ void __launch_bounds__(256) ta_rows_kernel(const TaRowsArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);   // of [B, Hq, qtiles * 128]
  const int per = a.qtiles * TA_TILE, u = threadIdx.x & 7;
  const int64_t bh = row / per;
  const int i = (int)(row % per), b = (int)(bh / a.Hq), h = (int)(bh % a.Hq);
  if (bh >= (int64_t)a.B * a.Hq) return;   // 32 rows divide a tile: whole warps
  float s = 0.f;
  if (i < a.Sq) {
    const T* o = (const T*)a.out + b * a.os[0] + h * a.os[1] + i * a.os[2];
    const T* g = (const T*)a.grad + b * a.gs[0] + h * a.gs[1] + i * a.gs[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int d = (u + 8 * k) * 8;
      if (d < a.D) {
        Run<T, 8> x, y;
        x.load(o + d);
        y.load(g + d);
#pragma unroll
        for (int e = 0; e < 8; e++) s = __fmaf_rn(x.get(e), y.get(e), s);
      }
    }
  }
#pragma unroll
  for (int m = 4; m; m >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, m));
  if (u == 0) {
    const float l = i < a.Sq ? a.lse[bh * a.Sq + i] : -INFINITY;
    const bool none = l == -INFINITY;
    float* const at = a.rows + (row / TA_TILE) * 256 + row % TA_TILE;
    at[0] = none ? -INFINITY : -l * 1.4426950408889634f;
    at[128] = none ? 0.f : -s;
  }
}

}  // namespace

cudaError_t ta_rows(const TaRowsArgs& a, cudaStream_t st) {
  const int64_t n = (int64_t)a.B * a.Hq * a.qtiles * TA_TILE;
  if (n == 0) return cudaSuccess;
  const unsigned grid = (unsigned)(n / 32);
  if (a.bf) ta_rows_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  else ta_rows_kernel<__half><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t ta_bounds(const int* docs, int B, int Skv, int S, TaBounds* out, cudaStream_t st) {
  const int tiles = (S + TA_TILE - 1) / TA_TILE;
  if (B == 0 || tiles == 0) return cudaSuccess;
  ta_bounds_kernel<<<dim3((tiles + 3) / 4, B), 128, 0, st>>>(docs, Skv, S, tiles, out);
  return cudaGetLastError();
}

}  // namespace detattn
