// Internal interface of the training attention (capped, distance-biased and masked scores):
// forward, its join of key ranges, and the backward passes.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace detattn {

constexpr int TA_TILE = 128;          // queries, and keys, of a tile

// smallest and largest document id of a 128-key tile (negative ids left out) and whether it has
// negative ones (or ends past the last key)
struct TaBounds {
  int lo, hi, neg;
};

// f tanh(k t) of a product t, in log2 units: f = softcap log2 e, k = scale / softcap.  Odd polynomials f k t P((k t)^2) with k
// and f folded into the coefficients, each twice for the packed arithmetic: c up to |t| = most, s up to least.  far: a cap of more
// than 4096 times the scale, s tanh's series.
struct TaCap {
  unsigned long long c[6], s[4];
  float k, f, most, least;
  int far;
};

struct TaArgs {
  // rank-5 maps {D, heads of the box's group, S, groups, B}, boxes of 64 columns
  CUtensorMap q, k, v, o, go, dq, dk, dv;
  const float* slopes;                // [Hq] or null
  const int* docs;                    // [B, Skv] or null
  const TaBounds* bounds;             // [B, key tiles] with docs
  const TaBounds* qbounds;            // backward: [B, query tiles] with docs
  const int* prefix;                  // [B] or null
  float* lse;                         // [B, Hq, Sq], natural logarithm
  float* rows;                        // backward, from the dq kernel to the other: [B, Hq, query tiles][2][128]
                                      // (-lse log2 e), (-delta); -inf, 0 for a row that sees nothing and past the last query
  float* part;                        // split forward: sums [2 splits][B Hkv][128][DP], then (max, total, total of the rounded weights, 0)
  void* out;                          // join of the split forward; strides of b, h, s
  int64_t os[3];
  int* status;
  int B, Hq, Hkv, Sq, Skv, D;
  int group;                          // query heads of a key head
  int pack;                           // query heads in one tile: group when Sq * group <= 128, else 1
  int qrows;                          // queries of a tile
  int qtiles;                         // query tiles (of a head, or of a group of heads when packed)
  int ktiles;
  int causal;
  int splits;                         // > 0: key ranges, each CTA's two softmax groups on every other tile
  float scale;                        // of the products
  float softcap;
  TaCap cap;
};

template <int DP, bool BF>
cudaError_t ta_forward(const TaArgs& a, cudaStream_t st);
template <int DP, bool BF>
cudaError_t ta_dkv(const TaArgs& a, cudaStream_t st);
template <int DP, bool BF>
cudaError_t ta_dq(const TaArgs& a, cudaStream_t st);
// bounds of the key tiles and, unless null, of the tiles of the last Sq tokens (the queries)
cudaError_t ta_bounds(const int* docs, int B, int Skv, int Sq, TaBounds* keys, TaBounds* queries, cudaStream_t st);

}  // namespace detattn
