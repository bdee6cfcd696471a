// Internal kernel interface of the training operators: attention with capped, biased and
// masked scores, layer norm and AdamW (not part of the C ABI).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace detattn {

// ---- layer norm ----
struct NormArgs {
  const void* x;         // [rows, cols], row stride xs (elements), columns contiguous
  const void* dy;        // backward: [rows, cols], row stride dys
  void* y;               // forward: y; backward: dx; row stride ys
  const void* w;         // [cols] or null (ones)
  const void* b;         // [cols] or null (zeros); forward only
  float* mean;           // [rows]; forward: with rstd, or null
  float* rstd;           // [rows]
  void* dw;              // [cols] or null; the type of w
  void* db;              // [cols] or null
  float* part;           // backward workspace: [2][nparts][cols] partial sums of dw and db
  int64_t rows, cols, xs, dys, ys;
  int dtype, wdtype;     // DA_F32, DA_BF16, DA_F16
  float eps;
};
// Row groups whose dw / db partial sums are formed apart: a function of the sizes alone, so the
// order of the sums, and with it every bit of dw and db, does not depend on the GPU.
int64_t norm_parts(int64_t rows, int64_t cols);
cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t st);

// ---- AdamW ----
constexpr int ADAMW_BLOCK = 256;       // elements of an 8-bit state under one scale
constexpr int ADAMW_CHUNK = 2048;      // elements of one CTA
constexpr int ADAMW_TABLE = 120;       // tensors of one launch
struct AdamWTensor {
  void* p;
  const void* g;
  int64_t n;
  int64_t state;                       // first element of its states
};
struct AdamWArgs {
  AdamWTensor t[ADAMW_TABLE];
  uint32_t first[ADAMW_TABLE + 1];     // chunks before each tensor of this launch
  int nt;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  const float* grad_scale;             // optional device scalar
  float b1, c1, b2, c2, keep, rate, undo, eps;
};
cudaError_t launch_adamw(const AdamWArgs& a, int dtype, int bits, cudaStream_t st);

}  // namespace detattn
