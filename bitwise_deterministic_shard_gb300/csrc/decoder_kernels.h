// Internal kernel interface of the operators at the ends and in the middle of a decoder: embedding
// lookup, gated feed-forward projections, log probabilities (not part of the C ABI).
#pragma once
#include <cuda.h>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace detattn {

// ---- gated feed-forward ----
constexpr int GL_FEW = 8;        // tokens up to which the weights are read once by plain loads

struct GlArgs {
  CUtensorMap a[2], b[2];        // operands of the pair products (see gated_kernels.cuh)
  void* out[2];                  // forward: h; dx; or dWg and dWu
  int64_t os[2];                 // their row strides
  unsigned char* saved;          // forward: factors of the backward pass, or null
  int T, D, F;                   // tokens, width, hidden units
  int activation;
  int* status;
};
struct GlFewArgs {
  const void* x;
  const void* wg;
  const void* wu;
  void* h;
  int64_t xs, gs, us, hs;
  int T, D, F, activation;
};
struct GlScaleArgs {             // dg = dh p, du = dh q
  const void* dh;
  int64_t ds;
  const unsigned char* saved;
  void* dg;                      // [T, F], du behind it
  int64_t T, F;
};
// The saved factors p and q of [T, F]: the high 16 bits of each binary32 value (p's plane, q's plane), then the next 8.
inline size_t gl_saved_bytes(int64_t T, int64_t F) { return (size_t)6 * T * F; }

template <bool BF>
cudaError_t gl_forward(const GlArgs& a, cudaStream_t st);
template <bool BF>
cudaError_t gl_dx(const GlArgs& a, cudaStream_t st);
template <bool BF>
cudaError_t gl_dw(const GlArgs& a, cudaStream_t st);
template <bool BF>
cudaError_t gl_few(const GlFewArgs& a, cudaStream_t st);
template <bool BF>
cudaError_t gl_scale(const GlScaleArgs& a, cudaStream_t st);

}  // namespace detattn
