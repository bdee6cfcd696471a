// Internal kernel interface of the operators at the ends and in the middle of a decoder: embedding
// lookup, gated feed-forward projections, log probabilities (not part of the C ABI).
#pragma once
#include <cuda.h>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace detattn {

// ---- gated feed-forward ----
constexpr int GL_FEW = 16;       // tokens up to which the weights are read once by plain loads

struct GlArgs {
  CUtensorMap x, wg, wu;         // boxes of 64 x 64
  CUtensorMap dg, du;            // backward
  void* h;                       // forward
  void* dx;                      // backward; either may be null
  void* dwg;
  void* dwu;
  int64_t hs, dxs, dwgs, dwus;   // row strides
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
  void* dg;                      // [T, F] in rows of gl_grad_row(F), du behind it
  int64_t T, F;
};
// The saved factors p and q of [T, F], rounded to 24 bits, in planes of rows of F rounded up to 16: the high 16 bits of each binary32
// value of p, those of q, then the next 8 bits of p, those of q.
__host__ __device__ inline int64_t gl_saved_row(int64_t F) { return (F + 15) / 16 * 16; }
__host__ __device__ inline size_t gl_saved_bytes(int64_t T, int64_t F) { return (size_t)6 * T * gl_saved_row(F); }

// Rows of dg and du [T, F] in the workspace: whole 128-byte lines apart (a copied row of 128 bytes otherwise touches two lines).
__host__ __device__ inline int64_t gl_grad_row(int64_t F) { return (F + 63) / 64 * 64; }

template <bool BF>
cudaError_t gl_forward(const GlArgs& a, cudaStream_t st);
template <bool BF>
cudaError_t gl_backward(const GlArgs& a, cudaStream_t st);
template <bool BF>
cudaError_t gl_few(const GlFewArgs& a, cudaStream_t st);
template <bool BF>
cudaError_t gl_scale(const GlScaleArgs& a, cudaStream_t st);

// ---- log probabilities ----
constexpr int LP_TOP = 32;       // most alternatives of a row

struct LpArgs {
  const void* x;                 // [rows, cols], row stride xs
  const int64_t* targets;        // [rows]
  float* lp;                     // [rows]
  float* entropy;                // [rows]
  float* stats;                  // [rows][3] or null: largest logit, sum of exponentials, entropy
  float* top_lp;                 // [rows, top]
  int64_t* top_index;
  int64_t rows, xs;
  uint32_t cols;
  int top;
  int dtype;
  float temperature;
  int* status;
};
struct LpGradArgs {
  const void* x;
  const int64_t* targets;
  const float* stats;
  const float* grad;             // [rows] or null
  const float* grad_entropy;     // [rows] or null
  void* dx;                      // [rows, cols], row stride ds
  int64_t rows, xs, ds;
  uint32_t cols;
  int dtype;
  float temperature;
};
cudaError_t launch_log_probs(const LpArgs& a, cudaStream_t st);
cudaError_t launch_log_probs_grad(const LpGradArgs& a, cudaStream_t st);

// ---- embedding ----
constexpr int EM_CHUNK = 32;     // tokens of a row whose sum is one chain
constexpr int EM_SMALL = 4096;   // tokens that one CTA sorts in shared memory
// Tokens of a CTA of the passes of a longer sort: fewer start more CTAs, more leave fewer counts to add up (16384 tokens, 200000 rows
// of 128: 39 us with 1024 and 44 with 2048; 60000 tokens, 128256 rows of 512: 90 and 81).
inline int em_block(int64_t n) { return n <= 32768 ? 1024 : 2048; }
constexpr int EM_BINS = 512;     // values of a digit

constexpr int EM_FEW = 8;        // tokens of a short chunk
constexpr uint32_t EM_MORE = 0x80000000u;   // of a chunk: one of several of its row
struct EmUnits {
  uint32_t few, many, rows;      // short chunks, long ones, rows of several
};

struct EmArgs {
  const void* ids;               // [n], int32 or int64
  int wide;                      // int64
  const void* w;                 // lookup: [rows, cols], row stride ws
  void* y;                       // lookup: [n, cols], row stride ys
  const void* dy;                // gradient: [n, cols], row stride ys
  void* dw;                      // gradient: [rows, cols], row stride ws
  int64_t n, rows, cols, ws, ys;
  int64_t padding;               // its tokens give no gradient; -1: none
  float scale;
  int dtype;
  int* status;
  // workspace of the gradient
  uint32_t* key[2];              // longer sorts: [n] ids in sorted order (rows: no gradient), and of the pass before
  uint32_t* pos[2];              // [n] their tokens
  uint32_t* count;               // longer sorts: [blocks][EM_BINS] or [bins][blocks]
  EmUnits* found;
  uint4* unit;                   // [n]: chunks (first place, tokens and EM_MORE, row): short ones from the front, long ones from the back
  uint4* row;                    // [n / EM_CHUNK + 1]: rows of several chunks (first place, end, row)
  float* part;                   // [2 (n / EM_CHUNK + 1)][cols] sums of such chunks
};
cudaError_t launch_embedding(const EmArgs& a, cudaStream_t st);
cudaError_t launch_embedding_grad(const EmArgs& a, cudaStream_t st);

}  // namespace detattn
