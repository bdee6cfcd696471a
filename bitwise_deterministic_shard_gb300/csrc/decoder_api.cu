// Host side of the operators at the ends and in the middle of a decoder (include/detattn.h): argument
// checks, workspace layout, tensor maps and launches.
#include <cmath>
#include <cstring>

#include "../../include/detattn.h"
#include "decoder_kernels.h"
#include "host_util.h"

using namespace detattn;

namespace {

// boxes of 64 x 64 of a matrix of 16-bit elements
bool tensor_map(CUtensorMap* m, const void* at, int dtype, int64_t rows, int64_t cols, int64_t stride) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? stride : cols) * 2};   // one row: not used, but must be valid
  const cuuint32_t box[2] = {64, 64}, one[2] = {1, 1};
  const CUtensorMapDataType type = dtype == DA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(m, type, 2, const_cast<void*>(at), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool tensor_map(CUtensorMap* m, const da_matrix& x) { return tensor_map(m, x.ptr, x.dtype, x.rows, x.cols, x.row_stride); }

// ---- gated feed-forward ----
constexpr int64_t kMaxRows = (int64_t)1 << 24;

int check(const da_matrix* x) {   // a matrix that tensor maps and 16-byte accesses can take
  if (!x) return DA_EINVAL;
  if (x->dtype != DA_BF16 && x->dtype != DA_F16) return DA_EDTYPE;
  if (x->rows < 0 || x->cols < 8 || x->cols % 8 || x->rows > kMaxRows || x->cols > kMaxRows) return DA_ESHAPE;
  if (x->rows > 1 && (x->row_stride < x->cols || x->row_stride >= ((int64_t)1 << 38))) return DA_ESHAPE;
  if (x->rows > 0 && !x->ptr) return DA_EINVAL;
  if (!aligned(x->ptr, 16) || (x->rows > 1 && x->row_stride % 8)) return DA_EALIGN;
  return DA_OK;
}
int check(const da_matrix* x, int dtype, int64_t rows, int64_t cols) {
  const int e = check(x);
  if (e) return e;
  if (x->dtype != dtype) return DA_EDTYPE;
  return x->rows == rows && x->cols == cols ? DA_OK : DA_ESHAPE;
}
int check(const da_matrix* x, const da_matrix* wg, const da_matrix* wu) {
  int e = check(x);
  if (e || (e = check(wg)) || (e = check(wu, wg->dtype, wg->rows, wg->cols))) return e;
  if (wg->dtype != x->dtype) return DA_EDTYPE;
  if (wg->cols != x->cols || wg->rows < 8 || wg->rows % 8) return DA_ESHAPE;
  // tiles of a launch, the narrow ones
  if (((x->rows >> 8) + 1) * ((wg->rows >> 6) + 1) > (int64_t)1 << 28 || ((wg->rows >> 7) + 2) * ((wg->cols >> 7) + 1) > (int64_t)1 << 28 ||
      ((x->rows >> 8) + 1) * ((wg->cols >> 7) + 1) > (int64_t)1 << 28)
    return DA_ESHAPE;
  return DA_OK;
}
int64_t stride(const da_matrix& x) { return x.rows > 1 ? x.row_stride : x.cols; }

// ---- log probabilities and embedding ----
size_t size_of(int dtype) { return dtype == DA_F32 ? 4 : 2; }
int check_rows(const da_matrix* x) {
  if (!x) return DA_EINVAL;
  if (x->dtype != DA_F32 && x->dtype != DA_BF16 && x->dtype != DA_F16) return DA_EDTYPE;
  if (x->rows < 0 || x->cols < 1 || (x->rows > 1 && (x->row_stride < x->cols || x->row_stride >= ((int64_t)1 << 40)))) return DA_ESHAPE;
  if (x->rows > ((int64_t)1 << 31) - 2 || x->cols > (int64_t)1 << 30) return DA_ESHAPE;
  if (x->rows > 0 && !x->ptr) return DA_EINVAL;
  return aligned(x->ptr, size_of(x->dtype)) ? DA_OK : DA_EALIGN;
}
int check_logits(const da_matrix* x, float temperature) {
  const int e = check_rows(x);
  if (e) return e;
  if (!(temperature >= 0x1p-60f && temperature <= 0x1p60f)) return DA_EINVAL;
  return x->rows * (x->cols / 4096 + 8) >= (int64_t)1 << 31 ? DA_ESHAPE : DA_OK;   // CTAs of a launch
}
int check_ids(const void* ids, int bits, int64_t n, const da_matrix* like) {
  if (bits != 32 && bits != 64) return DA_EINVAL;
  if (n > 0 && !ids) return DA_EINVAL;
  if (!aligned(ids, bits / 8)) return DA_EALIGN;
  return n * (like->cols / 128 + 1) >= (int64_t)1 << 33 ? DA_ESHAPE : DA_OK;       // warps of a launch
}
struct EmWs {
  size_t key[2], pos[2], found, unit, row, count, part, total;
};
EmWs em_layout(int64_t n, int64_t cols) {
  EmWs w;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes);
    return here;
  };
  const bool small = n <= EM_SMALL;
  for (int i = 0; i < 2; i++) {
    w.key[i] = take(small ? 0 : (size_t)n * 4);
    w.pos[i] = take(small && i ? 0 : (size_t)n * 4);
  }
  w.found = take(sizeof(EmUnits));
  w.unit = take((size_t)n * 16);
  w.row = take(n <= EM_CHUNK ? 0 : (size_t)(n / EM_CHUNK + 1) * 16);
  w.count = take(small ? 0 : (size_t)((n + em_block(n) - 1) / em_block(n)) * EM_BINS * 4);
  w.part = take(n <= EM_CHUNK ? 0 : (size_t)2 * (n / EM_CHUNK + 1) * cols * 4);
  w.total = at;
  return w;
}

}  // namespace

#define DA_EXPORT __attribute__((visibility("default")))

extern "C" {

DA_EXPORT size_t dgl_saved_bytes(int64_t tokens, int64_t hidden) {
  return tokens < 0 || hidden < 0 || tokens > kMaxRows || hidden > kMaxRows ? 0 : gl_saved_bytes(tokens, hidden);
}

DA_EXPORT int dgl_forward(const da_matrix* x, const da_matrix* wg, const da_matrix* wu, int activation, const da_matrix* h,
                          void* saved, int32_t* dev_status, da_stream_t stream) {
  int e = check(x, wg, wu);
  if (e || (e = check(h, x->dtype, x->rows, wg->rows))) return e;
  if (activation < DGL_SILU || activation > DGL_RELU) return DA_EINVAL;
  if (!aligned(saved, 16) || !aligned(dev_status, 4)) return DA_EALIGN;
  if (x->rows == 0) return DA_OK;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = x->dtype == DA_BF16;
  if (!saved && x->rows <= GL_FEW) {
    const GlFewArgs f = {x->ptr, wg->ptr, wu->ptr, const_cast<void*>(h->ptr), stride(*x), stride(*wg), stride(*wu), stride(*h),
                         (int)x->rows, (int)x->cols, (int)wg->rows, activation};
    return launched(bf ? gl_few<true>(f, st) : gl_few<false>(f, st));
  }
  GlArgs a;
  std::memset(&a, 0, sizeof(a));
  a.T = (int)x->rows; a.D = (int)x->cols; a.F = (int)wg->rows;
  a.h = const_cast<void*>(h->ptr); a.hs = stride(*h);
  a.saved = static_cast<unsigned char*>(saved);
  a.activation = activation;
  a.status = dev_status;
  if (!tensor_map(&a.x, *x) || !tensor_map(&a.wg, *wg) || !tensor_map(&a.wu, *wu)) return DA_ECUDA;
  return launched(bf ? gl_forward<true>(a, st) : gl_forward<false>(a, st));
}

DA_EXPORT size_t dgl_workspace_bytes(int64_t tokens, int64_t hidden) {
  return tokens < 0 || hidden < 0 || tokens > kMaxRows || hidden > kMaxRows ? 0 : round_up((size_t)4 * tokens * gl_grad_row(hidden));
}

DA_EXPORT int dgl_backward(const da_matrix* dh, const da_matrix* x, const da_matrix* wg, const da_matrix* wu, const void* saved,
                           const da_matrix* dx, const da_matrix* dwg, const da_matrix* dwu, void* ws, size_t ws_bytes,
                           int32_t* dev_status, da_stream_t stream) {
  int e = check(x, wg, wu);
  if (e || (e = check(dh, x->dtype, x->rows, wg->rows))) return e;
  if (dx && (e = check(dx, x->dtype, x->rows, x->cols))) return e;
  if (!dwg != !dwu) return DA_EINVAL;
  if (dwg && ((e = check(dwg, x->dtype, wg->rows, wg->cols)) || (e = check(dwu, x->dtype, wg->rows, wg->cols)))) return e;
  const int64_t T = x->rows, D = x->cols, F = wg->rows;
  if (T > 0 && !saved) return DA_EINVAL;
  const size_t need = dgl_workspace_bytes(T, F);
  if (need > 0 && (!ws || ws_bytes < need)) return DA_EWORKSPACE;
  if (!aligned(saved, 16) || !aligned(ws, 256) || !aligned(dev_status, 4)) return DA_EALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = x->dtype == DA_BF16;
  if (T == 0) {   // sums of nothing
    for (const da_matrix* w : {dwg, dwu})
      if (w && (e = launched(cudaMemset2DAsync(const_cast<void*>(w->ptr), 2 * stride(*w), 0, 2 * D, F, st)))) return e;
    return DA_OK;
  }
  if (!dx && !dwg) return DA_OK;
  uint16_t* const dg = static_cast<uint16_t*>(ws);
  const GlScaleArgs s = {dh->ptr, stride(*dh), static_cast<const unsigned char*>(saved), dg, T, F};
  if ((e = launched(bf ? gl_scale<true>(s, st) : gl_scale<false>(s, st)))) return e;
  GlArgs a;
  std::memset(&a, 0, sizeof(a));
  a.T = (int)T; a.D = (int)D; a.F = (int)F;
  a.status = dev_status;
  const int64_t row = gl_grad_row(F);
  if (!tensor_map(&a.x, *x) || !tensor_map(&a.wg, *wg) || !tensor_map(&a.wu, *wu) ||
      !tensor_map(&a.dg, dg, x->dtype, T, F, row) || !tensor_map(&a.du, dg + T * row, x->dtype, T, F, row))
    return DA_ECUDA;
  if (dx) a.dx = const_cast<void*>(dx->ptr), a.dxs = stride(*dx);
  if (dwg) {
    a.dwg = const_cast<void*>(dwg->ptr), a.dwgs = stride(*dwg);
    a.dwu = const_cast<void*>(dwu->ptr), a.dwus = stride(*dwu);
  }
  return launched(bf ? gl_backward<true>(a, st) : gl_backward<false>(a, st));
}

DA_EXPORT int dlp_forward(const da_matrix* logits, const int64_t* targets, float temperature, int top, float* log_probs,
                          float* entropy, float* saved, float* top_log_probs, int64_t* top_indices, int32_t* dev_status,
                          da_stream_t stream) {
  const int e = check_logits(logits, temperature);
  if (e) return e;
  if (top < 0 || top > LP_TOP || top > logits->cols) return DA_EINVAL;
  if (logits->rows == 0) return DA_OK;
  if (!targets || !log_probs || !entropy || (top > 0 && (!top_log_probs || !top_indices))) return DA_EINVAL;
  if (!aligned(targets, 8) || !aligned(top_indices, 8) || !aligned(log_probs, 4) || !aligned(entropy, 4) || !aligned(saved, 4) ||
      !aligned(top_log_probs, 4) || !aligned(dev_status, 4))
    return DA_EALIGN;
  LpArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = logits->ptr; a.targets = targets; a.lp = log_probs; a.entropy = entropy; a.stats = saved;
  a.top_lp = top_log_probs; a.top_index = top_indices;
  a.rows = logits->rows; a.xs = stride(*logits); a.cols = (uint32_t)logits->cols;
  a.top = top; a.dtype = logits->dtype; a.temperature = temperature; a.status = dev_status;
  return launched(launch_log_probs(a, (cudaStream_t)stream));
}

DA_EXPORT int dlp_backward(const da_matrix* logits, const int64_t* targets, const float* saved, const float* grad,
                           const float* grad_entropy, float temperature, const da_matrix* dlogits, da_stream_t stream) {
  int e = check_logits(logits, temperature);
  if (e || (e = check_rows(dlogits))) return e;
  if (dlogits->dtype != logits->dtype) return DA_EDTYPE;
  if (dlogits->rows != logits->rows || dlogits->cols != logits->cols) return DA_ESHAPE;
  if (logits->rows == 0) return DA_OK;
  if (!targets || !saved) return DA_EINVAL;
  if (!aligned(targets, 8) || !aligned(saved, 4) || !aligned(grad, 4) || !aligned(grad_entropy, 4)) return DA_EALIGN;
  LpGradArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = logits->ptr; a.targets = targets; a.stats = saved; a.grad = grad; a.grad_entropy = grad_entropy;
  a.dx = const_cast<void*>(dlogits->ptr);
  a.rows = logits->rows; a.xs = stride(*logits); a.ds = stride(*dlogits); a.cols = (uint32_t)logits->cols;
  a.dtype = logits->dtype; a.temperature = temperature;
  return launched(launch_log_probs_grad(a, (cudaStream_t)stream));
}

DA_EXPORT int dte_forward(const void* ids, int id_bits, const da_matrix* w, float scale, const da_matrix* y, int32_t* dev_status,
                          da_stream_t stream) {
  int e = check_rows(w);
  if (e || (e = check_rows(y))) return e;
  if (y->dtype != w->dtype) return DA_EDTYPE;
  if (y->cols != w->cols || w->rows < 1) return DA_ESHAPE;
  if ((e = check_ids(ids, id_bits, y->rows, w))) return e;
  if (!std::isfinite(scale)) return DA_EINVAL;
  if (!aligned(dev_status, 4)) return DA_EALIGN;
  if (y->rows == 0) return DA_OK;
  EmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.ids = ids; a.wide = id_bits == 64; a.w = w->ptr; a.y = const_cast<void*>(y->ptr);
  a.n = y->rows; a.rows = w->rows; a.cols = w->cols; a.ws = stride(*w); a.ys = stride(*y);
  a.padding = -1; a.scale = scale; a.dtype = w->dtype; a.status = dev_status;
  return launched(launch_embedding(a, (cudaStream_t)stream));
}

DA_EXPORT size_t dte_workspace_bytes(int64_t n, int64_t cols) {
  if (n < 0 || n > ((int64_t)1 << 31) - 2 || cols < 1 || cols > (int64_t)1 << 30) return 0;
  return em_layout(n, cols).total;
}

DA_EXPORT int dte_backward(const void* ids, int id_bits, const da_matrix* dy, float scale, int64_t padding, const da_matrix* dw,
                           void* ws, size_t ws_bytes, int32_t* dev_status, da_stream_t stream) {
  int e = check_rows(dw);
  if (e || (e = check_rows(dy))) return e;
  if (dy->dtype != dw->dtype) return DA_EDTYPE;
  if (dy->cols != dw->cols || dw->rows < 1) return DA_ESHAPE;
  if ((e = check_ids(ids, id_bits, dy->rows, dw))) return e;
  if (!std::isfinite(scale) || padding < -1 || padding >= dw->rows) return DA_EINVAL;
  const EmWs w = em_layout(dy->rows, dy->cols);
  if (w.total > 0 && (!ws || ws_bytes < w.total)) return DA_EWORKSPACE;
  if (!aligned(ws, 256) || !aligned(dev_status, 4)) return DA_EALIGN;
  EmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.ids = ids; a.wide = id_bits == 64; a.dy = dy->ptr; a.dw = const_cast<void*>(dw->ptr);
  a.n = dy->rows; a.rows = dw->rows; a.cols = dw->cols; a.ws = stride(*dw); a.ys = stride(*dy);
  a.padding = padding; a.scale = scale; a.dtype = dw->dtype; a.status = dev_status;
  char* const p = static_cast<char*>(ws);
  for (int i = 0; i < 2; i++) {
    a.key[i] = reinterpret_cast<uint32_t*>(p + w.key[i]);
    a.pos[i] = reinterpret_cast<uint32_t*>(p + w.pos[i]);
  }
  a.found = reinterpret_cast<EmUnits*>(p + w.found);
  a.unit = reinterpret_cast<uint4*>(p + w.unit);
  a.row = reinterpret_cast<uint4*>(p + w.row);
  a.count = reinterpret_cast<uint32_t*>(p + w.count);
  a.part = reinterpret_cast<float*>(p + w.part);
  return launched(launch_embedding_grad(a, (cudaStream_t)stream));
}

}  // extern "C"
