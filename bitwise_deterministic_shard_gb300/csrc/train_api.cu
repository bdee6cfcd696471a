// Host side of the training operators of include/detattn.h: argument checks, workspace layout,
// tensor maps and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/detattn.h"
#include "attn_train.h"
#include "host_util.h"
#include "train_kernels.h"

using namespace detattn;

namespace {

constexpr int64_t kMaxS = (int64_t)1 << 24;   // positions are exact in binary32

int check(const da_tensor& t) {
  if (t.dtype != DA_BF16 && t.dtype != DA_F16) return DA_EDTYPE;
  if (t.B < 0 || t.H < 1 || t.S < 0 || t.D < 8 || t.D > 128 || t.D % 8 != 0) return DA_ESHAPE;
  if (t.S > kMaxS || t.B > 65535 || t.H > 65535) return DA_ESHAPE;
  if (t.stride[3] != 1) return DA_ESHAPE;
  const int64_t n[3] = {t.B, t.H, t.S};
  for (int i = 0; i < 3; i++)
    if (n[i] > 1 && (t.stride[i] <= 0 || t.stride[i] >= ((int64_t)1 << 38))) return DA_ESHAPE;
  if (t.B * t.S > 0 && !t.ptr) return DA_EINVAL;
  if (!aligned(t.ptr, 16)) return DA_EALIGN;
  for (int i = 0; i < 3; i++)
    if (n[i] > 1 && t.stride[i] % 8 != 0) return DA_EALIGN;
  return DA_OK;
}

bool same_shape(const da_tensor& a, const da_tensor& b) {
  return a.B == b.B && a.H == b.H && a.S == b.S && a.D == b.D;
}

int check(const dta_desc* d) {
  if (!d) return DA_EINVAL;
  int e;
  if ((e = check(d->q)) || (e = check(d->k)) || (e = check(d->v))) return e;
  if (d->q.dtype != d->k.dtype || d->q.dtype != d->v.dtype) return DA_EDTYPE;
  if (!same_shape(d->k, d->v) || d->k.B != d->q.B || d->k.D != d->q.D) return DA_ESHAPE;
  if (d->q.H % d->k.H != 0 || d->q.S > d->k.S) return DA_ESHAPE;
  if (d->q.B * d->q.H * (d->k.S / TA_TILE + 1) > (int64_t)1 << 30) return DA_ESHAPE;   // CTAs of a launch
  if (!std::isnan(d->scale) && !std::isfinite(d->scale)) return DA_EINVAL;
  // beyond these the cap's factors, their squares or the scale over it leave binary32's range
  if (d->softcap != 0.f && (!(d->softcap >= 0x1p-60f && d->softcap <= 0x1p60f) || std::fabs(d->scale) > 0x1p60f)) return DA_EINVAL;
  if (d->prefix && !d->causal) return DA_EINVAL;
  if (!aligned(d->slopes, 4) || !aligned(d->docs, 4) || !aligned(d->prefix, 4) || !aligned(d->dev_status, 4))
    return DA_EALIGN;
  return DA_OK;
}

int check_like(const da_tensor* t, const da_tensor& like) {
  if (!t) return DA_EINVAL;
  const int e = check(*t);
  if (e) return e;
  if (t->dtype != like.dtype) return DA_EDTYPE;
  return same_shape(*t, like) ? DA_OK : DA_ESHAPE;
}

// {D, pack heads, S, H / pack, B}; boxes of 64 columns x (pack heads x rows) of one group of heads
bool tensor_map(CUtensorMap* m, const da_tensor& t, int pack, int rows) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t some = 16;   // the stride of a dimension of one element is not used, but must be valid
  const cuuint64_t sb = t.B > 1 ? t.stride[0] * 2 : some, sh = t.H > 1 ? t.stride[1] * 2 : some,
                   ss = t.S > 1 ? t.stride[2] * 2 : some;
  const cuuint64_t dims[5] = {(cuuint64_t)t.D, (cuuint64_t)pack, (cuuint64_t)t.S, (cuuint64_t)(t.H / pack), (cuuint64_t)t.B};
  const cuuint64_t strides[4] = {sh, ss, t.H / pack > 1 ? sh * pack : some, sb};
  const cuuint32_t box[5] = {64, (cuuint32_t)pack, (cuuint32_t)rows, 1, 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const CUtensorMapDataType type = t.dtype == DA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(m, type, 5, const_cast<void*>(t.ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cap's coefficients (see attn_train_fwd.cuh): fitted for the least greatest error, least squares with weights moved
// toward the largest errors.
TaCap cap_of(float scale, float softcap) {
  constexpr double full[6] = {0x1.ffff96p-1, -0x1.553ce0p-2, 0x1.0f6ea4p-3, -0x1.a191cep-5, 0x1.0803b2p-6, -0x1.742c6ap-9};
  constexpr double less[4] = {0x1.ffffb2p-1, -0x1.55341ap-2, 0x1.0d366ap-3, -0x1.634ea8p-5};
  const auto twice = [](double x) {
    const float f = (float)x;
    uint32_t b;
    std::memcpy(&b, &f, 4);
    return ((unsigned long long)b << 32) | b;
  };
  TaCap c;
  std::memset(&c, 0, sizeof(c));
  if (!(softcap > 0.f)) {
    c.f = 1.f;
    return c;
  }
  const double k = (double)scale / softcap, f = softcap * 1.4426950408889634;
  double power = k * f;
  for (int i = 0; i < 6; i++) {
    c.c[i] = twice(full[i] * power);
    if (i < 4) c.s[i] = twice(less[i] * power);
    power *= k * k;
  }
  c.k = (float)k;
  c.f = (float)f;
  // Beyond these factors a coefficient could leave binary32's range, and an error in units of the cap would be one of many
  // scores (2^-22 of a cap of 10^5 is 0.02).
  const double a = std::fabs(k);
  if (a >= 0x1p-12 && a <= 0x1p10) {
    c.most = (float)(1 / a);
    c.least = 0.5f * c.most;
  } else if (a > 0x1p10) {
    c.most = c.least = -1.f;   // the general form, for a score of 0 too
  } else {
    // A cap of more than 4096 times the scale: tanh's series, as many terms as binary32 holds, up to where the next one is 2^-22
    // of the value; the scores beyond (a quarter to a 32nd of the cap) take the general form.
    constexpr double series[4] = {1, -1. / 3, 2. / 15, -17. / 315};
    const int terms = a >= 0x1p-20 ? 4 : a >= 0x1p-30 ? 3 : 2;
    power = k * f;
    for (int i = 0; i < 4; i++) {
      c.s[i] = twice(i < terms ? series[i] * power : 0);
      power *= k * k;
    }
    c.far = 1;
    c.most = c.least = (float)std::min((terms == 4 ? 0x1p-2 : terms == 3 ? 0x1p-3 : 0x1p-5) / a, 0x1p60);
  }
  return c;
}

void shapes(const dta_desc* d, TaArgs& a, bool backward) {
  std::memset(&a, 0, sizeof(a));
  a.B = (int)d->q.B; a.Hq = (int)d->q.H; a.Hkv = (int)d->k.H;
  a.Sq = (int)d->q.S; a.Skv = (int)d->k.S; a.D = (int)d->q.D;
  a.group = a.Hq / a.Hkv;
  a.pack = !backward && (int64_t)a.Sq * a.group <= TA_TILE ? a.group : 1;
  a.qrows = TA_TILE / a.pack;
  a.qtiles = a.pack > 1 ? 1 : (a.Sq + TA_TILE - 1) / TA_TILE;
  a.ktiles = (a.Skv + TA_TILE - 1) / TA_TILE;
  a.causal = d->causal ? 1 : 0;
  a.scale = std::isnan(d->scale) ? (float)(1.0 / std::sqrt((double)d->q.D)) : d->scale;
  a.softcap = d->softcap;
  a.cap = cap_of(a.scale, a.softcap);
  a.slopes = d->slopes; a.docs = d->docs; a.prefix = d->prefix; a.status = d->dev_status;
}

int head_width(int D) { return D <= 64 ? 64 : 128; }

// Key ranges of the forward pass in the form whose groups share a query tile, 0 for the form with a tile each.  A
// function of the sizes alone (152 SMs), so the order of the sums is too.
//   One tile of queries a head group (few queries): so many ranges that rounds of CTAs times a CTA's key tiles are least, where
//   filling the pipeline and the join cost about four key tiles more (0.8 us each) and every range two thirds of one in
//   the join: 2 key heads of 32768 keys 34 us in 16 or 24 ranges, 49 in 64, 224 in one; 32 of them 93 us in 4, 106 in 8;
//   512 keys 12.9 us in one range, 12.8 to 14.1 in two.
//   Else the shared form, unsplit, where the other would leave half of the SMs without a CTA (18 heads of 777 queries: 22.6
//   against 24.6 us); with more CTAs its second reading of the keys costs more (16 heads of 4096: 120 against 92 us).
constexpr int TA_SHARED = 152 / 2;
int split_rule(const TaArgs& a) {
  const int64_t units = (int64_t)a.B * (a.Hq / a.pack);
  if (a.ktiles < 2) return 0;
  if (a.qtiles > 1 || a.ktiles < 4) return units * ((a.qtiles + 1) / 2) <= TA_SHARED ? 1 : 0;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= a.ktiles / 2 && s <= 64; s++) {
    const int64_t cost = 3 * ((units * s + 151) / 152) * ((a.ktiles + s - 1) / s + (s > 1 ? 4 : 2)) + 2 * s;   // in thirds of a tile
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

struct Ws {
  size_t bounds, qbounds, part, total;   // part: the split forward's sums, or the backward's rows array
};
Ws layout(const TaArgs& a, bool backward) {
  Ws w;
  w.bounds = 0;
  w.qbounds = round_up(a.docs ? (size_t)a.B * a.ktiles * sizeof(TaBounds) : 0);
  w.part = w.qbounds + round_up(a.docs && backward ? (size_t)a.B * a.qtiles * sizeof(TaBounds) : 0);
  size_t more = 0;
  if (backward) {
    more = (size_t)a.B * a.Hq * a.qtiles * TA_TILE * 2 * sizeof(float);
  } else if (const int s = split_rule(a); s > 1) {
    more = (size_t)2 * s * a.B * (a.Hq / a.pack) * TA_TILE * (head_width(a.D) + 4) * 4;
  }
  w.total = w.part + round_up(more);
  return w;
}

int check_matrix(const da_matrix* x, int dtype, int64_t rows, int64_t cols) {
  if (!x) return DA_EINVAL;
  if (x->dtype != DA_F32 && x->dtype != DA_BF16 && x->dtype != DA_F16) return DA_EDTYPE;
  if (dtype >= 0 && x->dtype != dtype) return DA_EDTYPE;
  if (x->rows < 0 || x->cols < 1 || (x->rows > 1 && x->row_stride < x->cols)) return DA_ESHAPE;
  if (rows >= 0 && (x->rows != rows || x->cols != cols)) return DA_ESHAPE;
  if (x->rows > ((int64_t)1 << 31) - 1 || x->cols > ((int64_t)1 << 31) - 1) return DA_ESHAPE;
  if (x->rows > 0 && !x->ptr) return DA_EINVAL;
  return aligned(x->ptr, x->dtype == DA_F32 ? 4 : 2) ? DA_OK : DA_EALIGN;
}

int check_weight(const void* w, int wdtype, int dtype) {
  if (wdtype != DA_F32 && wdtype != dtype) return DA_EDTYPE;
  return aligned(w, wdtype == DA_F32 ? 4 : 2) ? DA_OK : DA_EALIGN;
}

}  // namespace

#define DA_EXPORT __attribute__((visibility("default")))

extern "C" {

DA_EXPORT size_t dta_workspace_bytes(const dta_desc* d, int backward) {
  if (check(d)) return 0;
  TaArgs a;
  shapes(d, a, backward != 0);
  return layout(a, backward != 0).total;
}

DA_EXPORT int dta_forward(const dta_desc* d, const da_tensor* out, float* lse, void* ws, size_t ws_bytes,
                          da_stream_t stream) {
  int e = check(d);
  if (e || (e = check_like(out, d->q))) return e;
  if (!aligned(lse, 4)) return DA_EALIGN;
  TaArgs a;
  shapes(d, a, false);
  const Ws w = layout(a, false);
  if (w.total > 0 && (!ws || ws_bytes < w.total)) return DA_EWORKSPACE;
  if (!aligned(ws, 256)) return DA_EALIGN;
  if (a.B == 0 || a.Sq == 0) return DA_OK;
  cudaStream_t st = (cudaStream_t)stream;
  a.splits = split_rule(a);
  a.lse = lse;
  a.bounds = reinterpret_cast<const TaBounds*>((char*)ws + w.bounds);
  a.part = reinterpret_cast<float*>((char*)ws + w.part);
  a.out = const_cast<void*>(out->ptr);
  for (int i = 0; i < 3; i++) a.os[i] = out->stride[i];
  if (!tensor_map(&a.q, d->q, a.pack, a.qrows) || !tensor_map(&a.o, *out, a.pack, a.qrows) ||
      !tensor_map(&a.k, d->k, 1, TA_TILE) || !tensor_map(&a.v, d->v, 1, TA_TILE))
    return DA_ECUDA;
  if (a.docs && (e = launched(ta_bounds(a.docs, a.B, a.Skv, a.Sq, const_cast<TaBounds*>(a.bounds), nullptr, st)))) return e;
  const bool bf = d->q.dtype == DA_BF16;
  if (head_width(a.D) == 64) return launched(bf ? ta_forward<64, true>(a, st) : ta_forward<64, false>(a, st));
  return launched(bf ? ta_forward<128, true>(a, st) : ta_forward<128, false>(a, st));
}

DA_EXPORT int dta_backward(const dta_desc* d, const da_tensor* out, const float* lse, const da_tensor* grad,
                           const da_tensor* dq, const da_tensor* dk, const da_tensor* dv, void* ws, size_t ws_bytes,
                           da_stream_t stream) {
  int e = check(d);
  if (e || (e = check_like(out, d->q)) || (e = check_like(grad, d->q)) || (e = check_like(dq, d->q)) ||
      (e = check_like(dk, d->k)) || (e = check_like(dv, d->v)))
    return e;
  if (!lse && d->q.B * d->q.S > 0) return DA_EINVAL;
  if (!aligned(lse, 4)) return DA_EALIGN;
  TaArgs a;
  shapes(d, a, true);
  const Ws w = layout(a, true);
  if (w.total > 0 && (!ws || ws_bytes < w.total)) return DA_EWORKSPACE;
  if (!aligned(ws, 256)) return DA_EALIGN;
  if (a.B == 0 || a.Skv == 0) return DA_OK;
  cudaStream_t st = (cudaStream_t)stream;
  a.rows = reinterpret_cast<float*>((char*)ws + w.part);
  a.bounds = reinterpret_cast<const TaBounds*>((char*)ws + w.bounds);
  a.qbounds = reinterpret_cast<const TaBounds*>((char*)ws + w.qbounds);
  if (!tensor_map(&a.k, d->k, 1, TA_TILE) || !tensor_map(&a.v, d->v, 1, TA_TILE) || !tensor_map(&a.dk, *dk, 1, TA_TILE) ||
      !tensor_map(&a.dv, *dv, 1, TA_TILE))
    return DA_ECUDA;
  if (a.Sq > 0 && (!tensor_map(&a.q, d->q, 1, TA_TILE) || !tensor_map(&a.go, *grad, 1, TA_TILE) ||
                   !tensor_map(&a.o, *out, 1, TA_TILE) ||
                   !tensor_map(&a.dq, *dq, 1, TA_TILE)))
    return DA_ECUDA;
  if (a.docs && (e = launched(ta_bounds(a.docs, a.B, a.Skv, a.Sq, const_cast<TaBounds*>(a.bounds),
                                       const_cast<TaBounds*>(a.qbounds), st))))
    return e;
  const bool bf = d->q.dtype == DA_BF16;
  a.lse = const_cast<float*>(lse);
  const bool narrow = head_width(a.D) == 64;
  // dq first: it leaves the rows array that the other kernel takes
  e = launched(narrow ? bf ? ta_dq<64, true>(a, st) : ta_dq<64, false>(a, st)
                      : bf ? ta_dq<128, true>(a, st) : ta_dq<128, false>(a, st));
  if (e) return e;
  return launched(narrow ? bf ? ta_dkv<64, true>(a, st) : ta_dkv<64, false>(a, st)
                         : bf ? ta_dkv<128, true>(a, st) : ta_dkv<128, false>(a, st));
}

DA_EXPORT int dln_forward(const da_matrix* x, const void* w, const void* b, int wdtype, float eps, const da_matrix* y,
                          float* mean, float* rstd, da_stream_t stream) {
  int e = check_matrix(x, -1, -1, -1);
  if (e || (e = check_matrix(y, x->dtype, x->rows, x->cols)) || (e = check_weight(w, wdtype, x->dtype)) ||
      (e = check_weight(b, wdtype, x->dtype)))
    return e;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return DA_EINVAL;
  if (x->rows == 0) return DA_OK;
  if (!mean != !rstd) return DA_EINVAL;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return DA_EALIGN;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x->ptr; a.y = const_cast<void*>(y->ptr); a.w = w; a.b = b; a.mean = mean; a.rstd = rstd;
  a.rows = x->rows; a.cols = x->cols; a.xs = x->row_stride; a.ys = y->row_stride;
  a.dtype = x->dtype; a.wdtype = wdtype; a.eps = eps;
  return launched(launch_norm_forward(a, (cudaStream_t)stream));
}

DA_EXPORT size_t dln_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return 0;
  return round_up((size_t)2 * norm_parts(rows, cols) * cols * 4);
}

DA_EXPORT int dln_backward(const da_matrix* dy, const da_matrix* x, const void* w, int wdtype, const float* mean,
                           const float* rstd, const da_matrix* dx, void* dw, void* db, void* ws, size_t ws_bytes,
                           da_stream_t stream) {
  int e = check_matrix(x, -1, -1, -1);
  if (e || (e = check_matrix(dy, x->dtype, x->rows, x->cols)) || (e = check_matrix(dx, x->dtype, x->rows, x->cols)) ||
      (e = check_weight(w, wdtype, x->dtype)) || (e = check_weight(dw, wdtype, x->dtype)) ||
      (e = check_weight(db, wdtype, x->dtype)))
    return e;
  if (x->rows > 0 && (!mean || !rstd)) return DA_EINVAL;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return DA_EALIGN;
  const size_t need = dw || db ? dln_workspace_bytes(x->rows, x->cols) : 0;
  if (need > 0 && (!ws || ws_bytes < need)) return DA_EWORKSPACE;
  if (!aligned(ws, 256)) return DA_EALIGN;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x->ptr; a.dy = dy->ptr; a.y = const_cast<void*>(dx->ptr); a.w = w;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.dw = dw; a.db = db; a.part = need ? (float*)ws : nullptr;
  a.rows = x->rows; a.cols = x->cols; a.xs = x->row_stride; a.dys = dy->row_stride; a.ys = dx->row_stride;
  a.dtype = x->dtype; a.wdtype = wdtype;
  return launched(launch_norm_backward(a, (cudaStream_t)stream));
}

DA_EXPORT int dow_adamw(const dow_tensor* t, int n, int dtype, int bits, void* m, void* v, float* m_scale, float* v_scale,
                        int64_t state_len, const dow_hyper* h, const float* grad_scale, da_stream_t stream) {
  if (n < 0 || (n > 0 && !t) || !h) return DA_EINVAL;
  if (dtype != DA_F32 && dtype != DA_BF16 && dtype != DA_F16) return DA_EDTYPE;
  if (bits != 32 && bits != 8) return DA_EINVAL;
  if (!(h->beta1 >= 0 && h->beta1 < 1) || !(h->beta2 >= 0 && h->beta2 < 1) || !(h->eps >= 0) || h->step < 1 ||
      !std::isfinite(h->lr) || !std::isfinite(h->weight_decay) || !std::isfinite(h->eps))
    return DA_EINVAL;
  if (state_len < 0 || state_len % ADAMW_BLOCK) return DA_ESHAPE;
  const size_t es = dtype == DA_F32 ? 4 : 2;
  bool some = false;
  for (int i = 0; i < n; i++) {
    if (t[i].numel < 0 || t[i].state < 0 || t[i].state % ADAMW_BLOCK) return DA_ESHAPE;
    if (t[i].numel > state_len || t[i].state > state_len - t[i].numel) return DA_ESHAPE;
    if (t[i].numel / ADAMW_CHUNK >= ((int64_t)1 << 30)) return DA_ESHAPE;
    if (t[i].numel == 0) continue;
    some = true;
    if (!t[i].param || !t[i].grad) return DA_EINVAL;
    if (!aligned(t[i].param, es) || !aligned(t[i].grad, es)) return DA_EALIGN;
  }
  if (!some) return DA_OK;
  if (!m || !v || (bits == 8 && (!m_scale || !v_scale))) return DA_EINVAL;
  if (!aligned(m, 16) || !aligned(v, 16) || !aligned(m_scale, 4) || !aligned(v_scale, 4) || !aligned(grad_scale, 4))
    return DA_EALIGN;
  AdamWArgs a;
  a.m = m; a.v = v; a.m_scale = m_scale; a.v_scale = v_scale; a.grad_scale = grad_scale;
  a.b1 = (float)h->beta1; a.c1 = (float)(1 - h->beta1);
  a.b2 = (float)h->beta2; a.c2 = (float)(1 - h->beta2);
  a.keep = (float)(1 - h->lr * h->weight_decay);
  a.rate = (float)(h->lr / (1 - std::pow(h->beta1, (double)h->step)));
  a.undo = (float)(1 / std::sqrt(1 - std::pow(h->beta2, (double)h->step)));
  a.eps = (float)h->eps;
  a.nt = 0;
  a.first[0] = 0;
  for (int i = 0; i < n; i++) {
    if (t[i].numel == 0) continue;
    const uint32_t chunks = (uint32_t)((t[i].numel + ADAMW_CHUNK - 1) / ADAMW_CHUNK);
    if (a.nt == ADAMW_TABLE || (uint64_t)a.first[a.nt] + chunks > 0x7fffffffu) {
      const int e = launched(launch_adamw(a, dtype, bits, (cudaStream_t)stream));
      if (e) return e;
      a.nt = 0;
    }
    a.t[a.nt] = {t[i].param, t[i].grad, t[i].numel, t[i].state};
    a.first[a.nt + 1] = a.first[a.nt] + chunks;
    a.nt++;
  }
  return launched(launch_adamw(a, dtype, bits, (cudaStream_t)stream));
}

}  // extern "C"
