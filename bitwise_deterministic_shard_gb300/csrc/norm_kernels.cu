// Layer norm, forward and backward, with the reduction of the weight's and bias's gradients.
//
//   mean = sum x / N;  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps);  h = (x - mean) rstd
//   y = h w + b;   a = dy w;   dx = rstd (a - mean(a) - h mean(a h))
//   dw = sum over rows of dy h;   db = sum over rows of dy
//
// What bounds it: HBM (x and y once forward, x, dy and dx once backward).  A row is read once
// and stays in the registers of its group of threads (a warp up to 128 16-byte vectors, else a
// CTA of up to 1024 threads with two vectors each); both statistics come from those
// registers, so the variance is the centred sum, not a difference of sums.  Wider rows are read
// again from L2 by a looping variant.  Rows that do not start on 16 bytes are read element by
// element with the threads of a warp on neighbouring elements (a warp's access is still one run).
// In the backward pass a group keeps its columns over a run of rows, so dw and db are sums in
// its registers; each run writes one row of partial sums and a second kernel adds these in a fixed
// order.  The runs depend on the sizes alone.  All sums are binary32.
#include "../../include/detattn.h"
#include "train_kernels.h"
#include "train_math.cuh"

namespace detattn {
namespace {

constexpr int WARP_ROWS = 4;      // rows (warps) of a CTA of the warp-per-row variants

// element e of vector k of thread t of G: 16-byte vectors, or runs of single elements
template <int G, int VEC, bool AL>
__device__ __forceinline__ int64_t col(int k, int e, int t) {
  return AL ? ((int64_t)k * G + t) * VEC + e : ((int64_t)k * VEC + e) * G + t;
}

// the row's elements of this thread, as packed registers; zero past the end
template <typename T, int G, int NV, bool AL>
struct Row {
  static constexpr int VEC = Elem<T>::VEC;
  Pack<T, VEC> r[NV];
  __device__ __forceinline__ void load(const T* row, int64_t cols, int t) {
#pragma unroll
    for (int k = 0; k < NV; k++) {
      if (AL && col<G, VEC, AL>(k, VEC, t) <= cols) {
        r[k] = *reinterpret_cast<const Pack<T, VEC>*>(row + col<G, VEC, AL>(k, 0, t));
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e++) {
          const int64_t c = col<G, VEC, AL>(k, e, t);
          r[k].e[e] = c < cols ? row[c] : Elem<T>::put(0.f);
        }
      }
    }
  }
  __device__ __forceinline__ float get(int k, int e) const { return Elem<T>::get(r[k].e[e]); }
};

template <typename T, int G, int NV, bool AL>
__device__ __forceinline__ void store_vec(T* row, int64_t cols, int t, int k, const float* v) {
  constexpr int VEC = Elem<T>::VEC;
  if (AL && col<G, VEC, AL>(k, VEC, t) <= cols) {
    Pack<T, VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; e++) r.e[e] = Elem<T>::put(v[e]);
    *reinterpret_cast<Pack<T, VEC>*>(row + col<G, VEC, AL>(k, 0, t)) = r;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e++) {
      const int64_t c = col<G, VEC, AL>(k, e, t);
      if (c < cols) row[c] = Elem<T>::put(v[e]);
    }
  }
}

// weights of the thread's vector k: f32 or the rows' type, ones (or zeros) without a tensor
template <typename T, int G, bool AL>
__device__ __forceinline__ void load_w(const void* w, bool f32, float none, int64_t cols, int t, int k, float* v) {
  constexpr int VEC = Elem<T>::VEC;
  if (!w) {
#pragma unroll
    for (int e = 0; e < VEC; e++) v[e] = none;
    return;
  }
  const int64_t c0 = col<G, VEC, AL>(k, 0, t);
  if (AL && col<G, VEC, AL>(k, VEC, t) <= cols) {
    if (f32) {
#pragma unroll
      for (int q = 0; q < VEC / 4; q++) {
        const float4 f = *reinterpret_cast<const float4*>((const float*)w + c0 + 4 * q);
        v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
      }
    } else {
      const Pack<T, VEC> r = *reinterpret_cast<const Pack<T, VEC>*>((const T*)w + c0);
#pragma unroll
      for (int e = 0; e < VEC; e++) v[e] = Elem<T>::get(r.e[e]);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < VEC; e++) {
    const int64_t c = col<G, VEC, AL>(k, e, t);
    v[e] = c >= cols ? 0.f : f32 ? ((const float*)w)[c] : Elem<T>::get(((const T*)w)[c]);
  }
}

// sum over the group of G threads, the same bits in each
template <int G>
__device__ __forceinline__ float group_sum(float x, float* sh) {
  x = warp_sum(x);
  if constexpr (G > 32) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();                   // the words of the sum before may still be read
    if (lane == 0) sh[w] = x;
    __syncthreads();
    x = warp_sum(lane < G / 32 ? sh[lane] : 0.f);
  }
  return x;
}
// two sums at once
template <int G>
__device__ __forceinline__ void group_sum2(float& x, float& y, float* sh) {
  x = warp_sum(x);
  y = warp_sum(y);
  if constexpr (G > 32) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) {
      sh[w] = x;
      sh[32 + w] = y;
    }
    __syncthreads();
    x = warp_sum(lane < G / 32 ? sh[lane] : 0.f);
    y = warp_sum(lane < G / 32 ? sh[32 + lane] : 0.f);
  }
}

template <typename T, int G, int NV, bool AL>
__global__ void __launch_bounds__(G == 32 ? 32 * WARP_ROWS : G) norm_fwd_kernel(const NormArgs a) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ float sh[64];
  const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = G == 32 ? (int64_t)blockIdx.x * WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
  if (G == 32 && row >= a.rows) return;
  Row<T, G, NV, AL> x;
  x.load((const T*)a.x + row * a.xs, a.cols, t);
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int e = 0; e < VEC; e++) s = __fadd_rn(s, x.get(k, e));
  const float n = (float)a.cols;
  const float mean = __fdiv_rn(group_sum<G>(s, sh), n);
  s = 0.f;
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int e = 0; e < VEC; e++) {
      const float d = col<G, VEC, AL>(k, e, t) < a.cols ? x.get(k, e) - mean : 0.f;
      s = __fmaf_rn(d, d, s);
    }
  const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(group_sum<G>(s, sh), n) + a.eps));
  const bool wf = a.wdtype == DA_F32;
#pragma unroll
  for (int k = 0; k < NV; k++) {
    float w[VEC], b[VEC], y[VEC];
    load_w<T, G, AL>(a.w, wf, 1.f, a.cols, t, k, w);
    load_w<T, G, AL>(a.b, wf, 0.f, a.cols, t, k, b);
#pragma unroll
    for (int e = 0; e < VEC; e++) y[e] = __fmaf_rn((x.get(k, e) - mean) * rstd, w[e], b[e]);
    store_vec<T, G, NV, AL>((T*)a.y + row * a.ys, a.cols, t, k, y);
  }
  if (t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

// rows wider than the registers of a CTA: three passes over the row, the later two from L2
template <typename T>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const NormArgs a) {
  __shared__ float sh[64];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.xs;
  T* y = (T*)a.y + row * a.ys;
  const float n = (float)a.cols;
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < a.cols; c += 1024) s = __fadd_rn(s, Elem<T>::get(x[c]));
  const float mean = __fdiv_rn(group_sum<1024>(s, sh), n);
  s = 0.f;
  for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
    const float d = Elem<T>::get(x[c]) - mean;
    s = __fmaf_rn(d, d, s);
  }
  const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(group_sum<1024>(s, sh), n) + a.eps));
  const bool wf = a.wdtype == DA_F32;
  for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
    const float w = !a.w ? 1.f : wf ? ((const float*)a.w)[c] : Elem<T>::get(((const T*)a.w)[c]);
    const float b = !a.b ? 0.f : wf ? ((const float*)a.b)[c] : Elem<T>::get(((const T*)a.b)[c]);
    y[c] = Elem<T>::put(__fmaf_rn((Elem<T>::get(x[c]) - mean) * rstd, w, b));
  }
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

// One CTA takes the rows [part * per, ...); in the warp variants its warps take every fourth.
template <typename T, int G, int NV, bool AL>
__global__ void __launch_bounds__(G == 32 ? 32 * WARP_ROWS : G) norm_bwd_kernel(const NormArgs a, int64_t per) {
  constexpr int VEC = Elem<T>::VEC;
  constexpr int STEP = G == 32 ? WARP_ROWS : 1;
  __shared__ float sh[G == 32 ? 32 * NV * VEC * 2 : 64];
  const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.x * per, r1 = min(r0 + per, a.rows);
  const float inv_n = __fdiv_rn(1.f, (float)a.cols);
  const bool wf = a.wdtype == DA_F32;
  float gw[NV][VEC], gb[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int e = 0; e < VEC; e++) gw[k][e] = gb[k][e] = 0.f;
  for (int64_t row = r0 + (G == 32 ? threadIdx.x >> 5 : 0); row < r1; row += STEP) {
    Row<T, G, NV, AL> x, dy;
    x.load((const T*)a.x + row * a.xs, a.cols, t);
    dy.load((const T*)a.dy + row * a.dys, a.cols, t);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; k++) {
      float w[VEC];
      load_w<T, G, AL>(a.w, wf, 1.f, a.cols, t, k, w);
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        const float d = dy.get(k, e), h = (x.get(k, e) - mean) * rstd, ad = d * w[e];
        gw[k][e] = __fmaf_rn(d, h, gw[k][e]);   // past the row's end d is zero
        gb[k][e] = __fadd_rn(gb[k][e], d);
        s1 = __fadd_rn(s1, ad);
        s2 = __fmaf_rn(ad, h, s2);
      }
    }
    group_sum2<G>(s1, s2, sh);
    s1 *= inv_n;
    s2 *= inv_n;
#pragma unroll
    for (int k = 0; k < NV; k++) {
      float w[VEC], dx[VEC];
      load_w<T, G, AL>(a.w, wf, 1.f, a.cols, t, k, w);
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        const float h = (x.get(k, e) - mean) * rstd;
        dx[e] = __fmaf_rn(-h, s2, __fmaf_rn(dy.get(k, e), w[e], -s1)) * rstd;
      }
      store_vec<T, G, NV, AL>((T*)a.y + row * a.ys, a.cols, t, k, dx);
    }
  }
  if (!a.part) return;
  if constexpr (G == 32) {   // the warps' sums in the order of the warps
    const int w = threadIdx.x >> 5;
    for (int turn = 0; turn < WARP_ROWS; turn++) {
      if (w == turn) {
#pragma unroll
        for (int k = 0; k < NV; k++)
#pragma unroll
          for (int e = 0; e < VEC; e++) {
            float* at = sh + (k * VEC + e) * 64 + t;
            if (turn) {
              gw[k][e] = __fadd_rn(at[0], gw[k][e]);
              gb[k][e] = __fadd_rn(at[32], gb[k][e]);
            }
            at[0] = gw[k][e];
            at[32] = gb[k][e];
          }
      }
      __syncthreads();
    }
    if (w != WARP_ROWS - 1) return;
  }
  float* pw = a.part + (int64_t)blockIdx.x * a.cols;
  float* pb = pw + (int64_t)gridDim.x * a.cols;
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int e = 0; e < VEC; e++) {
      const int64_t c = col<G, VEC, AL>(k, e, t);
      if (c < a.cols) {
        pw[c] = gw[k][e];
        pb[c] = gb[k][e];
      }
    }
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const NormArgs a, int64_t per) {
  __shared__ float sh[64];
  const int64_t r0 = (int64_t)blockIdx.x * per, r1 = min(r0 + per, a.rows);
  const float inv_n = __fdiv_rn(1.f, (float)a.cols);
  const bool wf = a.wdtype == DA_F32;
  float* pw = a.part + (int64_t)blockIdx.x * a.cols;
  float* pb = a.part + ((int64_t)gridDim.x + blockIdx.x) * a.cols;
  for (int64_t row = r0; row < r1; row++) {
    const T* x = (const T*)a.x + row * a.xs;
    const T* dy = (const T*)a.dy + row * a.dys;
    T* dx = (T*)a.y + row * a.ys;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float w = !a.w ? 1.f : wf ? ((const float*)a.w)[c] : Elem<T>::get(((const T*)a.w)[c]);
      const float d = Elem<T>::get(dy[c]), h = (Elem<T>::get(x[c]) - mean) * rstd;
      s1 = __fadd_rn(s1, d * w);
      s2 = __fmaf_rn(d * w, h, s2);
      if (a.part) {          // this CTA's own words: the columns of a thread stay its own
        pw[c] = __fmaf_rn(d, h, row == r0 ? 0.f : pw[c]);
        pb[c] = __fadd_rn(d, row == r0 ? 0.f : pb[c]);
      }
    }
    group_sum2<1024>(s1, s2, sh);
    s1 *= inv_n;
    s2 *= inv_n;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float w = !a.w ? 1.f : wf ? ((const float*)a.w)[c] : Elem<T>::get(((const T*)a.w)[c]);
      const float h = (Elem<T>::get(x[c]) - mean) * rstd;
      dx[c] = Elem<T>::put(__fmaf_rn(-h, s2, __fmaf_rn(Elem<T>::get(dy[c]), w, -s1)) * rstd);
    }
  }
}

// dw and db from the partial rows: 32 columns a CTA, 32 warps over the rows, then the warps' sums
// in their order.  blockIdx.y: 0 dw, 1 db.
template <typename W>
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float* part, int64_t nparts, int64_t cols, W* dw, W* db) {
  __shared__ float sh[32][33];
  W* out = blockIdx.y ? db : dw;
  if (!out) return;
  const float* p = part + (blockIdx.y ? nparts * cols : 0);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = w; r < nparts; r += 32) s = __fadd_rn(s, p[r * cols + c]);
  }
  sh[w][lane] = s;
  __syncthreads();
  s = warp_sum(sh[lane][w]);           // column w of this CTA
  const int64_t cc = (int64_t)blockIdx.x * 32 + w;
  if (lane == 0 && cc < cols) out[cc] = Elem<W>::put(s);
}

bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, int G, int NV>
void fwd_go(const NormArgs& a, bool al, cudaStream_t st) {
  const unsigned grid = (unsigned)(G == 32 ? (a.rows + WARP_ROWS - 1) / WARP_ROWS : a.rows);
  const int threads = G == 32 ? 32 * WARP_ROWS : G;
  if (al) norm_fwd_kernel<T, G, NV, true><<<grid, threads, 0, st>>>(a);
  else norm_fwd_kernel<T, G, NV, false><<<grid, threads, 0, st>>>(a);
}
template <typename T, int G, int NV>
void bwd_go(const NormArgs& a, bool al, unsigned grid, int64_t per, cudaStream_t st) {
  const int threads = G == 32 ? 32 * WARP_ROWS : G;
  if (al) norm_bwd_kernel<T, G, NV, true><<<grid, threads, 0, st>>>(a, per);
  else norm_bwd_kernel<T, G, NV, false><<<grid, threads, 0, st>>>(a, per);
}

template <typename T>
void fwd(const NormArgs& a, cudaStream_t st) {
  constexpr int VEC = Elem<T>::VEC;
  const bool al = al16(a.x) && al16(a.y) && a.xs % VEC == 0 && a.ys % VEC == 0 && al16(a.w) && al16(a.b);
  const int64_t nv = (a.cols + VEC - 1) / VEC;
  if (nv <= 32) fwd_go<T, 32, 1>(a, al, st);
  else if (nv <= 128) fwd_go<T, 32, 4>(a, al, st);
  else if (nv <= 256) fwd_go<T, 128, 2>(a, al, st);
  else if (nv <= 512) fwd_go<T, 256, 2>(a, al, st);
  else if (nv <= 1024) fwd_go<T, 512, 2>(a, al, st);
  else if (nv <= 2048) fwd_go<T, 1024, 2>(a, al, st);
  else norm_fwd_wide_kernel<T><<<(unsigned)a.rows, 1024, 0, st>>>(a);
}
template <typename T>
void bwd(const NormArgs& a, unsigned grid, int64_t per, cudaStream_t st) {
  constexpr int VEC = Elem<T>::VEC;
  const bool al = al16(a.x) && al16(a.y) && al16(a.dy) && a.xs % VEC == 0 && a.ys % VEC == 0 && a.dys % VEC == 0 && al16(a.w);
  const int64_t nv = (a.cols + VEC - 1) / VEC;
  if (nv <= 32) bwd_go<T, 32, 1>(a, al, grid, per, st);
  else if (nv <= 128) bwd_go<T, 32, 4>(a, al, grid, per, st);
  else if (nv <= 256) bwd_go<T, 128, 2>(a, al, grid, per, st);
  else if (nv <= 512) bwd_go<T, 256, 2>(a, al, grid, per, st);
  else if (nv <= 1024) bwd_go<T, 512, 2>(a, al, grid, per, st);
  else if (nv <= 2048) bwd_go<T, 1024, 2>(a, al, grid, per, st);
  else norm_bwd_wide_kernel<T><<<grid, 1024, 0, st>>>(a, per);
}

int64_t rows_per(int64_t rows, int64_t cols) {
  // about two resident CTAs (eight of the warp variants) on each of 152 SMs; a run has at least
  // as many rows as the CTA has warps that share them
  const bool narrow = cols <= 1024;
  const int64_t want = narrow ? 152 * 8 : 152 * 2;
  const int64_t per = (rows + want - 1) / want;
  return narrow ? (per + WARP_ROWS - 1) / WARP_ROWS * WARP_ROWS : per < 1 ? 1 : per;
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols) {
  if (rows <= 0) return 0;
  const int64_t per = rows_per(rows, cols);
  return (rows + per - 1) / per;
}

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t st) {
  if (a.dtype == DA_F32) fwd<float>(a, st);
  else if (a.dtype == DA_BF16) fwd<__nv_bfloat16>(a, st);
  else fwd<__half>(a, st);
  return cudaGetLastError();
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t st) {
  const int64_t n = norm_parts(a.rows, a.cols);
  if (n > 0) {
    const int64_t per = rows_per(a.rows, a.cols);
    if (a.dtype == DA_F32) bwd<float>(a, (unsigned)n, per, st);
    else if (a.dtype == DA_BF16) bwd<__nv_bfloat16>(a, (unsigned)n, per, st);
    else bwd<__half>(a, (unsigned)n, per, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.dw || a.db) {
    const dim3 grid((unsigned)((a.cols + 31) / 32), 2);
    if (a.wdtype == DA_F32) norm_sum_kernel<float><<<grid, 1024, 0, st>>>(a.part, n, a.cols, (float*)a.dw, (float*)a.db);
    else if (a.wdtype == DA_BF16) norm_sum_kernel<__nv_bfloat16><<<grid, 1024, 0, st>>>(a.part, n, a.cols, (__nv_bfloat16*)a.dw, (__nv_bfloat16*)a.db);
    else norm_sum_kernel<__half><<<grid, 1024, 0, st>>>(a.part, n, a.cols, (__half*)a.dw, (__half*)a.db);
  }
  return cudaGetLastError();
}

}  // namespace detattn
