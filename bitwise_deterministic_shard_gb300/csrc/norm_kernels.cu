// Layer norm, forward and backward, with the reduction of the weight's and bias's gradients.
//
//   mean = sum x / N;  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps);  h = (x - mean) rstd
//   y = h w + b;   a = dy w;   dx = rstd (a - mean(a) - h mean(a h))
//   dw = sum over rows of dy h;   db = sum over rows of dy
//
// What bounds it: HBM (x and y once forward, x, dy and dx once backward).  A row is read once: it stays in the
// registers, or the shared memory, of its warp or CTA, and both statistics come from there, so the
// variance is the centred sum, not a difference of sums.  Variants, by the 16-byte vectors of a row:
//   aligned, 129 to 1024 vectors, many rows: streaming CTAs (below) that copy the next rows while they work
//     on the present ones and keep the weights in registers;
//   not aligned, more than 128 vectors up to 8192 columns: staged CTAs (below), except f32 forward;
//   otherwise, up to 128 vectors: a warp a row; up to 2048: a CTA a row (forward) or a run of rows (backward),
//     rows that do not start and end on 16 bytes element by element, the threads of a warp on
//     neighbouring elements (a warp's access is still one run);
//   wider rows are read again from L2 by looping variants.
// In the backward pass a group of threads keeps its columns over a run of rows, so dw and db are sums in
// its registers; each run writes one row of partial sums and a second kernel adds these in a fixed order.
// The runs depend on the sizes alone.  All sums are binary32; pairs of elements go through the packed
// multiplier and adder.
// 8192 x 4096 bf16, f32 weights: forward 30 us (0.65 of the measured copy bandwidth; 46 with a CTA a row that
// reads the weights again for each, 49 with a warp a row), backward 48 us with the sum of the partial rows
// (0.62; 79 + 5 and 59 so).  3001 x 5003 f32, unaligned: 27 and 45 us (0.66, 0.59).
#include <algorithm>

#include "../../include/detattn.h"
#include "device_once.h"
#include "train_kernels.h"
#include "train_math.cuh"

namespace detattn {
namespace {

using f2::u64;

constexpr int WARP_ROWS = 4;      // rows (warps) of a CTA of the warp-per-row variants

// element e of vector k of thread t of G: 16-byte vectors, or runs of single elements
template <int G, int VEC, bool AL>
__device__ __forceinline__ int col(int k, int e, int t) {   // rows of the register variants have under 2^15 columns
  return AL ? (k * G + t) * VEC + e : (k * VEC + e) * G + t;
}

// the row's elements of this thread, as 32-bit words; zero past the end
template <typename T, int G, int NV, bool AL>
struct Row {
  static constexpr int VEC = Elem<T>::VEC;
  Run<T, VEC> r[NV];
  __device__ __forceinline__ void load(const T* row, int cols, int t) {
#pragma unroll
    for (int k = 0; k < NV; k++) {
      r[k].zero();
      if constexpr (AL) {
        if (col<G, VEC, AL>(k, 0, t) < cols) r[k].load(row + col<G, VEC, AL>(k, 0, t));
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e++) {
          const int c = col<G, VEC, AL>(k, e, t);
          if (c < cols) r[k].put_bits(e, row[c]);
        }
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < NV; k++) r[k].zero();
  }
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int k = 0; k < NV; k++) r[k].keep();
  }
  __device__ __forceinline__ u64 get2(int k, int i) const { return r[k].get2(i); }
};

template <typename T, int G, bool AL>
__device__ __forceinline__ void store_vec(T* row, int cols, int t, int k, const Run<T, Elem<T>::VEC>& r) {
  constexpr int VEC = Elem<T>::VEC;
  if constexpr (AL) {
    if (col<G, VEC, AL>(k, 0, t) < cols) r.store(row + col<G, VEC, AL>(k, 0, t));
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e++) {
      const int c = col<G, VEC, AL>(k, e, t);
      if (c < cols) row[c] = r.bits(e);
    }
  }
}

// weights of the thread's vector k: f32 or the rows' type, ones (or zeros) without a tensor
template <typename T, int G, bool AL>
__device__ __forceinline__ void load_w(const void* w, bool f32, float none, int cols, int t, int k, u64 (&v)[Elem<T>::VEC / 2]) {
  constexpr int VEC = Elem<T>::VEC;
  if (!w) {
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) v[i] = f2::splat(none);
    return;
  }
  const int c0 = col<G, VEC, AL>(k, 0, t);
  if constexpr (AL) {
    if (c0 >= cols) {
#pragma unroll
      for (int i = 0; i < VEC / 2; i++) v[i] = 0;
    } else if (f32) {
#pragma unroll
      for (int q = 0; q < VEC / 4; q++) {
        const float4 f = *reinterpret_cast<const float4*>((const float*)w + c0 + 4 * q);
        v[2 * q] = f2::pack(f.x, f.y);
        v[2 * q + 1] = f2::pack(f.z, f.w);
      }
    } else {
      Run<T, VEC> r;
      r.load((const T*)w + c0);
#pragma unroll
      for (int i = 0; i < VEC / 2; i++) v[i] = r.get2(i);
    }
  } else {
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e++) {
      const int c = col<G, VEC, AL>(k, e, t);
      f[e] = c >= cols ? 0.f : f32 ? ((const float*)w)[c] : Elem<T>::get(((const T*)w)[c]);
    }
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) v[i] = f2::pack(f[2 * i], f[2 * i + 1]);
  }
}
__device__ __forceinline__ float both(u64 v) {
  float a, b;
  f2::unpack(v, a, b);
  return __fadd_rn(a, b);
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

// CTAs of an SM that the registers have to allow: enough loads in flight, but the row stays in registers
constexpr int fwd_ctas(int g) { return g == 32 ? 8 : g == 128 ? 10 : 4; }
constexpr int bwd_ctas(int g, int nv) { return g == 32 ? nv == 1 ? 8 : 4 : g == 128 ? 4 : g == 256 ? 2 : 1; }

template <typename T, int G, int NV, bool AL>
__global__ void __launch_bounds__(G == 32 ? 32 * WARP_ROWS : G, fwd_ctas(G)) norm_fwd_kernel(const NormArgs a) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ float sh[64];
  const int cols = (int)a.cols;
  const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = G == 32 ? (int64_t)blockIdx.x * WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
  if (G == 32 && row >= a.rows) return;
  Row<T, G, NV, AL> x;
  x.load((const T*)a.x + row * a.xs, cols, t);
  u64 s = 0;
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) s = f2::add(s, x.get2(k, i));
  const float n = (float)a.cols;
  const float mean = __fdiv_rn(group_sum<G>(both(s), sh), n);
  x.keep();
  s = 0;
  const u64 off = f2::splat(-mean);
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) {
      u64 d = f2::add(x.get2(k, i), off);
      if (AL) {
        if (col<G, VEC, AL>(k, 0, t) >= cols) d = 0;
      } else {
        float p, q;
        f2::unpack(d, p, q);
        d = f2::pack(col<G, VEC, AL>(k, 2 * i, t) < cols ? p : 0.f, col<G, VEC, AL>(k, 2 * i + 1, t) < cols ? q : 0.f);
      }
      s = f2::fma(d, d, s);
    }
  const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(group_sum<G>(both(s), sh), n) + a.eps));
  const u64 rstd2 = f2::splat(rstd);
  const bool wf = a.wdtype == DA_F32;
  x.keep();
#pragma unroll
  for (int k = 0; k < NV; k++) {
    u64 w[VEC / 2], b[VEC / 2];
    load_w<T, G, AL>(a.w, wf, 1.f, cols, t, k, w);
    load_w<T, G, AL>(a.b, wf, 0.f, cols, t, k, b);
    Run<T, VEC> y;
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) y.set2(i, f2::fma(f2::mul(f2::add(x.get2(k, i), off), rstd2), w[i], b[i]));
    store_vec<T, G, AL>((T*)a.y + row * a.ys, cols, t, k, y);
  }
  if (t == 0 && a.mean) {
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
  if (threadIdx.x == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

// One CTA takes the rows [part * per, ...), R at a time; in the warp variants each warp takes every
// fourth group of R.
template <typename T, int G, int NV, int R, bool AL>
__global__ void __launch_bounds__(G == 32 ? 32 * WARP_ROWS : G, bwd_ctas(G, NV)) norm_bwd_kernel(const NormArgs a, int64_t per) {
  constexpr int VEC = Elem<T>::VEC, W = G / 32;
  const int cols = (int)a.cols;
  constexpr int STEP = G == 32 ? WARP_ROWS * R : R;
  __shared__ __align__(8) float sh[G == 32 ? 32 * NV * VEC * 2 : 4 * R * W];
  const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r0 = (int64_t)blockIdx.x * per, r1 = min(r0 + per, a.rows);
  const float inv_n = __fdiv_rn(1.f, (float)a.cols);
  const bool wf = a.wdtype == DA_F32;
  u64 gw[NV][VEC / 2], gb[NV][VEC / 2];
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) gw[k][i] = gb[k][i] = 0;
  Row<T, G, NV, AL> x[R], dy[R];
  float mean[R], rstd[R];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; r++) {
      if (row + r < r1) {
        x[r].load((const T*)a.x + (row + r) * a.xs, cols, t);
        dy[r].load((const T*)a.dy + (row + r) * a.dys, cols, t);
        mean[r] = a.mean[row + r];
        rstd[r] = a.rstd[row + r];
      } else {                       // no row: adds nothing
        x[r].zero();
        dy[r].zero();
        mean[r] = rstd[r] = 0.f;
      }
    }
  };
  int turn = 0;
  for (int64_t row = r0 + (G == 32 ? warp * R : 0); row < r1; row += STEP, turn ^= 1) {
    fetch(row);
    u64 t1[R], t2[R];
#pragma unroll
    for (int r = 0; r < R; r++) t1[r] = t2[r] = 0;
#pragma unroll
    for (int k = 0; k < NV; k++) {
      u64 w[VEC / 2];
      load_w<T, G, AL>(a.w, wf, 1.f, cols, t, k, w);
#pragma unroll
      for (int r = 0; r < R; r++)
#pragma unroll
        for (int i = 0; i < VEC / 2; i++) {
          const u64 d = dy[r].get2(k, i), h = f2::mul(f2::add(x[r].get2(k, i), f2::splat(-mean[r])), f2::splat(rstd[r]));
          const u64 ad = f2::mul(d, w[i]);
          gw[k][i] = f2::fma(d, h, gw[k][i]);   // past the row's end d is zero
          gb[k][i] = f2::add(gb[k][i], d);
          t1[r] = f2::add(t1[r], ad);
          t2[r] = f2::fma(ad, h, t2[r]);
        }
    }
    float s1[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      s1[r] = warp_sum(both(t1[r]));
      s2[r] = warp_sum(both(t2[r]));
    }
    if constexpr (G > 32) {          // two sets of words by turns: one barrier a step
      float* at = sh + turn * (2 * R * W);
      if (lane == 0) {
#pragma unroll
        for (int r = 0; r < R; r++) {
          at[(2 * r) * W + warp] = s1[r];
          at[(2 * r + 1) * W + warp] = s2[r];
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; r++) {
        s1[r] = warp_sum(lane < W ? at[(2 * r) * W + lane] : 0.f);
        s2[r] = warp_sum(lane < W ? at[(2 * r + 1) * W + lane] : 0.f);
      }
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
      x[r].keep();
      dy[r].keep();
    }
#pragma unroll
    for (int k = 0; k < NV; k++) {
      u64 w[VEC / 2];
      load_w<T, G, AL>(a.w, wf, 1.f, cols, t, k, w);
#pragma unroll
      for (int r = 0; r < R; r++) {
        const u64 m1 = f2::splat(-s1[r] * inv_n), m2 = f2::splat(-s2[r] * inv_n), rr = f2::splat(rstd[r]);
        Run<T, VEC> dx;
#pragma unroll
        for (int i = 0; i < VEC / 2; i++) {
          const u64 h = f2::mul(f2::add(x[r].get2(k, i), f2::splat(-mean[r])), rr);
          dx.set2(i, f2::mul(f2::fma(h, m2, f2::fma(dy[r].get2(k, i), w[i], m1)), rr));
        }
        if (row + r < r1) store_vec<T, G, AL>((T*)a.y + (row + r) * a.ys, cols, t, k, dx);
      }
    }
  }
  if (!a.part) return;
  if constexpr (G == 32) {   // the warps' sums in the order of the warps
    u64* at = reinterpret_cast<u64*>(sh) + t;
    for (int turn = 0; turn < WARP_ROWS; turn++) {
      if (warp == turn) {
#pragma unroll
        for (int k = 0; k < NV; k++)
#pragma unroll
          for (int i = 0; i < VEC / 2; i++) {
            const int o = (k * VEC / 2 + i) * 64;
            if (turn) {
              gw[k][i] = f2::add(at[o], gw[k][i]);
              gb[k][i] = f2::add(at[o + 32], gb[k][i]);
            }
            at[o] = gw[k][i];
            at[o + 32] = gb[k][i];
          }
      }
      __syncthreads();
    }
    if (warp != WARP_ROWS - 1) return;
  }
  float* pw = a.part + (int64_t)blockIdx.x * a.cols;
  float* pb = pw + (int64_t)gridDim.x * a.cols;
#pragma unroll
  for (int k = 0; k < NV; k++)
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) {
      float w0, w1, b0, b1;
      f2::unpack(gw[k][i], w0, w1);
      f2::unpack(gb[k][i], b0, b1);
      const int c0 = col<G, VEC, AL>(k, 2 * i, t), c1 = col<G, VEC, AL>(k, 2 * i + 1, t);
      if (c0 < cols) {
        pw[c0] = w0;
        pb[c0] = b0;
      }
      if (c1 < cols) {
        pw[c1] = w1;
        pb[c1] = b1;
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

// ---- streaming variants: aligned rows of more than 128 vectors ----
//
// A CTA stays for a run of rows (backward) or every gridDim-th group of rows (forward).  Each thread owns
// NV 16-byte vectors of the columns, keeps their weights in registers, and copies its own parts of the
// next rows into its own slots of shared memory (cp.async: no register holds a load in flight, and no
// barrier is needed for data that only the copying thread reads).  R rows share the barriers of a step.

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {   // zeros where there is no row or column
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
__device__ __forceinline__ Run<T, Elem<T>::VEC> slot(uint32_t at) {
  Run<T, Elem<T>::VEC> r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(at));
  return r;
}

// N sums at once over the CTA of G threads, by turns in two sets of words: one barrier
template <int G, int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float* sh, int turn) {
  constexpr int W = G / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* at = sh + turn * (N * W);
#pragma unroll
  for (int i = 0; i < N; i++) {
    v[i] = warp_sum(v[i]);
    if (lane == 0) at[i * W + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; i++) {
    float x = lane < W ? at[i * W + lane] : 0.f;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
    v[i] = __shfl_sync(0xffffffffu, x, 0);
  }
}

template <typename T, int G, int NV, int R, int ST>
__global__ void __launch_bounds__(G, 512 / G) norm_fwd_stream_kernel(const NormArgs a) {
  constexpr int VEC = Elem<T>::VEC, W = G / 32;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float sh[2 * R * W];
  const int cols = (int)a.cols, t = threadIdx.x;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + t * 16;
  const bool wf = a.wdtype == DA_F32;
  u64 w[NV][VEC / 2], b[NV][VEC / 2];
#pragma unroll
  for (int k = 0; k < NV; k++) {
    load_w<T, G, true>(a.w, wf, 1.f, cols, t, k, w[k]);
    load_w<T, G, true>(a.b, wf, 0.f, cols, t, k, b[k]);
  }
  const auto fetch = [&](int64_t row, int st) {
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int k = 0; k < NV; k++) {
        const int c = col<G, VEC, true>(k, 0, t);
        const bool real = row + r < a.rows && c < cols;
        copy16(mine + ((st * R + r) * NV + k) * (G * 16), (const T*)a.x + (real ? (row + r) * a.xs + c : 0), real);
      }
    copy_commit();
  };
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t row = (int64_t)blockIdx.x * R;
#pragma unroll
  for (int s = 0; s < ST - 1; s++) fetch(row + s * step, s);
  const float n = (float)a.cols;
  int st = 0, turn = 0;
  for (; row < a.rows; row += step) {
    fetch(row + (ST - 1) * step, st == 0 ? ST - 1 : st - 1);
    copy_wait<ST - 1>();
    const uint32_t at = mine + st * R * NV * (G * 16);
    float v[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      u64 s = 0;
#pragma unroll
      for (int k = 0; k < NV; k++) {
        const auto x = slot<T>(at + (r * NV + k) * (G * 16));
#pragma unroll
        for (int i = 0; i < VEC / 2; i++) s = f2::add(s, x.get2(i));
      }
      v[r] = both(s);
    }
    cta_sums<G, R>(v, sh, turn);
    turn ^= 1;
    float mean[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      mean[r] = __fdiv_rn(v[r], n);
      u64 s = 0;
#pragma unroll
      for (int k = 0; k < NV; k++) {
        const auto x = slot<T>(at + (r * NV + k) * (G * 16));
        if (col<G, VEC, true>(k, 0, t) < cols) {
#pragma unroll
          for (int i = 0; i < VEC / 2; i++) {
            const u64 d = f2::add(x.get2(i), f2::splat(-mean[r]));
            s = f2::fma(d, d, s);
          }
        }
      }
      v[r] = both(s);
    }
    cta_sums<G, R>(v, sh, turn);
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < R; r++) {
      const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(v[r], n) + a.eps));
      if (row + r < a.rows) {
#pragma unroll
        for (int k = 0; k < NV; k++) {
          const auto x = slot<T>(at + (r * NV + k) * (G * 16));
          Run<T, VEC> y;
#pragma unroll
          for (int i = 0; i < VEC / 2; i++)
            y.set2(i, f2::fma(f2::mul(f2::add(x.get2(i), f2::splat(-mean[r])), f2::splat(rstd)), w[k][i], b[k][i]));
          store_vec<T, G, true>((T*)a.y + (row + r) * a.ys, cols, t, k, y);
        }
        if (t == 0 && a.mean) {
          a.mean[row + r] = mean[r];
          a.rstd[row + r] = rstd;
        }
      }
    }
    st = st == ST - 1 ? 0 : st + 1;
  }
}

template <typename T, int G, int NV, int R, int ST>
__global__ void __launch_bounds__(G, 512 / G) norm_bwd_stream_kernel(const NormArgs a, int64_t per) {
  constexpr int VEC = Elem<T>::VEC, W = G / 32;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float sh[4 * R * W];
  const int cols = (int)a.cols, t = threadIdx.x;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + t * 16;
  const bool wf = a.wdtype == DA_F32;
  const int64_t r0 = (int64_t)blockIdx.x * per, r1 = min(r0 + per, a.rows);
  const float inv_n = __fdiv_rn(1.f, (float)a.cols);
  u64 w[NV][VEC / 2], gw[NV][VEC / 2], gb[NV][VEC / 2];
#pragma unroll
  for (int k = 0; k < NV; k++) {
    load_w<T, G, true>(a.w, wf, 1.f, cols, t, k, w[k]);
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) gw[k][i] = gb[k][i] = 0;
  }
  const auto fetch = [&](int64_t row, int st) {
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int k = 0; k < NV; k++) {
        const int c = col<G, VEC, true>(k, 0, t);
        const bool real = row + r < r1 && c < cols;
        const uint32_t at = mine + ((st * R + r) * NV + k) * (G * 32);
        copy16(at, (const T*)a.x + (real ? (row + r) * a.xs + c : 0), real);
        copy16(at + G * 16, (const T*)a.dy + (real ? (row + r) * a.dys + c : 0), real);
      }
    copy_commit();
  };
  float mean[R], rstd[R], nmean[R], nrstd[R];
  const auto stats = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; r++) {
      nmean[r] = row + r < r1 ? a.mean[row + r] : 0.f;
      nrstd[r] = row + r < r1 ? a.rstd[row + r] : 0.f;
    }
  };
#pragma unroll
  for (int s = 0; s < ST - 1; s++) fetch(r0 + s * R, s);
  stats(r0);
  int st = 0, turn = 0;
  for (int64_t row = r0; row < r1; row += R) {
    fetch(row + (ST - 1) * R, st == 0 ? ST - 1 : st - 1);
#pragma unroll
    for (int r = 0; r < R; r++) {
      mean[r] = nmean[r];
      rstd[r] = nrstd[r];
    }
    stats(row + R);
    copy_wait<ST - 1>();
    const uint32_t at = mine + st * R * NV * (G * 32);
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; r++) {
      u64 t1 = 0, t2 = 0;
#pragma unroll
      for (int k = 0; k < NV; k++) {
        const auto x = slot<T>(at + (r * NV + k) * (G * 32)), dy = slot<T>(at + (r * NV + k) * (G * 32) + G * 16);
#pragma unroll
        for (int i = 0; i < VEC / 2; i++) {
          const u64 d = dy.get2(i), h = f2::mul(f2::add(x.get2(i), f2::splat(-mean[r])), f2::splat(rstd[r]));
          const u64 ad = f2::mul(d, w[k][i]);
          gw[k][i] = f2::fma(d, h, gw[k][i]);
          gb[k][i] = f2::add(gb[k][i], d);
          t1 = f2::add(t1, ad);
          t2 = f2::fma(ad, h, t2);
        }
      }
      s[2 * r] = both(t1);
      s[2 * r + 1] = both(t2);
    }
    cta_sums<G, 2 * R>(s, sh, turn);
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < R; r++) {
      const u64 m1 = f2::splat(-s[2 * r] * inv_n), m2 = f2::splat(-s[2 * r + 1] * inv_n), rr = f2::splat(rstd[r]);
      if (row + r < r1) {
#pragma unroll
        for (int k = 0; k < NV; k++) {
          const auto x = slot<T>(at + (r * NV + k) * (G * 32)), dy = slot<T>(at + (r * NV + k) * (G * 32) + G * 16);
          Run<T, VEC> dx;
#pragma unroll
          for (int i = 0; i < VEC / 2; i++) {
            const u64 h = f2::mul(f2::add(x.get2(i), f2::splat(-mean[r])), rr);
            dx.set2(i, f2::mul(f2::fma(h, m2, f2::fma(dy.get2(i), w[k][i], m1)), rr));
          }
          store_vec<T, G, true>((T*)a.y + (row + r) * a.ys, cols, t, k, dx);
        }
      }
    }
    st = st == ST - 1 ? 0 : st + 1;
  }
  if (!a.part) return;
  float* pw = a.part + (int64_t)blockIdx.x * a.cols;
  float* pb = pw + (int64_t)gridDim.x * a.cols;
#pragma unroll
  for (int k = 0; k < NV; k++) {
    const int c = col<G, VEC, true>(k, 0, t);
    if (c < cols) {
#pragma unroll
      for (int i = 0; i < VEC / 2; i++) {
        float p, q;
        f2::unpack(gw[k][i], p, q);
        pw[c + 2 * i] = p;
        pw[c + 2 * i + 1] = q;
        f2::unpack(gb[k][i], p, q);
        pb[c + 2 * i] = p;
        pb[c + 2 * i + 1] = q;
      }
    }
  }
}

// ---- staged variants: rows that do not start and end on 16 bytes, of more than 128 vectors up to 8192 columns ----
//
// The 16-byte units that hold a row (a few bytes of its neighbour before it; cut at its end) are copied to shared
// memory, from where the threads read their own columns element by element, t + j G of thread t: every
// global read stays 16 bytes wide and is in flight without a register.  Otherwise as the streaming variants.
// Against the variants that read single elements: 8192 x 4097 bf16 forward 80 -> 68 us, backward 128 -> 90;
// 3001 x 5003 f32 backward 54 -> 45; 20000 x 1501 bf16 53 -> 43 and 121 -> 72; what bounds 16-bit rows now is the
// single-element shared-memory reads and stores.

// copies the row of `cols` elements at p to the buffer at `to`; the row starts p % 16 bytes into it
template <typename T, int G>
__device__ __forceinline__ void stage_row(uint32_t to, const T* p, int cols) {
  const uintptr_t at = (uintptr_t)p;
  const int off = (int)(at & 15), bytes = off + cols * (int)sizeof(T);
  const char* from = (const char*)(at - off);
  for (int c = threadIdx.x * 16; c < bytes; c += G * 16) {
    const int left = bytes - c;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + c), "l"(from + c), "r"(left < 16 ? left : 16) : "memory");
  }
}
template <typename T>
__device__ __forceinline__ float staged(uint32_t at) {
  if constexpr (sizeof(T) == 4) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
  } else {
    uint16_t b;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(at));
    return Elem<T>::get(*reinterpret_cast<const T*>(&b));
  }
}
// elements j and j + 1 of the thread, zero past the end
template <typename T, int G>
__device__ __forceinline__ u64 staged2(uint32_t row, int j, int cols) {
  const int c = threadIdx.x + j * G;
  return f2::pack(c < cols ? staged<T>(row + c * (int)sizeof(T)) : 0.f,
                  c + G < cols ? staged<T>(row + (c + G) * (int)sizeof(T)) : 0.f);
}
template <typename T, int G>
__device__ __forceinline__ void put2(T* row, int j, int cols, u64 v) {
  float a, b;
  f2::unpack(v, a, b);
  const int c = threadIdx.x + j * G;
  if (c < cols) row[c] = Elem<T>::put(a);
  if (c + G < cols) row[c + G] = Elem<T>::put(b);
}
template <typename T, int G>
__device__ __forceinline__ u64 weight2(const void* w, bool f32, float none, int j, int cols) {
  const int c = threadIdx.x + j * G;
  const auto one = [&](int k) { return k >= cols ? 0.f : f32 ? ((const float*)w)[k] : Elem<T>::get(((const T*)w)[k]); };
  return w ? f2::pack(one(c), one(c + G)) : f2::splat(none);
}

template <typename T, int G, int NJ>
__global__ void __launch_bounds__(G, 1024 / G) norm_fwd_staged_kernel(const NormArgs a, int room) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float sh[2 * (G / 32)];
  const int cols = (int)a.cols, t = threadIdx.x;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  const bool wf = a.wdtype == DA_F32;
  const float n = (float)a.cols;
  u64 w[NJ / 2], b[NJ / 2];
#pragma unroll
  for (int j = 0; j < NJ; j += 2) {
    w[j / 2] = weight2<T, G>(a.w, wf, 1.f, j, cols);
    b[j / 2] = weight2<T, G>(a.b, wf, 0.f, j, cols);
  }
  const auto fetch = [&](int64_t row, int st) {
    if (row < a.rows) stage_row<T, G>(base + st * room, (const T*)a.x + row * a.xs, cols);
    copy_commit();
  };
  int64_t row = blockIdx.x;
  for (int s = 0; s < 2; s++) fetch(row + (int64_t)s * gridDim.x, s);
  int st = 0;
  for (; row < a.rows; row += gridDim.x) {
    copy_wait<1>();
    __syncthreads();
    fetch(row + 2 * (int64_t)gridDim.x, st == 0 ? 2 : st - 1);   // the buffer of the row before, which all have left
    const T* p = (const T*)a.x + row * a.xs;
    const uint32_t x = base + st * room + (int)((uintptr_t)p & 15);
    u64 s = 0;
#pragma unroll
    for (int j = 0; j < NJ; j += 2) s = f2::add(s, staged2<T, G>(x, j, cols));
    float v[1] = {both(s)};
    cta_sums<G, 1>(v, sh, 0);
    const float mean = __fdiv_rn(v[0], n);
    s = 0;
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      float d, e;
      f2::unpack(f2::add(staged2<T, G>(x, j, cols), f2::splat(-mean)), d, e);
      const u64 k = f2::pack(t + j * G < cols ? d : 0.f, t + (j + 1) * G < cols ? e : 0.f);
      s = f2::fma(k, k, s);
    }
    v[0] = both(s);
    cta_sums<G, 1>(v, sh, 1);
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(v[0], n) + a.eps));
    T* y = (T*)a.y + row * a.ys;
#pragma unroll
    for (int j = 0; j < NJ; j += 2)
      put2<T, G>(y, j, cols, f2::fma(f2::mul(f2::add(staged2<T, G>(x, j, cols), f2::splat(-mean)), f2::splat(rstd)), w[j / 2], b[j / 2]));
    if (t == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    st = st == 2 ? 0 : st + 1;
  }
}

template <typename T, int G, int NJ>
__global__ void __launch_bounds__(G, 512 / G) norm_bwd_staged_kernel(const NormArgs a, int64_t per, int room) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float sh[4 * (G / 32)];
  const int cols = (int)a.cols;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  const bool wf = a.wdtype == DA_F32;
  const int64_t r0 = (int64_t)blockIdx.x * per, r1 = min(r0 + per, a.rows);
  const float inv_n = __fdiv_rn(1.f, (float)a.cols);
  u64 w[NJ / 2], gw[NJ / 2], gb[NJ / 2];
#pragma unroll
  for (int j = 0; j < NJ; j += 2) {
    w[j / 2] = weight2<T, G>(a.w, wf, 1.f, j, cols);
    gw[j / 2] = gb[j / 2] = 0;
  }
  const auto fetch = [&](int64_t row, int st) {
    if (row < r1) {
      stage_row<T, G>(base + st * 2 * room, (const T*)a.x + row * a.xs, cols);
      stage_row<T, G>(base + (st * 2 + 1) * room, (const T*)a.dy + row * a.dys, cols);
    }
    copy_commit();
  };
  for (int s = 0; s < 2; s++) fetch(r0 + s, s);
  float nmean = a.mean[r0], nrstd = a.rstd[r0];
  int st = 0, turn = 0;
  for (int64_t row = r0; row < r1; row++, turn ^= 1) {
    const float mean = nmean, rstd = nrstd;
    if (row + 1 < r1) {
      nmean = a.mean[row + 1];
      nrstd = a.rstd[row + 1];
    }
    copy_wait<1>();
    __syncthreads();
    fetch(row + 2, st == 0 ? 2 : st - 1);
    const uint32_t x = base + st * 2 * room + (int)((uintptr_t)((const T*)a.x + row * a.xs) & 15);
    const uint32_t dy = base + (st * 2 + 1) * room + (int)((uintptr_t)((const T*)a.dy + row * a.dys) & 15);
    const u64 off = f2::splat(-mean), rr = f2::splat(rstd);
    u64 t1 = 0, t2 = 0;
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      const u64 d = staged2<T, G>(dy, j, cols), h = f2::mul(f2::add(staged2<T, G>(x, j, cols), off), rr);
      const u64 ad = f2::mul(d, w[j / 2]);
      gw[j / 2] = f2::fma(d, h, gw[j / 2]);   // past the row's end d is zero
      gb[j / 2] = f2::add(gb[j / 2], d);
      t1 = f2::add(t1, ad);
      t2 = f2::fma(ad, h, t2);
    }
    float s[2] = {both(t1), both(t2)};
    cta_sums<G, 2>(s, sh, turn);
    const u64 m1 = f2::splat(-s[0] * inv_n), m2 = f2::splat(-s[1] * inv_n);
    T* dx = (T*)a.y + row * a.ys;
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      const u64 h = f2::mul(f2::add(staged2<T, G>(x, j, cols), off), rr);
      put2<T, G>(dx, j, cols, f2::mul(f2::fma(h, m2, f2::fma(staged2<T, G>(dy, j, cols), w[j / 2], m1)), rr));
    }
    st = st == 2 ? 0 : st + 1;
  }
  if (!a.part) return;
  float* pw = a.part + (int64_t)blockIdx.x * a.cols;
  float* pb = pw + (int64_t)gridDim.x * a.cols;
#pragma unroll
  for (int j = 0; j < NJ; j += 2) {
    put2<float, G>(pw, j, cols, gw[j / 2]);
    put2<float, G>(pb, j, cols, gb[j / 2]);
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
template <typename T, int G, int NV, int R>
void bwd_go(const NormArgs& a, bool al, unsigned grid, int64_t per, cudaStream_t st) {
  const int threads = G == 32 ? 32 * WARP_ROWS : G;
  if (al) norm_bwd_kernel<T, G, NV, R, true><<<grid, threads, 0, st>>>(a, per);
  else norm_bwd_kernel<T, G, NV, R, false><<<grid, threads, 0, st>>>(a, per);
}

// a launch whose shared memory could not be allowed fails, and the caller sees that
template <typename T, int G, int R, int ST>
void fwd_stream(const NormArgs& a, cudaStream_t st) {
  constexpr int bytes = ST * R * 2 * G * 16;
  static DeviceOnce once;
  (void)allow_smem(once, norm_fwd_stream_kernel<T, G, 2, R, ST>, bytes);
  norm_fwd_stream_kernel<T, G, 2, R, ST><<<(unsigned)std::min<int64_t>(152 * 512 / G, (a.rows + R - 1) / R), G, bytes, st>>>(a);
}
template <typename T, int G, int R, int ST>
void bwd_stream(const NormArgs& a, unsigned grid, int64_t per, cudaStream_t st) {
  constexpr int bytes = ST * R * 2 * G * 32;
  static DeviceOnce once;
  (void)allow_smem(once, norm_bwd_stream_kernel<T, G, 2, R, ST>, bytes);
  norm_bwd_stream_kernel<T, G, 2, R, ST><<<grid, G, bytes, st>>>(a, per);
}

// bytes of a staged row's buffer
template <typename T>
int staged_room(const NormArgs& a) {
  return ((int)a.cols * (int)sizeof(T) + 31) / 16 * 16;
}
template <typename T, int G, int NJ>
void fwd_staged(const NormArgs& a, cudaStream_t st) {
  static DeviceOnce once;
  (void)allow_smem(once, norm_fwd_staged_kernel<T, G, NJ>, 3 * (G * NJ * 4 + 32));
  const int room = staged_room<T>(a);
  norm_fwd_staged_kernel<T, G, NJ><<<(unsigned)std::min<int64_t>(152 * 1024 / G, a.rows), G, 3 * room, st>>>(a, room);
}
template <typename T, int G, int NJ>
void bwd_staged(const NormArgs& a, unsigned grid, int64_t per, cudaStream_t st) {
  static DeviceOnce once;
  (void)allow_smem(once, norm_bwd_staged_kernel<T, G, NJ>, 6 * (G * NJ * 4 + 32));
  const int room = staged_room<T>(a);
  norm_bwd_staged_kernel<T, G, NJ><<<grid, G, 6 * room, st>>>(a, per, room);
}

template <typename T>
void fwd(const NormArgs& a, cudaStream_t st) {
  constexpr int VEC = Elem<T>::VEC;
  const bool al = a.cols % VEC == 0 && al16(a.x) && al16(a.y) && a.xs % VEC == 0 && a.ys % VEC == 0 && al16(a.w) && al16(a.b);
  const int64_t nv = (a.cols + VEC - 1) / VEC;
  if (al && nv > 128 && nv <= 1024 && a.rows >= 1216) {
    if (nv <= 256) fwd_stream<T, 128, 2, 2>(a, st);
    else if (nv <= 512) fwd_stream<T, 256, 2, 2>(a, st);
    else fwd_stream<T, 512, 2, 2>(a, st);
    return;
  }
  if constexpr (sizeof(T) == 2)   // f32's single-element reads are 128 bytes a warp: 27 us against 33 (3001 x 5003)
  if (!al && nv > 128 && a.cols <= 8192 && al16(a.x) && a.rows >= 304) {
    if (a.cols <= 1024) fwd_staged<T, 128, 8>(a, st);
    else if (a.cols <= 1536) fwd_staged<T, 128, 12>(a, st);
    else if (a.cols <= 2048) fwd_staged<T, 256, 8>(a, st);
    else if (a.cols <= 3072) fwd_staged<T, 256, 12>(a, st);
    else if (a.cols <= 4096) fwd_staged<T, 512, 8>(a, st);
    else if (a.cols <= 6144) fwd_staged<T, 512, 12>(a, st);
    else fwd_staged<T, 512, 16>(a, st);
    return;
  }
  if (nv <= 32) fwd_go<T, 32, 1>(a, al, st);
  else if (nv <= 128) fwd_go<T, 32, 4>(a, al, st);
  else if (nv <= 256) fwd_go<T, 128, 2>(a, al, st);
  else if (nv <= 512) fwd_go<T, 128, 4>(a, al, st);
  else if (nv <= 1024) fwd_go<T, 256, 4>(a, al, st);
  else if (nv <= 1536) fwd_go<T, 256, 6>(a, al, st);
  else if (nv <= 2048) fwd_go<T, 256, 8>(a, al, st);
  else norm_fwd_wide_kernel<T><<<(unsigned)a.rows, 1024, 0, st>>>(a);
}
template <typename T>
void bwd(const NormArgs& a, unsigned grid, int64_t per, cudaStream_t st) {
  constexpr int VEC = Elem<T>::VEC;
  const bool al = a.cols % VEC == 0 && al16(a.x) && al16(a.y) && al16(a.dy) && a.xs % VEC == 0 && a.ys % VEC == 0 && a.dys % VEC == 0 && al16(a.w);
  const int64_t nv = (a.cols + VEC - 1) / VEC;
  if (al && nv > 128 && nv <= 1024) {
    if (nv <= 256) bwd_stream<T, 128, 2, 2>(a, grid, per, st);
    else if (nv <= 512) bwd_stream<T, 256, 2, 2>(a, grid, per, st);
    else bwd_stream<T, 512, 2, 2>(a, grid, per, st);
    return;
  }
  if (!al && nv > 128 && (sizeof(T) == 2 || a.cols > 1024) && a.cols <= 8192 && al16(a.x) && al16(a.dy)) {
    if (a.cols <= 1024) bwd_staged<T, 128, 8>(a, grid, per, st);
    else if (a.cols <= 1536) bwd_staged<T, 128, 12>(a, grid, per, st);
    else if (a.cols <= 2048) bwd_staged<T, 256, 8>(a, grid, per, st);
    else if (a.cols <= 3072) bwd_staged<T, 256, 12>(a, grid, per, st);
    else if (a.cols <= 4096) bwd_staged<T, 512, 8>(a, grid, per, st);
    else if (a.cols <= 6144) bwd_staged<T, 512, 12>(a, grid, per, st);
    else bwd_staged<T, 512, 16>(a, grid, per, st);
    return;
  }
  if (nv <= 32) bwd_go<T, 32, 1, 2>(a, al, grid, per, st);
  else if (nv <= 128) bwd_go<T, 32, 4, 1>(a, al, grid, per, st);
  else if (nv <= 256) bwd_go<T, 128, 2, 2>(a, al, grid, per, st);
  else if (nv <= 512) bwd_go<T, 256, 2, 2>(a, al, grid, per, st);
  else if (nv <= 1024) bwd_go<T, 512, 2, 1>(a, al, grid, per, st);
  else if (nv <= 1536) bwd_go<T, 512, 3, 1>(a, al, grid, per, st);
  else if (nv <= 2048) bwd_go<T, 512, 4, 1>(a, al, grid, per, st);
  else norm_bwd_wide_kernel<T><<<grid, 1024, 0, st>>>(a, per);
}

int64_t rows_per(int64_t rows, int64_t cols) {
  // about two resident CTAs (eight of the warp variants) on each of 152 SMs; a run has a multiple
  // of the rows that a CTA takes at a time
  const int64_t want = cols <= 1024 ? 152 * 8 : 152 * 2, by = cols <= 1024 ? 8 : 2;
  return ((rows + want - 1) / want + by - 1) / by * by;
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
