// AdamW over many tensors in one launch, with f32 or 8-bit states.
//
// Per element, every operation rounded once to binary32 (so the same operations on f32 tensors
// give the same bits):
//   m = RN(m b1) + RN(g (1 - b1));  v = RN(v b2) + RN(RN(g g) (1 - b2));
//   p = RN(p (1 - lr wd)) - RN(RN(m / RN(RN(sqrt(v) undo) + eps)) rate),
// undo = 1 / sqrt(1 - b2^t), rate = lr / (1 - b1^t); p rounded once more to its own type.
//
// 8-bit states: a block of 256 elements of a tensor holds e4m3 values and one f32 scale,
// max |x| / 448 over the block (0 below 2^-100, where the block's values become zero); x = value *
// scale.  Of the second moment its square root is kept, which halves the exponents it spans;
// a root above zero never becomes zero (it would leave m / eps), it takes the smallest value.
//
// What bounds it: HBM.  f32 states move 28 bytes an element, 8-bit ones with bf16 parameters
// 10.03.  Each CTA takes 2048 elements of one tensor, found by a search in a table that travels
// in the launch's parameters, so no table lies in device memory and a step is one launch for
// 120 tensors.  A thread takes two groups of four neighbours 1024 (f32) or 128 (8-bit) apart:
// every access of a warp is one run of whole sectors, and all of a thread's loads are issued
// before its arithmetic.  An 8-bit block belongs to one warp, whose largest value is one integer
// warp reduction (bits of non-negative floats are ordered).
#include <cuda_fp8.h>

#include "../../include/detattn.h"
#include "train_kernels.h"
#include "train_math.cuh"

namespace detattn {
namespace {

__device__ __forceinline__ float from_e4m3(uint32_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, int64_t i, int64_t n, bool vec, float (&x)[4]) {
  if (vec && i + 4 <= n) {
    const Pack<T, 4> r = *reinterpret_cast<const Pack<T, 4>*>(p + i);
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = Elem<T>::get(r.e[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = i + e < n ? Elem<T>::get(p[i + e]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int64_t i, int64_t n, bool vec, const float (&x)[4]) {
  if (vec && i + 4 <= n) {
    Pack<T, 4> r;
#pragma unroll
    for (int e = 0; e < 4; e++) r.e[e] = Elem<T>::put(x[e]);
    *reinterpret_cast<Pack<T, 4>*>(p + i) = r;
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (i + e < n) p[i + e] = Elem<T>::put(x[e]);
  }
}

// four values times inv, to e4m3 (saturating at 448)
__device__ __forceinline__ uint32_t to_e4m3(const float (&x)[4], float inv, bool keep_positive) {
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    float c = __fmul_rn(x[e], inv);
    if (keep_positive && c > 0.f && c < 0.001953125f) c = 0.001953125f;
    r |= (uint32_t)__nv_cvt_float_to_fp8(c, __NV_SATFINITE, __NV_E4M3) << (8 * e);
  }
  return r;
}

template <typename T, bool EIGHT>
__global__ void __launch_bounds__(256) adamw_kernel(const __grid_constant__ AdamWArgs a) {
  const uint32_t chunk = blockIdx.x;
  int lo = 0, hi = a.nt;                     // the last tensor whose first chunk is not above this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  const int64_t n = a.t[lo].n, base = (int64_t)(chunk - a.first[lo]) * ADAMW_CHUNK, s0 = a.t[lo].state;
  T* p = (T*)a.t[lo].p;
  const T* g = (const T*)a.t[lo].g;
  constexpr int APART = EIGHT ? 128 : 1024;
  const int64_t i0 = base + (EIGHT ? (threadIdx.x >> 5) * ADAMW_BLOCK + (threadIdx.x & 31) * 4 : threadIdx.x * 4);
  if (EIGHT && base + (threadIdx.x >> 5) * ADAMW_BLOCK >= n) return;   // whole warps: a block ends the tensor
  const bool vp = ((uintptr_t)p & (4 * sizeof(T) - 1)) == 0, vg = ((uintptr_t)g & (4 * sizeof(T) - 1)) == 0;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;

  float P[2][4], G[2][4], M[2][4], V[2][4];
  uint32_t mc[2], vc[2];
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int64_t i = i0 + k * APART;
    load4(p, i, n, vp, P[k]);
    load4(g, i, n, vg, G[k]);
    if constexpr (EIGHT) {
      mc[k] = *reinterpret_cast<const uint32_t*>((const uint8_t*)a.m + s0 + i);
      vc[k] = *reinterpret_cast<const uint32_t*>((const uint8_t*)a.v + s0 + i);
    } else {
      load4((const float*)a.m + s0, i, n, true, M[k]);
      load4((const float*)a.v + s0, i, n, true, V[k]);
    }
  }
  const int64_t blk = (s0 + i0) / ADAMW_BLOCK;
  if constexpr (EIGHT) {
    const float ms = a.m_scale[blk], vs = a.v_scale[blk];
#pragma unroll
    for (int k = 0; k < 2; k++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        M[k][e] = __fmul_rn(from_e4m3((mc[k] >> (8 * e)) & 0xFF), ms);
        const float r = __fmul_rn(from_e4m3((vc[k] >> (8 * e)) & 0xFF), vs);
        V[k][e] = __fmul_rn(r, r);
      }
  }
  uint32_t mtop = 0, vtop = 0;
#pragma unroll
  for (int k = 0; k < 2; k++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      float gr = G[k][e];
      if (a.grad_scale) gr = __fmul_rn(gr, gs);
      const float m = __fadd_rn(__fmul_rn(M[k][e], a.b1), __fmul_rn(gr, a.c1));
      const float v = __fadd_rn(__fmul_rn(V[k][e], a.b2), __fmul_rn(__fmul_rn(gr, gr), a.c2));
      const float root = __fsqrt_rn(v);
      const float step = __fdiv_rn(m, __fadd_rn(__fmul_rn(root, a.undo), a.eps));
      P[k][e] = __fsub_rn(__fmul_rn(P[k][e], a.keep), __fmul_rn(step, a.rate));
      const bool in = !EIGHT || i0 + k * APART + e < n;   // past the tensor's end a block's values are zero
      M[k][e] = in ? m : 0.f;
      V[k][e] = EIGHT ? (in ? root : 0.f) : v;
      if (EIGHT) {
        mtop = max(mtop, __float_as_uint(fabsf(M[k][e])));
        vtop = max(vtop, __float_as_uint(V[k][e]) & 0x7FFFFFFFu);
      }
    }
  if constexpr (EIGHT) {
    const float mt = __uint_as_float(__reduce_max_sync(0xffffffffu, mtop));
    const float vt = __uint_as_float(__reduce_max_sync(0xffffffffu, vtop));
    const float mi = mt >= 0x1p-100f ? __fdiv_rn(448.f, mt) : 0.f, vi = vt >= 0x1p-100f ? __fdiv_rn(448.f, vt) : 0.f;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      mc[k] = to_e4m3(M[k], mi, false);
      vc[k] = to_e4m3(V[k], vi, true);
    }
    if ((threadIdx.x & 31) == 0) {
      a.m_scale[blk] = mt >= 0x1p-100f ? __fdiv_rn(mt, 448.f) : 0.f;
      a.v_scale[blk] = vt >= 0x1p-100f ? __fdiv_rn(vt, 448.f) : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int64_t i = i0 + k * APART;
    store4(p, i, n, vp, P[k]);
    if constexpr (EIGHT) {
      *reinterpret_cast<uint32_t*>((uint8_t*)a.m + s0 + i) = mc[k];
      *reinterpret_cast<uint32_t*>((uint8_t*)a.v + s0 + i) = vc[k];
    } else {
      store4((float*)a.m + s0, i, n, true, M[k]);
      store4((float*)a.v + s0, i, n, true, V[k]);
    }
  }
}

template <typename T>
void go(const AdamWArgs& a, int bits, cudaStream_t st) {
  const uint32_t grid = a.first[a.nt];
  if (bits == 8) adamw_kernel<T, true><<<grid, 256, 0, st>>>(a);
  else adamw_kernel<T, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_adamw(const AdamWArgs& a, int dtype, int bits, cudaStream_t st) {
  if (a.nt == 0 || a.first[a.nt] == 0) return cudaSuccess;
  if (dtype == DA_F32) go<float>(a, bits, st);
  else if (dtype == DA_BF16) go<__nv_bfloat16>(a, bits, st);
  else go<__half>(a, bits, st);
  return cudaGetLastError();
}

}  // namespace detattn
