// AdamW over many tensors in one launch, with f32 or 8-bit states.
//
// Per element, every operation rounded once to binary32 (so the same operations on f32 tensors
// give the same bits):
//   m = RN(m b1) + RN(g (1 - b1));  v = RN(v b2) + RN(RN(g g) (1 - b2));
//   p = RN(p (1 - lr wd)) - RN(RN(m / RN(RN(sqrt(v) undo) + eps)) rate),
// undo = 1 / sqrt(1 - b2^t), rate = lr / (1 - b1^t); p rounded once more to its own type.
//
// 8-bit states: a block of 256 elements of a tensor holds e4m3 values and one f32 scale,
// max |x| / 448 over the block's finite x (0 below 2^-100, where the block's values become zero); x = value *
// scale; an x that is not finite becomes NaN.  Of the second moment its square root is kept, which halves the exponents it spans;
// a root above zero never becomes zero (it would leave m / eps), it takes the smallest value.
//
// What bounds it: HBM.  f32 states move 28 bytes an element, 8-bit ones with bf16 parameters
// 10.03.  Each CTA takes 2048 elements of one tensor, found by a search
// in a table that travels in the launch's parameters, so no table lies in device memory and a step
// is one launch for 120 tensors.  A thread's 8 elements are runs of 16 bytes of the parameter
// (8 for a 16-bit one with f32 states): every access of a warp is one run of whole sectors, and all of a
// thread's loads are issued before its arithmetic.  An 8-bit block belongs to one warp, whose largest
// value is one integer warp reduction (bits of non-negative floats are ordered).  Only a tensor's last CTA tests for its end.
#include "../../include/detattn.h"
#include "pack2.cuh"
#include "train_kernels.h"
#include "train_math.cuh"

namespace detattn {
namespace {

// two e4m3 values of the low 16 bits
__device__ __forceinline__ float2 from_e4m3x2(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(b));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// two values to e4m3, saturating at 448
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T, int E>
__device__ __forceinline__ void load_run(const T* p, int64_t i, int64_t n, bool vec, float* x) {
  if (vec && i + E <= n) {
    Run<T, E> r;
    r.load(p + i);
#pragma unroll
    for (int e = 0; e < E; e++) x[e] = r.get(e);
  } else {
#pragma unroll
    for (int e = 0; e < E; e++) x[e] = i + e < n ? Elem<T>::get(p[i + e]) : 0.f;
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_run(T* p, int64_t i, int64_t n, bool vec, const float* x) {
  if (vec && i + E <= n) {
    Run<T, E> r;
    r.set(x);
    r.store(p + i);
  } else {
#pragma unroll
    for (int e = 0; e < E; e++)
      if (i + e < n) p[i + e] = Elem<T>::put(x[e]);
  }
}

// Two elements: m, v -> the next ones and the parameters; root is sqrt(v).  The products go two at a time through
// the packed multiplier, each lane rounded as the scalar one; the sums stay scalar, so no
// product and sum can be contracted into one rounding.
struct Two {
  float a, b;
};
__device__ __forceinline__ Two times(Two x, float k) {
  Two r;
  f2::unpack(f2::mul(f2::pack(x.a, x.b), f2::splat(k)), r.a, r.b);
  return r;
}
__device__ __forceinline__ Two square(Two x) {
  Two r;
  const f2::u64 p = f2::pack(x.a, x.b);
  f2::unpack(f2::mul(p, p), r.a, r.b);
  return r;
}
__device__ __forceinline__ Two plus(Two x, Two y) { return {__fadd_rn(x.a, y.a), __fadd_rn(x.b, y.b)}; }
__device__ __forceinline__ void update(const AdamWArgs& k, Two g, Two& p, Two& m, Two& v, Two& root) {
  m = plus(times(m, k.b1), times(g, k.c1));
  v = plus(times(v, k.b2), times(square(g), k.c2));
  root = {__fsqrt_rn(v.a), __fsqrt_rn(v.b)};
  const Two d = times(root, k.undo);
  const Two step = {__fdiv_rn(m.a, __fadd_rn(d.a, k.eps)), __fdiv_rn(m.b, __fadd_rn(d.b, k.eps))};
  const Two kept = times(p, k.keep), back = times(step, k.rate);
  p = {__fsub_rn(kept.a, back.a), __fsub_rn(kept.b, back.b)};
}

// the tensor of a chunk: the last one whose first chunk is not above it
__device__ __forceinline__ int find(const AdamWArgs& a, uint32_t chunk) {
  int lo = 0, hi = a.nt;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

template <typename T>
__global__ void __launch_bounds__(256) adamw_kernel(const __grid_constant__ AdamWArgs a) {
  const int ti = find(a, blockIdx.x);
  const int64_t n = a.t[ti].n, i0 = (int64_t)(blockIdx.x - a.first[ti]) * ADAMW_CHUNK + threadIdx.x * 4;
  T* p = (T*)a.t[ti].p;
  const T* g = (const T*)a.t[ti].g;
  float* ms = (float*)a.m + a.t[ti].state;
  float* vs = (float*)a.v + a.t[ti].state;
  const bool vp = ((uintptr_t)p & (4 * sizeof(T) - 1)) == 0, vg = ((uintptr_t)g & (4 * sizeof(T) - 1)) == 0;
  float P[2][4], G[2][4], M[2][4], V[2][4];
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int64_t i = i0 + k * 1024;
    load_run<T, 4>(p, i, n, vp, P[k]);
    load_run<T, 4>(g, i, n, vg, G[k]);
    load_run<float, 4>(ms, i, n, true, M[k]);
    load_run<float, 4>(vs, i, n, true, V[k]);
  }
  if (a.grad_scale) {
    const float gs = *a.grad_scale;
#pragma unroll
    for (int k = 0; k < 2; k++)
#pragma unroll
      for (int e = 0; e < 4; e++) G[k][e] = __fmul_rn(G[k][e], gs);
  }
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int64_t i = i0 + k * 1024;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      Two pp = {P[k][e], P[k][e + 1]}, m = {M[k][e], M[k][e + 1]}, v = {V[k][e], V[k][e + 1]}, root;
      update(a, {G[k][e], G[k][e + 1]}, pp, m, v, root);
      P[k][e] = pp.a; P[k][e + 1] = pp.b;
      M[k][e] = m.a; M[k][e + 1] = m.b;
      V[k][e] = v.a; V[k][e + 1] = v.b;
    }
    store_run<T, 4>(p, i, n, vp, P[k]);
    store_run<float, 4>(ms, i, n, true, M[k]);
    store_run<float, 4>(vs, i, n, true, V[k]);
  }
}

// a run of words: whole, or element by element up to n
template <typename T, int E>
__device__ __forceinline__ void load_words(Run<T, E>& r, const T* p, int64_t i, int left, bool whole) {
  if (whole) {
    r.load(p + i);
  } else {
    r.zero();
#pragma unroll
    for (int e = 0; e < E; e++)
      if (e < left) r.put_bits(e, p[i + e]);
  }
}

// One warp a block of 256 elements.  Parameter and gradient stay packed words until their turn: registers, and
// with them the warps whose loads are in flight, bound this kernel beside the arithmetic of the roots and
// divisions.  144 M bf16 parameters: 329 us (4.4 TB/s) at 6 CTAs an SM (328 before
// infinities were kept apart, then 331 at 5, 343 with spills at 8); 482 with
// the operands unpacked first (4 CTAs), 650 with two blocks a warp (2 CTAs).
template <typename T>
__global__ void __launch_bounds__(256, 6) adamw8_kernel(const __grid_constant__ AdamWArgs a) {
  constexpr int E = sizeof(T) == 4 ? 4 : 8, RUNS = 8 / E;   // a lane's runs of the block
  const int ti = find(a, blockIdx.x), lane = threadIdx.x & 31;
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * ADAMW_CHUNK + (threadIdx.x >> 5) * ADAMW_BLOCK;
  const int size = (int)min(a.t[ti].n - i0, (int64_t)ADAMW_BLOCK);
  if (size <= 0) return;                                     // whole warps
  const int at = lane * E;
  T* p = (T*)a.t[ti].p + i0 + at;
  const T* g = (const T*)a.t[ti].g + i0 + at;
  const int64_t s0 = a.t[ti].state + i0;
  uint8_t* ms = (uint8_t*)a.m + s0 + at;
  uint8_t* vs = (uint8_t*)a.v + s0 + at;
  float* msc = a.m_scale + s0 / ADAMW_BLOCK;
  float* vsc = a.v_scale + s0 / ADAMW_BLOCK;
  const bool full = size == ADAMW_BLOCK;
  const bool vp = full && ((uintptr_t)p & (E * sizeof(T) - 1)) == 0, vg = full && ((uintptr_t)g & (E * sizeof(T) - 1)) == 0;
  Run<T, E> P[RUNS], G[RUNS];
  uint32_t mc[2], vc[2];
#pragma unroll
  for (int k = 0; k < RUNS; k++) {
    load_words<T, E>(P[k], p, k * 128, size - at - k * 128, vp);
    load_words<T, E>(G[k], g, k * 128, size - at - k * 128, vg);
  }
  if constexpr (E == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(ms), y = *reinterpret_cast<const uint2*>(vs);
    mc[0] = x.x; mc[1] = x.y;
    vc[0] = y.x; vc[1] = y.y;
  } else {
    mc[0] = *reinterpret_cast<const uint32_t*>(ms);
    mc[1] = *reinterpret_cast<const uint32_t*>(ms + 128);
    vc[0] = *reinterpret_cast<const uint32_t*>(vs);
    vc[1] = *reinterpret_cast<const uint32_t*>(vs + 128);
  }
  const float sm = *msc, sv = *vsc;
  float M[8], R[8], mtop = 0.f, vtop = 0.f;
#pragma unroll
  for (int w = 0; w < 4; w++) {
    const int k = 2 * w / E, e = 2 * w % E;
    const float2 m2 = from_e4m3x2(mc[w >> 1] >> (16 * (w & 1))), r2 = from_e4m3x2(vc[w >> 1] >> (16 * (w & 1)));
    Two m = times({m2.x, m2.y}, sm), v = square(times({r2.x, r2.y}, sv)), root;
    Two p2 = {P[k].get(e), P[k].get(e + 1)}, g2 = {G[k].get(e), G[k].get(e + 1)};
    if (a.grad_scale) g2 = times(g2, *a.grad_scale);
    update(a, g2, p2, m, v, root);
    P[k].set2(e / 2, f2::pack(p2.a, p2.b));
    if (!full) {   // past the end a block holds zeros
      if (at + k * 128 + e >= size) m.a = root.a = 0.f;
      if (at + k * 128 + e + 1 >= size) m.b = root.b = 0.f;
    }
    M[2 * w] = m.a; M[2 * w + 1] = m.b;
    R[2 * w] = root.a; R[2 * w + 1] = root.b;
    mtop = fmaxf(fmaxf(mtop, fabsf(m.a)), fabsf(m.b));   // NaN left out: it stays in its own element
    vtop = fmaxf(fmaxf(vtop, root.a), root.b);
  }
#pragma unroll
  for (int k = 0; k < RUNS; k++) {
    if (vp) {
      P[k].store(p + k * 128);
    } else {
#pragma unroll
      for (int e = 0; e < E; e++)
        if (at + k * 128 + e < size) p[k * 128 + e] = P[k].bits(e);
    }
  }
  float mt = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop)));
  float vt = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)));
  if (fmaxf(mt, vt) == INFINITY) {   // an infinity would be the block's scale: it stays in its own element, as NaN
    const auto finite_top = [](float (&x)[8]) {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        if (fabsf(x[e]) == INFINITY) x[e] = __uint_as_float(0x7fffffffu);
        top = fmaxf(top, fabsf(x[e]));
      }
      return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    };
    mt = finite_top(M);
    vt = finite_top(R);
  }
  const bool ml = mt >= 0x1p-100f, vl = vt >= 0x1p-100f;
  const float mi = ml ? __fdiv_rn(448.f, mt) : 0.f, vi = vl ? __fdiv_rn(448.f, vt) : 0.f;
  const float floor = vl ? 0x1p-9f : 0.f;
  mc[0] = mc[1] = vc[0] = vc[1] = 0;
#pragma unroll
  for (int w = 0; w < 4; w++) {
    const Two m = times({M[2 * w], M[2 * w + 1]}, mi), r = times({R[2 * w], R[2 * w + 1]}, vi);
    mc[w >> 1] |= to_e4m3x2(m.a, m.b) << (16 * (w & 1));
    vc[w >> 1] |= to_e4m3x2(r.a > 0.f ? fmaxf(r.a, floor) : r.a, r.b > 0.f ? fmaxf(r.b, floor) : r.b) << (16 * (w & 1));
  }
  if constexpr (E == 8) {
    *reinterpret_cast<uint2*>(ms) = make_uint2(mc[0], mc[1]);
    *reinterpret_cast<uint2*>(vs) = make_uint2(vc[0], vc[1]);
  } else {
    *reinterpret_cast<uint32_t*>(ms) = mc[0];
    *reinterpret_cast<uint32_t*>(ms + 128) = mc[1];
    *reinterpret_cast<uint32_t*>(vs) = vc[0];
    *reinterpret_cast<uint32_t*>(vs + 128) = vc[1];
  }
  if (lane == 0) {
    *msc = ml ? __fdiv_rn(mt, 448.f) : 0.f;
    *vsc = vl ? __fdiv_rn(vt, 448.f) : 0.f;
  }
}

template <typename T>
void go(const AdamWArgs& a, int bits, cudaStream_t st) {
  const uint32_t grid = a.first[a.nt];
  if (bits == 8) adamw8_kernel<T><<<grid, 256, 0, st>>>(a);
  else adamw_kernel<T><<<grid, 256, 0, st>>>(a);
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
