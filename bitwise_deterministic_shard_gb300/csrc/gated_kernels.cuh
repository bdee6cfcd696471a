// The gated feed-forward projections and their gradient.
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u
//   dg = dh p,  du = dh q,  p = act'(g) u,  q = act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// Forward: one kernel of pair products (gemm_pair.cuh).  The 256 rows of its second operand are 128 rows of Wg (one CTA's half)
// and the same 128 of Wu (the other's), so g and u of a token and hidden unit lie in one TMEM lane, 128 columns apart,
// and a thread forms h from them.  For the backward pass it also writes p and q, the only values of the activation that the
// gradient needs: 24 bits of each (2^-15 of the value left out), as 16 would add a rounding of the size of the result's own to dg
// and du (dx then 2.9e-3 off in bf16 instead of 2.4e-3; 1.7e-3 is a result only rounded).
// Backward: dg and du as one pass over dh, p and q, rounded to 16 bits (the tensor cores take operands of one 16-bit type), then two
// kernels of pair products: dx contracts over both halves of [dg | du] in one chain, dW has the tiles of both weights.
//
// Up to 8 tokens the forward pass reads the weights once with plain loads instead: a warp a hidden unit.
#pragma once
#include "../../include/detattn.h"
#include "decoder_kernels.h"
#include "device_once.h"
#include "gemm_pair.cuh"
#include "train_math.cuh"

namespace detattn {
namespace gl {

using tc5::ex2;
using tc5::rcp;

constexpr float LOG2E = 1.4426950408889634f;

// act(g) and act'(g), ACT a DGL_* code.  With s the logistic function: silu g s(g); gelu g Phi(g); its tanh form g s(2 y),
// y = sqrt(2 / pi) (g + 0.044715 g^3), as (1 + tanh y) / 2 = s(2 y) has no cancellation.
__device__ __forceinline__ float logistic(float x) { return rcp(1.f + ex2(-LOG2E * x)); }
template <int ACT>
__device__ __forceinline__ void activate(float g, float& a, float& d) {
  if constexpr (ACT == DGL_SILU) {
    const float s = logistic(g);
    a = g * s;
    d = s * __fmaf_rn(g, 1.f - s, 1.f);
  } else if constexpr (ACT == DGL_GELU) {
    const float s = normcdff(g);
    a = g * s;
    d = __fmaf_rn(g * 0.3989422804014327f, ex2(-0.5f * LOG2E * g * g), s);
  } else if constexpr (ACT == DGL_GELU_TANH) {
    constexpr float c = 0.7978845608028654f, k = 0.044715f;
    const float g2 = g * g;
    const float s = logistic(2.f * c * g * __fmaf_rn(k, g2, 1.f));
    a = g * s;
    d = s * __fmaf_rn(2.f * c * g * __fmaf_rn(3.f * k, g2, 1.f), 1.f - s, 1.f);
  } else {
    a = g > 0.f ? g : g != g ? g : 0.f;
    d = g > 0.f ? 1.f : g != g ? g : 0.f;
  }
}

// ---- forward ----
template <bool BF, int ACT, bool SAVE>
__global__ void __launch_bounds__(pair::THREADS, 1) __cluster_dims__(2, 1, 1) gl_fwd_kernel(const __grid_constant__ GlArgs a) {
  using namespace tc5;
  extern __shared__ unsigned char raw[];
  __shared__ pair::Shared sh;
  const int mt = (a.T + 255) / 256, nt = (a.F + 127) / 128, steps = (a.D + pair::BK - 1) / pair::BK;
  const uint32_t rank = pair::cta_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t n = (size_t)a.T * a.F;
  pair::run<BF, false, false>(
      sh, raw, mt * nt, steps, a.status,
      [&](int t, int k, uint32_t A, uint32_t B, uint32_t bar) {
        const int2 at = pair::tile_of(t, mt, nt);
        pair::load2(A, &a.a[0], k * pair::BK, at.x * 256 + rank * 128, bar);
        pair::load2(B, &a.b[rank], k * pair::BK, at.y * 128, bar);
      },
      [&](int t, uint32_t tm, auto release) {
        const int2 at = pair::tile_of(t, mt, nt);
        const int row = at.x * 256 + rank * 128 + (warp & 3) * 32 + lane;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          const int cc = (warp >> 2) * 64 + c, col = at.y * 128 + cc;   // columns of the tile and of h
          float g[32], u[32];
          __syncwarp();   // the loads are the whole warp's
          ld_x32(tm + cc, g);
          ld_x32(tm + 128 + cc, u);
          ld_wait();
          if (c == 32) release();
          if (row >= a.T) continue;
          uint32_t h[16];
          const size_t out = (size_t)row * a.F + col;
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float p[8], q[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
              float d;
              activate<ACT>(g[e + i], q[i], d);
              p[i] = d * u[e + i];
              g[e + i] = q[i] * u[e + i];
            }
#pragma unroll
            for (int i = 0; i < 4; i++) h[e / 2 + i] = pack16<BF>(g[e + 2 * i], g[e + 2 * i + 1]);
            if (col + e >= a.F) continue;
            if constexpr (SAVE) {
#pragma unroll
              for (int w = 0; w < 2; w++) {
                const float* const v = w ? q : p;
                uint32_t hi[4], lo[2];
#pragma unroll
                for (int i = 0; i < 4; i++)
                  hi[i] = __byte_perm(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), 0x7632);
#pragma unroll
                for (int i = 0; i < 2; i++)
                  lo[i] = __byte_perm(__byte_perm(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), 0x0051),
                                      __byte_perm(__float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]), 0x0051), 0x5410);
                *reinterpret_cast<uint4*>(a.saved + 2 * (w * n + out + e)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint2*>(a.saved + 4 * n + w * n + out + e) = make_uint2(lo[0], lo[1]);
              }
            }
            uint4* const to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[0]) + (size_t)row * a.os[0] + col + e);
            *to = make_uint4(h[e / 2], h[e / 2 + 1], h[e / 2 + 2], h[e / 2 + 3]);
          }
        }
      });
}

// One thread's row of a tile of a plain product: columns [c0, c0 + 128) of the tile.
template <bool BF, typename Release>
__device__ __forceinline__ void take_row(uint32_t tm, int c0, uint16_t* out, bool live, int left, Release release) {
  using namespace tc5;
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    float v[32];
    __syncwarp();   // the loads are the whole warp's
    ld_x32(tm + c0 + c, v);
    ld_wait();
    if (c == 96) release();
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < 32; e += 8)
      if (c0 + c + e < left)
        *reinterpret_cast<uint4*>(out + c0 + c + e) =
            make_uint4(pack16<BF>(v[e], v[e + 1]), pack16<BF>(v[e + 2], v[e + 3]), pack16<BF>(v[e + 4], v[e + 5]),
                       pack16<BF>(v[e + 6], v[e + 7]));
  }
}

// ---- dx [T, D] = [dg | du] [Wg; Wu]: a: dg and du (K-major), b: Wg and Wu (MN-major) ----
template <bool BF>
__global__ void __launch_bounds__(pair::THREADS, 1) __cluster_dims__(2, 1, 1) gl_dx_kernel(const __grid_constant__ GlArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ pair::Shared sh;
  const int mt = (a.T + 255) / 256, nt = (a.D + 255) / 256, half = (a.F + pair::BK - 1) / pair::BK;
  const uint32_t rank = pair::cta_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pair::run<BF, false, true>(
      sh, raw, mt * nt, 2 * half, a.status,
      [&](int t, int k, uint32_t A, uint32_t B, uint32_t bar) {
        const int2 at = pair::tile_of(t, mt, nt);
        const int w = k >= half, k0 = (k - w * half) * pair::BK, c = at.y * 256 + rank * 128;
        pair::load2(A, &a.a[w], k0, at.x * 256 + rank * 128, bar);
        pair::load2(B, &a.b[w], c, k0, bar);
        pair::load2(B + pair::HALF / 2, &a.b[w], c + 64, k0, bar);
      },
      [&](int t, uint32_t tm, auto release) {
        const int2 at = pair::tile_of(t, mt, nt);
        const int row = at.x * 256 + rank * 128 + (warp & 3) * 32 + lane;
        uint16_t* const out = static_cast<uint16_t*>(a.out[0]) + (size_t)row * a.os[0] + at.y * 256;
        take_row<BF>(tm, (warp >> 2) * 128, out, row < a.T, a.D - at.y * 256, release);
      });
}

// ---- dWg, dWu [F, D] = dg^T x, du^T x: a: dg and du (MN-major), b: x (MN-major) ----
template <bool BF>
__global__ void __launch_bounds__(pair::THREADS, 1) __cluster_dims__(2, 1, 1) gl_dw_kernel(const __grid_constant__ GlArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ pair::Shared sh;
  const int half = (a.F + 255) / 256, mt = 2 * half, nt = (a.D + 255) / 256, steps = (a.T + pair::BK - 1) / pair::BK;
  const uint32_t rank = pair::cta_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pair::run<BF, true, true>(
      sh, raw, mt * nt, steps, a.status,
      [&](int t, int k, uint32_t A, uint32_t B, uint32_t bar) {
        const int2 at = pair::tile_of(t, mt, nt);
        const int w = at.x >= half, r = (at.x - w * half) * 256 + rank * 128, c = at.y * 256 + rank * 128;
        pair::load2(A, &a.a[w], r, k * pair::BK, bar);
        pair::load2(A + pair::HALF / 2, &a.a[w], r + 64, k * pair::BK, bar);
        pair::load2(B, &a.b[0], c, k * pair::BK, bar);
        pair::load2(B + pair::HALF / 2, &a.b[0], c + 64, k * pair::BK, bar);
      },
      [&](int t, uint32_t tm, auto release) {
        const int2 at = pair::tile_of(t, mt, nt);
        const int w = at.x >= half, row = (at.x - w * half) * 256 + rank * 128 + (warp & 3) * 32 + lane;
        uint16_t* const out = static_cast<uint16_t*>(a.out[w]) + (size_t)row * a.os[w] + at.y * 256;
        take_row<BF>(tm, (warp >> 2) * 128, out, row < a.F, a.D - at.y * 256, release);
      });
}

// ---- few tokens: a warp a hidden unit, 16 bytes of each weight row a lane ----
template <bool BF, int NT, int ACT>
__global__ void __launch_bounds__(256) gl_few_kernel(const GlFewArgs a) {
  using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
  using f2::u64;
  const int lane = threadIdx.x & 31, f = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (f >= a.F) return;
  const T* const wg = static_cast<const T*>(a.wg) + f * a.gs;
  const T* const wu = static_cast<const T*>(a.wu) + f * a.us;
  const T* const x = static_cast<const T*>(a.x);
  u64 g[NT], u[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) g[t] = u[t] = 0;
  constexpr int U = NT > 4 ? 2 : 4;   // runs of 256 elements at once
  for (int k0 = lane * 8; k0 < a.D; k0 += 256 * U) {
    Run<T, 8> rg[U], ru[U];
#pragma unroll
    for (int i = 0; i < U; i++) {
      rg[i].zero();
      ru[i].zero();
      if (k0 + 256 * i < a.D) {
        rg[i].load(wg + k0 + 256 * i);
        ru[i].load(wu + k0 + 256 * i);
      }
    }
#pragma unroll
    for (int i = 0; i < U; i++) {
      if (k0 + 256 * i >= a.D) break;
#pragma unroll
      for (int t = 0; t < NT; t++) {
        if (t >= a.T) break;
        Run<T, 8> rx;
        rx.load(x + t * a.xs + k0 + 256 * i);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const u64 v = rx.get2(e);
          g[t] = f2::fma(rg[i].get2(e), v, g[t]);
          u[t] = f2::fma(ru[i].get2(e), v, u[t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; t++) {
    if (t >= a.T) break;
    float a0, a1, b0, b1;
    f2::unpack(g[t], a0, a1);
    f2::unpack(u[t], b0, b1);
    const float gs = warp_sum(a0 + a1), us = warp_sum(b0 + b1);
    float q, d;
    activate<ACT>(gs, q, d);
    if (lane == 0) static_cast<T*>(a.h)[t * a.hs + f] = Elem<T>::put(q * us);
  }
}

// ---- dg = dh p, du = dh q: 8 elements a thread ----
template <bool BF>
__global__ void __launch_bounds__(256) gl_scale_kernel(const GlScaleArgs a) {
  using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
  const int64_t n = a.T * a.F, per = a.F / 8, all = n / 8;
  T* const dg = static_cast<T*>(a.dg);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    Run<T, 8> r;
    r.load(static_cast<const T*>(a.dh) + (i / per) * a.ds + (i % per) * 8);
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const uint4 hi = *reinterpret_cast<const uint4*>(a.saved + 2 * (w * n + 8 * i));
      const uint2 lo = *reinterpret_cast<const uint2*>(a.saved + 4 * n + w * n + 8 * i);
      const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e++)   // bits 31..16 and 15..8
        v[e] = r.get(e) * __uint_as_float((h[e >> 1] >> (16 * (e & 1)) << 16) | ((e < 4 ? lo.x : lo.y) >> (8 * (e & 3)) & 255) << 8);
      Run<T, 8> o;
      o.set(v);
      o.store(dg + w * n + 8 * i);
    }
  }
}

inline cudaError_t pairs_of_device(int* n) {
  int device;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, device);
  *n /= 2;
  return e;
}

template <typename K, typename A>
cudaError_t launch_pairs(DeviceOnce& once, K kernel, int64_t tiles, const A& a, cudaStream_t st) {
  if (tiles == 0) return cudaSuccess;
  int pairs;
  cudaError_t e = pairs_of_device(&pairs);
  if (e == cudaSuccess) e = allow_smem(once, kernel, pair::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<2 * (int)(tiles < pairs ? tiles : pairs), pair::THREADS, pair::SMEM, st>>>(a);
  return cudaGetLastError();
}

template <bool BF, int ACT, bool SAVE>
cudaError_t forward_of(const GlArgs& a, cudaStream_t st) {
  static DeviceOnce once;
  return launch_pairs(once, gl_fwd_kernel<BF, ACT, SAVE>, (int64_t)((a.T + 255) / 256) * ((a.F + 127) / 128), a, st);
}
template <bool BF, int ACT>
cudaError_t few_of(const GlFewArgs& a, cudaStream_t st) {
  const int grid = (a.F + 7) / 8;
  if (a.T <= 1) gl_few_kernel<BF, 1, ACT><<<grid, 256, 0, st>>>(a);
  else if (a.T <= 2) gl_few_kernel<BF, 2, ACT><<<grid, 256, 0, st>>>(a);
  else if (a.T <= 4) gl_few_kernel<BF, 4, ACT><<<grid, 256, 0, st>>>(a);
  else gl_few_kernel<BF, 8, ACT><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gl

template <bool BF>
cudaError_t gl_forward(const GlArgs& a, cudaStream_t st) {
  using namespace gl;
  if (a.saved) {
    switch (a.activation) {
      case DGL_SILU: return forward_of<BF, DGL_SILU, true>(a, st);
      case DGL_GELU: return forward_of<BF, DGL_GELU, true>(a, st);
      case DGL_GELU_TANH: return forward_of<BF, DGL_GELU_TANH, true>(a, st);
      default: return forward_of<BF, DGL_RELU, true>(a, st);
    }
  }
  switch (a.activation) {
    case DGL_SILU: return forward_of<BF, DGL_SILU, false>(a, st);
    case DGL_GELU: return forward_of<BF, DGL_GELU, false>(a, st);
    case DGL_GELU_TANH: return forward_of<BF, DGL_GELU_TANH, false>(a, st);
    default: return forward_of<BF, DGL_RELU, false>(a, st);
  }
}
template <bool BF>
cudaError_t gl_few(const GlFewArgs& a, cudaStream_t st) {
  using namespace gl;
  switch (a.activation) {
    case DGL_SILU: return few_of<BF, DGL_SILU>(a, st);
    case DGL_GELU: return few_of<BF, DGL_GELU>(a, st);
    case DGL_GELU_TANH: return few_of<BF, DGL_GELU_TANH>(a, st);
    default: return few_of<BF, DGL_RELU>(a, st);
  }
}
template <bool BF>
cudaError_t gl_dx(const GlArgs& a, cudaStream_t st) {
  static DeviceOnce once;
  return gl::launch_pairs(once, gl::gl_dx_kernel<BF>, (int64_t)((a.T + 255) / 256) * ((a.D + 255) / 256), a, st);
}
template <bool BF>
cudaError_t gl_dw(const GlArgs& a, cudaStream_t st) {
  static DeviceOnce once;
  return gl::launch_pairs(once, gl::gl_dw_kernel<BF>, (int64_t)2 * ((a.F + 255) / 256) * ((a.D + 255) / 256), a, st);
}
template <bool BF>
cudaError_t gl_scale(const GlScaleArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.T * a.F / 8 + 255) / 256;
  if (blocks == 0) return cudaSuccess;
  gl::gl_scale_kernel<BF><<<(int)(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace detattn
