// The gated feed-forward projections and their gradient.
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u
//   dg = dh p,  du = dh q,  p = act'(g) u,  q = act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// Forward: one kernel of pair products (gemm_pair.cuh).  Half the rows of its second operand are rows of Wg (one CTA's half)
// and the other half the same rows of Wu, so g and u of a token and hidden unit lie in one TMEM lane, half a tile apart,
// and a thread forms h from them.  For the backward pass it also writes p and q, the only values of the activation that the
// gradient needs: each rounded to 24 bits (2^-16 of the value at most), as 16 would add a rounding of the size of the result's own to dg
// and du (dx then 2.9e-3 off in bf16 instead of 2.35e-3; 1.66e-3 is a result only rounded).
// Backward: dg and du as one pass over dh, p and q, rounded to 16 bits (the tensor cores take operands of one 16-bit type), then one
// kernel of pair products: dx contracts over both halves of [dg | du] in one chain, dW has the tiles of both weights; the
// longer tiles come first and the shorter ones fill the pairs up.
//
// What bounds them: the tensor cores, busy 94 % (forward), 87 % (forward with factors) and 97 % (backward) of the cycles; 4096 tokens, width
// 4096, 12288 hidden units, bf16: 449 us alone (1.84 PFLOP/s), 488 in a row of calls under the power limit; 8192 tokens, width 2048,
// 8192 hidden units with gradient: 317 us, 127 (dg and du, 6.3 TB/s) and 587 (1.87 PFLOP/s).
// Up to 16 tokens the forward pass (without factors) reads the weights once with plain loads instead.
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
// Phi(g) = erfc(-g / sqrt 2) / 2, by erfc(z) = t 2^(P(t) - z^2 log2 e) for z >= 0, t = 2 / (2 + z): P of degree 9, fitted to log2(erfc(z)
// e^(z^2) / t) for the least greatest error (7.5e-8 of the value, so the tail keeps its digits; least squares with weights moved
// toward the largest errors).  The form t e^(polynomial in t - z^2) is published in Press, Teukolsky, Vetterling and Flannery, Numerical
// Recipes, section 6.2; the coefficients here are the fit's own.  CUDA's normcdff has branches and made the kernel wait for its results: 8192 hidden units, width
// 2048, 4096 tokens 190 us, the products alone 144.
__device__ __forceinline__ float normal_cdf(float g) {
  const float t = rcp(__fmaf_rn(0.35355339059f, fabsf(g), 1.f));
  float p = __fmaf_rn(0x1.0202b8p-2f, t, -0x1.363d26p+0f);
  p = __fmaf_rn(p, t, 0x1.19707ep+1f);
  p = __fmaf_rn(p, t, -0x1.b18d14p+0f);
  p = __fmaf_rn(p, t, 0x1.c0f0d6p-2f);
  p = __fmaf_rn(p, t, -0x1.21a9b2p-2f);
  p = __fmaf_rn(p, t, 0x1.249cb4p-3f);
  p = __fmaf_rn(p, t, 0x1.141e74p-1f);
  p = __fmaf_rn(p, t, 0x1.71583ap+0f);
  p = __fmaf_rn(p, t, -0x1.d36442p+0f);
  const float e = 0.5f * t * ex2(__fmaf_rn(-0.5f * LOG2E * g, g, p));
  return g < 0.f ? e : 1.f - e;
}
template <int ACT>
__device__ __forceinline__ void activate(float g, float& a, float& d) {
  if constexpr (ACT == DGL_SILU) {
    const float s = logistic(g);
    a = g * s;
    d = s * __fmaf_rn(g, 1.f - s, 1.f);
  } else if constexpr (ACT == DGL_GELU) {
    const float s = normal_cdf(g);
    a = g * s;
    d = __fmaf_rn(g * 0.3989422804014327f, ex2(-0.5f * LOG2E * g * g), s);
  } else if constexpr (ACT == DGL_GELU_TANH) {
    constexpr float c = 0.7978845608028654f, k = 0.044715f;
    const float g2 = g * g;
    const float s = logistic(2.f * c * g * __fmaf_rn(k, g2, 1.f));
    a = g * s;
    const float b = fminf(fmaxf(g, -16.f), 16.f);   // past these s is 0 or 1, and y' may be infinite
    d = s * __fmaf_rn(2.f * c * b * __fmaf_rn(3.f * k, b * b, 1.f), 1.f - s, 1.f);
  } else {
    a = g > 0.f ? g : g != g ? g : 0.f;
    d = g > 0.f ? 1.f : g != g ? g : 0.f;
  }
}

// copies of N boxes of 64 rows from row r on, contracted elements [k, k + 64): K-major
template <int N>
__device__ __forceinline__ void copy_k(uint32_t to, const CUtensorMap* m, int k, int r, uint32_t bar, uint32_t one) {
#pragma unroll
  for (int i = 0; i < N; i++) pair::load2(to + i * pair::BOX, m, k, r + 64 * i, bar, one);
}
// and of N panels of 64 columns from c on: MN-major
template <int N>
__device__ __forceinline__ void copy_mn(uint32_t to, const CUtensorMap* m, int k, int c, uint32_t bar, uint32_t one) {
#pragma unroll
  for (int i = 0; i < N; i++) pair::load2(to + i * pair::BOX, m, c + 64 * i, k, bar, one);
}

// ---- forward ----
// Results are staged in shared memory, here 32 columns of h and the factors at a time, and written 64 bytes a row by neighbouring lanes: a
// lane that wrote its own row's pieces would touch 32 lines an instruction (8192 tokens, width 2048, 8192 hidden units: 555 us; the
// products alone take 300).
template <bool SAVE>
constexpr int STAGED = SAVE ? pair::TAKERS * 4096 : 0;   // bytes

// 32 rows of 8 units of 16 bytes, unit u of row r at u ^ (r % 8)
__device__ __forceinline__ void stage_put(uint32_t stage, int r, int u, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + r * 128 + ((u ^ (r & 7)) << 4)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 stage_get(uint32_t stage, int r, int u) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(stage + r * 128 + ((u ^ (r & 7)) << 4))
               : "memory");
  return v;
}
// v rounded to the nearest 24-bit value, but for its low byte, which is left out later; ties away from zero.  (Cut off instead, all
// factors would be too small, by up to 2^-15.)  What would become an infinity, infinities and NaN stay as they are.
__device__ __forceinline__ float nearest_24(float v) {
  const uint32_t b = __float_as_uint(v);
  return __uint_as_float((b & 0x7fffffffu) < 0x7f7fff80u ? b + 0x80u : b);
}
// the high halves of 8 binary32 values; the bytes below them of 16
__device__ __forceinline__ uint4 high_halves(const float* v) {
  const auto two = [&](int i) { return __byte_perm(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), 0x7632); };
  return make_uint4(two(0), two(2), two(4), two(6));
}
__device__ __forceinline__ uint4 next_bytes(const float* v) {
  const auto four = [&](int i) {
    return __byte_perm(__byte_perm(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), 0x0051),
                       __byte_perm(__float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]), 0x0051), 0x5410);
  };
  return make_uint4(four(0), four(4), four(8), four(12));
}

template <bool BF, int ACT, bool SAVE, int TN>
__global__ void __launch_bounds__(pair::THREADS, 1) __cluster_dims__(2, 1, 1) gl_fwd_kernel(const __grid_constant__ GlArgs a) {
  using namespace tc5;
  extern __shared__ unsigned char raw[];
  __shared__ pair::Shared sh;
  constexpr int HALF = TN / 2;
  const int mt = (a.T + 255) / 256, nt = (a.F + HALF - 1) / HALF, steps = (a.D + pair::BK - 1) / pair::BK;
  const uint32_t rank = tc5::same(pair::cta_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CUtensorMap* const w = rank ? &a.wu : &a.wg;
  pair::run<BF, TN, STAGED<SAVE>, false>(
      sh, raw, a.status,
      [&](int j) {
        const int t = (int)(blockIdx.x >> 1) + j * (int)(gridDim.x >> 1);
        return t < mt * nt ? pair::tile_of(t, mt, nt, 0, steps) : pair::Tile{0, 0, 0, 0};
      },
      [](int) { return false; },
      [&](const pair::Tile& t, int k, uint32_t A, uint32_t B, uint32_t bar, uint32_t one) {
        copy_k<2>(A, &a.x, k * pair::BK, t.m * 256 + rank * 128, bar, one);
        copy_k<HALF / 64>(B, w, k * pair::BK, t.n * HALF, bar, one);
      },
      [&](const pair::Tile& t, uint32_t tm, uint32_t extra, auto release) {
        const int row0 = t.m * 256 + rank * 128 + (warp & 3) * 32, row = row0 + lane;
        const uint32_t stage = extra + warp * 4096;
        uint16_t* const h = static_cast<uint16_t*>(a.h);
        const int64_t fp = gl_saved_row(a.F), n = a.T * fp;
#pragma unroll
        for (int c = 0; c < HALF / 2; c += 32) {
          const int cc = (warp >> 2) * (HALF / 2) + c, col = t.n * HALF + cc;   // columns of the tile and of h
          float g[32], u[32];
          __syncwarp();   // the loads are the whole warp's
          ld_x32(tm + cc, g);
          ld_x32(tm + HALF + cc, u);
          ld_wait();
          if (c == HALF / 2 - 32) release();
          if (row0 >= a.T || col >= a.F) continue;   // the same in all lanes
          float q[32];
#pragma unroll
          for (int e = 0; e < 32; e++) {
            float d;
            activate<ACT>(g[e], q[e], d);
            g[e] = q[e] * u[e];
            u[e] *= d;
            if constexpr (SAVE) {
              q[e] = nearest_24(q[e]);
              u[e] = nearest_24(u[e]);
            }
          }
          const auto units = [&](int j) {
            return make_uint4(pack16<BF>(g[8 * j], g[8 * j + 1]), pack16<BF>(g[8 * j + 2], g[8 * j + 3]),
                              pack16<BF>(g[8 * j + 4], g[8 * j + 5]), pack16<BF>(g[8 * j + 6], g[8 * j + 7]));
          };
          if constexpr (SAVE) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
              stage_put(stage, lane, j, units(j));
              stage_put(stage, lane, 4 + j, high_halves(u + 8 * j));
            }
            __syncwarp();
            const int un = lane & 7, at = col + (un & 3) * 8;
#pragma unroll
            for (int it = 0; it < 8; it++) {
              const int r = it * 4 + (lane >> 3);
              const uint4 v = stage_get(stage, r, un);
              if (row0 + r < a.T && at < a.F) {
                if (un < 4) *reinterpret_cast<uint4*>(h + (row0 + r) * a.hs + at) = v;
                else *reinterpret_cast<uint4*>(a.saved + 2 * ((row0 + r) * fp + at)) = v;
              }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; j++) stage_put(stage, lane, j, high_halves(q + 8 * j));
#pragma unroll
            for (int j = 0; j < 2; j++) {
              stage_put(stage, lane, 4 + j, next_bytes(u + 16 * j));
              stage_put(stage, lane, 6 + j, next_bytes(q + 16 * j));
            }
            __syncwarp();
            const int lo = col + (un & 1) * 16;
#pragma unroll
            for (int it = 0; it < 8; it++) {
              const int r = it * 4 + (lane >> 3);
              const uint4 v = stage_get(stage, r, un);
              if (row0 + r < a.T) {
                if (un < 4) {
                  if (at < a.F) *reinterpret_cast<uint4*>(a.saved + 2 * (n + (row0 + r) * fp + at)) = v;
                } else if (lo < a.F) {
                  *reinterpret_cast<uint4*>(a.saved + 4 * n + (un < 6 ? 0 : n) + (row0 + r) * fp + lo) = v;
                }
              }
            }
          } else if (row < a.T) {
#pragma unroll
            for (int j = 0; j < 4; j++)
              if (col + 8 * j < a.F) *reinterpret_cast<uint4*>(h + row * a.hs + col + 8 * j) = units(j);
          }
        }
      });
}

// ---- backward: dx [T, D] = [dg | du] [Wg; Wu] (dg, du K-major), dW [F, D] = dg^T x and du^T x (dg, du MN-major) ----
// Of na long and nb short tiles, how many steps: each pair takes every P-th long one; the pairs that this leaves short take
// short ones until they are level (q each), then all pairs do by turns.
struct Shares {
  int na, nb, q;
};
__device__ __forceinline__ int share(const Shares& s, int j, int p, int P) {   // the pair's j-th tile, -1: none
  const int r = s.na % P, mine = s.na / P + (p < r);
  if (j < mine) return j * P + p;
  j -= mine;
  int k;
  if (r == 0) k = j * P + p;
  else if (p < r) k = s.q * (P - r) + j * P + P - r + p;
  else if (j < s.q) k = j * (P - r) + p - r;
  else k = s.q * (P - r) + (j - s.q) * P + p - r;
  return k < s.nb ? s.na + k : -1;
}

enum { DX = 0, DW = 1 };
template <bool BF, int TN>
__global__ void __launch_bounds__(pair::THREADS, 1) __cluster_dims__(2, 1, 1) gl_bwd_kernel(const __grid_constant__ GlArgs a) {
  using namespace tc5;
  extern __shared__ unsigned char raw[];
  __shared__ pair::Shared sh;
  const int tt = (a.T + 255) / 256, ft = (a.F + 255) / 256, nt = (a.D + TN - 1) / TN, half = (a.F + pair::BK - 1) / pair::BK;
  const int nx = a.dx ? tt * nt : 0, nw = a.dwg ? 2 * ft * nt : 0, sx = 2 * half, sw = (a.T + pair::BK - 1) / pair::BK;
  const bool x_first = sx >= sw;
  const Shares shares = x_first ? Shares{nx, nw, sx / sw} : Shares{nw, nx, sw / sx};
  const uint32_t rank = tc5::same(pair::cta_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pair::run<BF, TN, STAGED<true>, true>(
      sh, raw, a.status,
      [&](int j) {
        const int t = share(shares, j, blockIdx.x >> 1, gridDim.x >> 1);
        if (t < 0) return pair::Tile{0, 0, 0, 0};
        const bool first = t < shares.na;
        const int i = first ? t : t - shares.na;
        return first == x_first ? pair::tile_of(i, tt, nt, DX, sx) : pair::tile_of(i, 2 * ft, nt, DW, sw);
      },
      [](int kind) { return kind == DW; },
      [&](const pair::Tile& t, int k, uint32_t A, uint32_t B, uint32_t bar, uint32_t one) {
        const int c = t.n * TN + rank * (TN / 2);
        if (t.kind == DX) {
          const bool u = k >= half;
          const int k0 = (u ? k - half : k) * pair::BK;
          copy_k<2>(A, u ? &a.du : &a.dg, k0, t.m * 256 + rank * 128, bar, one);
          copy_mn<TN / 128>(B, u ? &a.wu : &a.wg, k0, c, bar, one);
        } else {
          const bool u = t.m >= ft;
          copy_mn<2>(A, u ? &a.du : &a.dg, k * pair::BK, (u ? t.m - ft : t.m) * 256 + rank * 128, bar, one);
          copy_mn<TN / 128>(B, &a.x, k * pair::BK, c, bar, one);
        }
      },
      [&](const pair::Tile& t, uint32_t tm, uint32_t extra, auto release) {
        const bool u = t.kind == DW && t.m >= ft;
        const int row0 = (u ? t.m - ft : t.m) * 256 + rank * 128 + (warp & 3) * 32, rows = t.kind == DX ? a.T : a.F;
        uint16_t* const out = static_cast<uint16_t*>(t.kind == DX ? a.dx : u ? a.dwu : a.dwg);
        const int64_t stride = t.kind == DX ? a.dxs : u ? a.dwus : a.dwgs;
        const uint32_t stage = extra + warp * 4096;
        const int un = lane & 7;
#pragma unroll
        for (int c = 0; c < TN / 2; c += 64) {
          const int cc = (warp >> 2) * (TN / 2) + c, col = t.n * TN + cc;
          __syncwarp();   // the loads are the whole warp's
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            float v[32];
            ld_x32(tm + cc + h, v);
            ld_wait();
            if (c + h == TN / 2 - 32) release();
#pragma unroll
            for (int j = 0; j < 4; j++)
              stage_put(stage, lane, h / 8 + j,
                        make_uint4(pack16<BF>(v[8 * j], v[8 * j + 1]), pack16<BF>(v[8 * j + 2], v[8 * j + 3]),
                                   pack16<BF>(v[8 * j + 4], v[8 * j + 5]), pack16<BF>(v[8 * j + 6], v[8 * j + 7])));
          }
          __syncwarp();
#pragma unroll
          for (int it = 0; it < 8; it++) {
            const int r = it * 4 + (lane >> 3);
            const uint4 v = stage_get(stage, r, un);
            if (row0 + r < rows && col + un * 8 < a.D) *reinterpret_cast<uint4*>(out + (row0 + r) * stride + col + un * 8) = v;
          }
        }
      });
}

// ---- few tokens: 1 to 8 warps for 8 hidden units ----
// Weights go from memory to registers once: a warp's products are of 16 rows (8 of Wg and the same 8 of Wu) by 8 tokens by 16, each
// lane holding 8 neighbouring elements of a row of each, and the same 8 of a token's x; which 16 of them one product
// contracts is free, as long as both operands agree.  A lane then has g and u of a unit for two tokens.  (Warp-wide products: at
// this size the reading of the weights bounds it, not the matrix rate.  Multiplying by single tokens on the FP32 pipe took 55 us for
// 4 and 98 for 8, width 4096, 12288 hidden units; the tiles of the other kernel 74 for 5 to 15 tokens, which all SMs read from the few
// slices of the L2 that hold so small an x.)
// As many warps as leave each up to eight runs of 32 elements a row.  One token, us (TB/s), one call after another with weights that the
// L2 does not hold: width 1024, 4096 hidden units 5.7 (2.9); 2048, 8192 13.5 (5.0); 4096, 12288 32.2 (6.3); 8192, 28672 136 (6.9): start
// and end of a launch, some 3 us, and the rest at the copy bandwidth.
template <typename R, typename T>
__device__ __forceinline__ void load_once(R& r, const T* p) {   // of a weight that no other warp reads
  asm("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "l"(p));
}
template <bool BF>
__device__ __forceinline__ void product(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool BF, int NT, int ACT>   // up to 8 NT tokens
__global__ void __launch_bounds__(256, 4) gl_few_kernel(const __grid_constant__ GlFewArgs a, int warps) {
  using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
  __shared__ float sums[8][NT][4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % warps, g = lane >> 2, t = lane & 3;
  const int f0 = (blockIdx.x * (8 / warps) + warp / warps) * 8;
  const bool live = f0 < a.F;
  const T* const wg = static_cast<const T*>(a.wg) + (live ? f0 + g : 0) * a.gs;
  const T* const wu = static_cast<const T*>(a.wu) + (live ? f0 + g : 0) * a.us;
  const T* x[NT];
  float c[NT][4];
#pragma unroll
  for (int n = 0; n < NT; n++) {
    x[n] = static_cast<const T*>(a.x) + min(8 * n + g, a.T - 1) * a.xs;   // tokens past the last: a copy of it, whose sums are not used
#pragma unroll
    for (int i = 0; i < 4; i++) c[n][i] = 0.f;
  }
  constexpr int U = 4;                                     // runs at once
  const int per = ((a.D + 32 * warps - 1) / (32 * warps)) * 32, k1 = min(a.D, (part + 1) * per);
  for (int k0 = part * per + t * 8; k0 < k1 + t * 8; k0 += 32 * U) {   // the same number of rounds in all lanes
    Run<T, 8> rg[U], ru[U];
#pragma unroll
    for (int i = 0; i < U; i++) {
      rg[i].zero();
      ru[i].zero();
      if (k0 + 32 * i < k1) {
        load_once(rg[i], wg + k0 + 32 * i);
        load_once(ru[i], wu + k0 + 32 * i);
      }
    }
#pragma unroll
    for (int i = 0; i < U; i++) {
#pragma unroll
      for (int n = 0; n < NT; n++) {
        Run<T, 8> rx;
        rx.zero();
        if (k0 + 32 * i < k1) rx.load(x[n] + k0 + 32 * i);
        __syncwarp();
        product<BF>(c[n], rg[i].w[0], ru[i].w[0], rg[i].w[1], ru[i].w[1], rx.w[0], rx.w[1]);
        product<BF>(c[n], rg[i].w[2], ru[i].w[2], rg[i].w[3], ru[i].w[3], rx.w[2], rx.w[3]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; n++)
#pragma unroll
    for (int i = 0; i < 4; i++) sums[warp][n][i][lane] = c[n][i];
  __syncthreads();
  if (part != 0 || !live) return;
#pragma unroll
  for (int n = 0; n < NT; n++)
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int token = 8 * n + 2 * t + i;
      float gs = 0.f, us = 0.f;
      for (int w = 0; w < warps; w++) {                    // in order
        gs += sums[warp + w][n][i][lane];
        us += sums[warp + w][n][2 + i][lane];
      }
      float q, d;
      activate<ACT>(gs, q, d);
      if (token < a.T) static_cast<T*>(a.h)[token * a.hs + f0 + g] = Elem<T>::put(q * us);
    }
}

// ---- dg = dh p, du = dh q: 8 elements a thread ----
template <bool BF>
__global__ void __launch_bounds__(256) gl_scale_kernel(const GlScaleArgs a) {
  using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
  const int64_t fp = gl_saved_row(a.F), n = a.T * fp, per = a.F / 8, all = a.T * per, dp = gl_grad_row(a.F);
  T* const dg = static_cast<T*>(a.dg);
  next_may_start();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, col = (i - row * per) * 8, at = row * fp + col;
    Run<T, 8> r;
    r.load(static_cast<const T*>(a.dh) + row * a.ds + col);
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const uint4 hi = *reinterpret_cast<const uint4*>(a.saved + 2 * (w * n + at));
      const uint2 lo = *reinterpret_cast<const uint2*>(a.saved + 4 * n + w * n + at);
      const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e++)   // bits 31..16 and 15..8
        v[e] = r.get(e) * __uint_as_float((h[e >> 1] >> (16 * (e & 1)) << 16) | ((e < 4 ? lo.x : lo.y) >> (8 * (e & 3)) & 255) << 8);
      Run<T, 8> o;
      o.set(v);
      o.store(dg + (w * a.T + row) * dp + col);
    }
  }
}

constexpr int PAIRS = 152 / 2;   // of the GPU this is written for: the choice of the tile, and with it no bit, depends on it

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <bool BF, int ACT, bool SAVE, int TN>
cudaError_t forward_as(const GlArgs& a, int64_t tiles, cudaStream_t st) {
  static DeviceOnce once;
  constexpr int smem = pair::Ring<TN, STAGED<SAVE>>::SMEM;
  const cudaError_t e = allow_smem(once, gl_fwd_kernel<BF, ACT, SAVE, TN>, smem);
  if (e != cudaSuccess) return e;
  gl_fwd_kernel<BF, ACT, SAVE, TN><<<2 * (unsigned)(tiles < PAIRS ? tiles : PAIRS), pair::THREADS, smem, st>>>(a);
  return cudaGetLastError();
}
// The tile: rounds of pairs times a tile's time.  A narrow one's is 0.7 of a wide one's (its products take half, its copies 0.75); where
// there is one row of tiles, and each weight comes from HBM for one pair, 0.55 (128 tokens, width 4096, 12288 hidden units: three
// rounds of narrow tiles 41 us, two of wide ones 50).
template <bool BF, int ACT, bool SAVE>
cudaError_t forward_of(const GlArgs& a, cudaStream_t st) {
  const int64_t mt = ceil_div(a.T, 256), wide = mt * ceil_div(a.F, 128), narrow = mt * ceil_div(a.F, 64);
  if (100 * ceil_div(wide, PAIRS) > (mt == 1 ? 55 : 70) * ceil_div(narrow, PAIRS)) return forward_as<BF, ACT, SAVE, 128>(a, narrow, st);
  return forward_as<BF, ACT, SAVE, 256>(a, wide, st);
}
template <bool BF, int TN>
cudaError_t backward_as(const GlArgs& a, int64_t tiles, cudaStream_t st) {
  static DeviceOnce once;
  constexpr int smem = pair::Ring<TN, STAGED<true>>::SMEM;
  const cudaError_t e = allow_smem(once, gl_bwd_kernel<BF, TN>, smem);
  if (e != cudaSuccess) return e;
  return launch_early(gl_bwd_kernel<BF, TN>, dim3(2 * (unsigned)(tiles < PAIRS ? tiles : PAIRS)), pair::THREADS, smem, st, a);
}
template <bool BF, int ACT>
cudaError_t few_of(const GlFewArgs& a, cudaStream_t st) {
  int warps = 1;
  while (warps < 8 && a.D > 256 * warps) warps *= 2;
  const int grid = (a.F / 8 + 8 / warps - 1) / (8 / warps);
  if (a.T <= 8) gl_few_kernel<BF, 1, ACT><<<grid, 256, 0, st>>>(a, warps);
  else gl_few_kernel<BF, 2, ACT><<<grid, 256, 0, st>>>(a, warps);
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
cudaError_t gl_backward(const GlArgs& a, cudaStream_t st) {
  using namespace gl;
  // steps of the pair with the most, at least those of the longest tile, for tiles of 256 and of 128 columns
  int64_t tiles[2], most[2];
  for (int i = 0; i < 2; i++) {
    const int64_t nt = ceil_div(a.D, i ? 128 : 256), nx = a.dx ? ceil_div(a.T, 256) * nt : 0, nw = a.dwg ? 2 * ceil_div(a.F, 256) * nt : 0;
    const int64_t sx = 2 * ceil_div(a.F, 64), sw = ceil_div(a.T, 64);
    const bool x = nx && (sx >= sw || !nw);
    tiles[i] = nx + nw;
    const int64_t even = ceil_div(nx * sx + nw * sw, PAIRS), first = x ? ceil_div(nx, PAIRS) * sx : ceil_div(nw, PAIRS) * sw;
    most[i] = even > first ? even : first;
  }
  return 10 * most[0] > 7 * most[1] ? backward_as<BF, 128>(a, tiles[1], st) : backward_as<BF, 256>(a, tiles[0], st);
}
template <bool BF>
cudaError_t gl_scale(const GlScaleArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.T * a.F / 8 + 255) / 256;
  if (blocks == 0) return cudaSuccess;
  gl::gl_scale_kernel<BF><<<(int)(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace detattn
