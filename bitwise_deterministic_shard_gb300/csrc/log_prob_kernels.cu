// Log probabilities of given tokens, the entropy and the most likely alternatives of each row of logits, and the
// gradient of the first two.
//
//   z = x / temperature;  lse = log sum exp z;  lp = z_target - lse;  H = lse - sum p z,  p = exp(z - lse)
//   dx_v = (a (1[v = target] - p_v) - b p_v (log p_v + H)) / temperature,  a = dL/dlp, b = dL/dH
//
// In log2 units with c = log2(e) / temperature, a reference M and t_v = fma(x_v, c, -M), one pass gives
//   S = sum 2^t,  E = sum 2^t t,  lp = (t_target - log2 S) ln 2,  H = ln S - ln 2 E / S;
// M is the rounded c max(x), and whatever its rounding, it is the same in every term and cancels.  M and S go to the gradient,
// where dx_v = 2^t (A + B t) + [v = target] a / temperature with A and B of the row: one product more than the softmax's own.
//
// What bounds it: HBM; x is read once, and once more and dx written in the gradient.  A round of 8 vectors of 16 bytes a
// thread stays in registers: its maximum, then (the reference moved where that is larger) its terms.
//
// Alternatives: the first round's maxima of single threads give a value that at least `top` elements of the row reach (each of the
// CTA's warps finds its ceil(top / warps)-th largest, the least of them is that value); what reaches it, a few hundred elements
// of a large row, is collected in shared memory, and one warp takes the largest `top` of that, equal ones by their index.
// Rows that go on growing fill the list; it is then cut to its `top` largest, which raises the value, and where even a
// round's own candidates do not fit they are taken again above the `top`-th largest of the threads' best, of which there are
// at most 64 top.
//
// A row is one CTA's; short rows a warp's; where few rows would leave SMs idle, a cluster's, whose parts the first CTA joins through
// distributed shared memory.  The order of the sums depends on the sizes, the type and what starts on 16 bytes.
#include <algorithm>

#include "../../include/detattn.h"
#include "decoder_kernels.h"
#include "tc5_tile.cuh"
#include "train_math.cuh"

namespace detattn {
namespace {

using f2::u64;
using tc5::ex2;

constexpr int NV = 8;                  // vectors of a thread in a round
constexpr float LN2 = 0.6931471805599453f;
constexpr float FAR = -1000.f;         // t of a probability of zero: 2^t t is 0 there and not NaN

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// orders like the value, -0 as +0
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }
// larger values first, then lower indices
__device__ __forceinline__ u64 key_of(float x, uint32_t index) { return (u64)ordered(x) << 32 | (uint32_t)~index; }

template <typename T>
__device__ __forceinline__ T lowest() {   // -inf
  if constexpr (sizeof(T) == 4) return -INFINITY;
  else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __ushort_as_bfloat16(0xFF80);
  else return __ushort_as_half(0xFC00);
}
template <typename T, int N>
__device__ __forceinline__ float largest(const Run<T, N>& r) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(r.get(0), r.get(1)), fmaxf(r.get(2), r.get(3)));
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const auto h = [&](int i) { return *reinterpret_cast<const __nv_bfloat162*>(&r.w[i]); };
    const __nv_bfloat162 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    const auto h = [&](int i) { return *reinterpret_cast<const __half2*>(&r.w[i]); };
    const __half2 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
    return fmaxf(__low2float(m), __high2float(m));
  }
}
// vector v of a row whose vectors start `off` elements before it: 16 bytes at once where all of them are the row's, else
// element by element, -inf outside
template <typename T>
__device__ __forceinline__ void load_vector(Run<T, Elem<T>::VEC>& r, const T* row, int64_t first, uint32_t cols) {
  constexpr int VEC = Elem<T>::VEC;
  if (first >= 0 && first + VEC <= cols) {
    r.load(row + first);
  } else {
    r.zero();
#pragma unroll
    for (int e = 0; e < VEC; e++) r.put_bits(e, first + e >= 0 && first + e < cols ? row[first + e] : lowest<T>());
  }
}

struct Sums {   // reference (log2 units), sum of 2^t, sum of 2^t t
  float M, S, E;
  __device__ __forceinline__ void to(float m) {   // m >= M
    if (m == M) return;
    const float d = M - m, k = M == -INFINITY ? 0.f : ex2(d);
    E = M == -INFINITY ? E : k * __fmaf_rn(d, S, E);   // a NaN stays
    S = M == -INFINITY ? S : k * S;
    M = m;
  }
  __device__ __forceinline__ void join(Sums o) {
    const float m = fmaxf(M, o.M);
    to(m);
    o.to(m);
    S += o.S;
    E += o.E;
  }
};

template <int W>
struct Shared {
  static constexpr int CAP = W == 1 ? 2048 : 4096;   // a warp's only round is never more
  u64 cand[CAP];
  u64 best[32 * W];
  u64 list[LP_TOP];
  uint32_t count, warps[W];
  u64 above;
  Sums sums[W];
};

// The largest n of the first `have` keys of `from`, in order, to `to`; by one whole warp.
__device__ __forceinline__ void select_largest(u64* from, int have, u64* to, int n) {
  const int lane = threadIdx.x & 31;
  u64 mine = 0;
  int at = -1;
  const auto scan = [&] {
    mine = 0;
    at = -1;
    for (int i = lane; i < have; i += 32)
      if (from[i] > mine) {
        mine = from[i];
        at = i;
      }
  };
  scan();
  for (int j = 0; j < n; j++) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
    const u64 top = (u64)hi << 32 | lo;
    if (lane == 0) to[j] = top;
    if (top != 0 && mine == top) {   // keys differ, so one lane
      from[at] = 0;
      scan();
    }
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ u64 peer_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float peer_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// W warps a CTA; parts: CTAs (a cluster) of a row
template <typename T, int W, bool TOP>
__global__ void __launch_bounds__(32 * W, W == 8 ? 3 : 16) lp_kernel(const __grid_constant__ LpArgs a, int parts) {
  constexpr int VEC = Elem<T>::VEC, G = 32 * W;
  __shared__ std::conditional_t<TOP, Shared<W>, Sums[W]> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t r = blockIdx.x / (uint32_t)parts;
  const uint32_t part = blockIdx.x % (uint32_t)parts;
  const T* const row = static_cast<const T*>(a.x) + r * a.xs;
  const int64_t target = a.targets[r];
  const float at_target = tid == 0 && target >= 0 && target < a.cols ? Elem<T>::get(row[target]) : 0.f;
  const float c = (float)(1.4426950408889634 / (double)a.temperature);

  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const uint32_t nv = (a.cols + off + VEC - 1) / VEC, per = (nv + parts - 1) / parts;
  const uint32_t v0 = min(nv, part * per), v1 = min(nv, v0 + per);

  float top_x = -INFINITY, M = -INFINITY;   // this thread's largest element, and its reference
  u64 S2 = 0, E2 = 0;
  float reach = -INFINITY;                  // elements below it are no candidates
  if constexpr (TOP) {
    if (tid == 0) sh.count = 0;
    __syncthreads();
  }
  for (uint32_t v = v0; v < v1; v += NV * G) {
    Run<T, VEC> x[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t at = v + i * G + tid;
      if (at < v1) load_vector(x[i], row, (int64_t)at * VEC - off, a.cols);
      else {
        x[i].zero();
#pragma unroll
        for (int e = 0; e < VEC; e++) x[i].put_bits(e, lowest<T>());
      }
    }
    float big = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; i++) big = fmaxf(big, largest(x[i]));
    if (big > top_x) {
      top_x = big;
      float s0, s1, e0, e1;
      f2::unpack(S2, s0, s1);
      f2::unpack(E2, e0, e1);
      Sums lo = {M, s0, e0}, hi = {M, s1, e1};
      M = big * c;
      lo.to(M);
      hi.to(M);
      S2 = f2::pack(lo.S, hi.S);
      E2 = f2::pack(lo.E, hi.E);
    }
    const u64 cc = f2::splat(c), mm = f2::splat(M == -INFINITY ? 0.f : -M);
#pragma unroll
    for (int i = 0; i < NV; i++) {
#pragma unroll
      for (int e = 0; e < VEC / 2; e++) {
        float t0, t1;
        f2::unpack(f2::fma(x[i].get2(e), cc, mm), t0, t1);
        t0 = max_nan(t0, FAR);
        t1 = max_nan(t1, FAR);
        const u64 p = f2::pack(ex2(t0), ex2(t1));
        S2 = f2::add(S2, p);
        E2 = f2::fma(p, f2::pack(t0, t1), E2);
      }
    }
    if constexpr (TOP) {
      using Sh = Shared<W>;
      if (v == v0) {   // a value that at least `top` elements reach
        const int need = (a.top + W - 1) / W;
        uint32_t o = ordered(big), least = 0;
        for (int j = 0; j < need; j++) {
          least = __reduce_max_sync(0xffffffffu, o);
          const uint32_t who = __ballot_sync(0xffffffffu, o == least);
          if (lane == __ffs(who) - 1) o = 0;
        }
        if (lane == 0) sh.warps[warp] = least;
        __syncthreads();
        least = sh.warps[0];
#pragma unroll
        for (int w = 1; w < W; w++) least = min(least, sh.warps[w]);
        reach = least <= ordered(-INFINITY) ? -INFINITY : value_of(least);
      }
      const auto each = [&](auto f) {   // this round's elements, those of the row
#pragma unroll
        for (int i = 0; i < NV; i++) {
          const uint32_t at = v + i * G + tid;
          const int64_t first = (int64_t)at * VEC - off;
          if (at < v1 && largest(x[i]) >= reach)
#pragma unroll
            for (int e = 0; e < VEC; e++)
              if (first + e >= 0 && first + e < a.cols) f(x[i].get(e), (uint32_t)(first + e));
        }
      };
      bool full = false;
      if (big >= reach)
        each([&](float y, uint32_t index) {
          if (y >= reach) {
            const uint32_t slot = atomicAdd(&sh.count, 1u);
            if (slot < Sh::CAP) sh.cand[slot] = key_of(y, index);
            full |= slot >= 2048;
          }
        });
      if (W > 1 && __syncthreads_or(full)) {   // the same in all threads
        const uint32_t count = sh.count, have = min(count, (uint32_t)Sh::CAP);
        if (warp == 0) select_largest(sh.cand, have, sh.list, a.top);
        __syncthreads();
        if (tid < a.top) sh.cand[tid] = sh.list[tid];
        if (tid == 0) {
          sh.count = a.top;
          sh.above = sh.list[a.top - 1];
        }
        __syncthreads();
        u64 above = sh.above;
        if (count > Sh::CAP) {
          u64 best = 0;
          if (big >= reach) each([&](float y, uint32_t index) { best = max(best, key_of(y, index)); });
          sh.best[tid] = best;
          __syncthreads();
          int rank = 0;
          for (int j = 0; j < G; j++) rank += sh.best[j] > best || (sh.best[j] == best && j < tid);
          if (rank == a.top - 1 && best > above) sh.above = best;
          __syncthreads();
          above = sh.above;
          if (best >= above && best != 0)
            each([&](float y, uint32_t index) {
              const u64 key = key_of(y, index);
              bool more = key >= above;
              for (int j = 0; j < a.top && more; j++) more = sh.list[j] != key;
              if (more) {
                const uint32_t slot = atomicAdd(&sh.count, 1u);
                if (slot < Sh::CAP) sh.cand[slot] = key;   // there are at most `top` and 64 top
              }
            });
          __syncthreads();
        }
        reach = value_of((uint32_t)(above >> 32) + 1);   // an equal one of a later round has a larger index
        if (reach != reach) reach = INFINITY;
      }
    }
  }

  float s0, s1, e0, e1;
  f2::unpack(S2, s0, s1);
  f2::unpack(E2, e0, e1);
  Sums m = {M, s0 + s1, e0 + e1};
#pragma unroll
  for (int o = 16; o; o >>= 1) {   // the lower lane's sums first, so that both get the same bits
    Sums u = {__shfl_xor_sync(0xffffffffu, m.M, o), __shfl_xor_sync(0xffffffffu, m.S, o), __shfl_xor_sync(0xffffffffu, m.E, o)};
    if (lane & o) {
      const Sums t = m;
      m = u;
      u = t;
    }
    m.join(u);
  }
  Sums* sums;
  if constexpr (TOP) sums = sh.sums;
  else sums = sh;
  if (lane == 0) sums[warp] = m;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < W; w++) m.join(sums[w]);
    if constexpr (TOP) select_largest(sh.cand, min(sh.count, (uint32_t)Shared<W>::CAP), sh.list, a.top);
  }
  if (parts > 1) {
    if (tid == 0) sums[0] = m;
    cluster_sync();
    if (part == 0 && warp == 0) {
      const uint32_t mine = tc5::smem_addr(&sums[0]);
      for (int p = 1; p < parts; p++) {
        const uint32_t at = peer(mine, p);
        m.join(Sums{peer_f32(at), peer_f32(at + 4), peer_f32(at + 8)});
      }
      if constexpr (TOP) {
        const uint32_t list = tc5::smem_addr(&sh.list[0]);
        if (lane < a.top)
          for (int p = 0; p < parts; p++) sh.cand[p * a.top + lane] = peer_u64(peer(list, p) + 8 * lane);
        __syncwarp();
        select_largest(sh.cand, parts * a.top, sh.list, a.top);
      }
    }
    cluster_sync();   // the parts stay until they are read
    if (part != 0) return;
  }
  if (warp != 0) return;
  const bool none = m.S == 0.f;                             // every logit is -inf
  const float log_s = none ? 0.f : log2f(m.S);
  if (lane == 0) {
    float lp = 0.f;
    if (target >= (int64_t)a.cols) {
      lp = __uint_as_float(0x7fffffffu);
      if (a.status) atomicOr(a.status, DA_STATUS_BAD_TARGET);
    } else if (target >= 0) {
      lp = none ? -INFINITY : (__fmaf_rn(at_target, c, -m.M) - log_s) * LN2;
    }
    a.lp[r] = lp;
    const float entropy = none ? 0.f : (log_s - m.E / m.S) * LN2;
    a.entropy[r] = entropy;
    if (a.stats) {
      a.stats[3 * r] = m.M;
      a.stats[3 * r + 1] = m.S;
      a.stats[3 * r + 2] = entropy;
    }
    if (!isfinite(m.S) && a.status) atomicOr(a.status, DA_STATUS_NONFINITE);
  }
  if constexpr (TOP) {
    if (lane < a.top) {
      const u64 key = sh.list[lane];
      const float y = value_of((uint32_t)(key >> 32));
      a.top_lp[r * a.top + lane] = none || y == -INFINITY ? -INFINITY : (__fmaf_rn(y, c, -m.M) - log_s) * LN2;
      a.top_index[r * a.top + lane] = (int64_t)(uint32_t)~(uint32_t)key;
    }
  }
}

// ---- gradient: a CTA a run of LG_RUN vectors of a row ----
constexpr int LG_U = 4, LG_RUN = 256 * LG_U;

template <typename T>
__global__ void __launch_bounds__(256) lp_grad_kernel(const __grid_constant__ LpGradArgs a, uint32_t runs) {
  constexpr int VEC = Elem<T>::VEC;
  const int64_t r = blockIdx.x / runs;
  const uint32_t run = blockIdx.x % runs;
  const T* const row = static_cast<const T*>(a.x) + r * a.xs;
  T* const out = static_cast<T*>(a.dx) + r * a.ds;
  const float c = (float)(1.4426950408889634 / (double)a.temperature), back = 1.f / a.temperature;
  const float M = a.stats[3 * r], S = a.stats[3 * r + 1], H = a.stats[3 * r + 2];
  const int64_t target = a.targets[r];
  const float g = a.grad && target >= 0 && target < (int64_t)a.cols ? a.grad[r] : 0.f, h = a.grad_entropy ? a.grad_entropy[r] : 0.f;
  const bool none = S == 0.f;
  const float inv = none ? 0.f : back / S, log_s = none ? 0.f : log2f(S);
  const float A = -(g + h * __fmaf_rn(-LN2, log_s, H)) * inv, B = -h * LN2 * inv;
  const float hit = none ? 0.f : g * back;
  const u64 cc = f2::splat(c), mm = f2::splat(none ? 0.f : -M), aa = f2::splat(A), bb = f2::splat(B);

  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const bool along = off == (int)((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));   // both start alike
  const int64_t base = ((int64_t)run * LG_RUN + threadIdx.x) * VEC - off;
  Run<T, VEC> x[LG_U];
#pragma unroll
  for (int i = 0; i < LG_U; i++) {
    const int64_t first = base + (int64_t)i * 256 * VEC;
    x[i].zero();
    if (first < a.cols) load_vector(x[i], row, first, a.cols);
  }
#pragma unroll
  for (int i = 0; i < LG_U; i++) {
    const int64_t first = base + (int64_t)i * 256 * VEC;
    if (first >= a.cols) break;
    float v[VEC];
#pragma unroll
    for (int e = 0; e < VEC / 2; e++) {
      float t0, t1;
      f2::unpack(f2::fma(x[i].get2(e), cc, mm), t0, t1);
      t0 = max_nan(t0, FAR);
      t1 = max_nan(t1, FAR);
      f2::unpack(f2::mul(f2::pack(ex2(t0), ex2(t1)), f2::fma(bb, f2::pack(t0, t1), aa)), v[2 * e], v[2 * e + 1]);
    }
    if (target >= first && target < first + VEC) {
#pragma unroll
      for (int e = 0; e < VEC; e++) v[e] += target == first + e ? hit : 0.f;
    }
    Run<T, VEC> o;
    o.set(v);
    if (along && first >= 0 && first + VEC <= a.cols) {
      o.store(out + first);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; e++)
        if (first + e >= 0 && first + e < a.cols) out[first + e] = o.bits(e);
    }
  }
}

template <typename T, int W>
cudaError_t forward(const LpArgs& a, int parts, cudaStream_t st) {
  cudaLaunchConfig_t config = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  config.gridDim = dim3((unsigned)(a.rows * parts));
  config.blockDim = dim3(32 * W);
  config.stream = st;
  config.attrs = attr;
  config.numAttrs = parts > 1 ? 1 : 0;
  return a.top ? cudaLaunchKernelEx(&config, lp_kernel<T, W, true>, a, parts)
               : cudaLaunchKernelEx(&config, lp_kernel<T, W, false>, a, parts);
}
template <typename T>
cudaError_t forward(const LpArgs& a, cudaStream_t st) {
  const int64_t vectors = (a.cols + Elem<T>::VEC - 1) / Elem<T>::VEC;
  if (vectors + 1 <= 32 * NV) return forward<T, 1>(a, 1, st);   // one round of a warp, wherever the row starts
  // parts of a row: as many as keep at most two CTAs an SM, and a round's vectors in each
  int parts = 1;
  while (parts < 8 && a.rows * parts * 2 <= 304 && vectors >= (int64_t)parts * 2 * 256 * NV / 2) parts *= 2;
  return forward<T, 8>(a, parts, st);
}
template <typename T>
cudaError_t backward(const LpGradArgs& a, cudaStream_t st) {
  const uint32_t runs = (uint32_t)(((int64_t)a.cols + 2 * Elem<T>::VEC - 2) / Elem<T>::VEC + LG_RUN - 1) / LG_RUN;
  lp_grad_kernel<T><<<(unsigned)(a.rows * runs), 256, 0, st>>>(a, runs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_log_probs(const LpArgs& a, cudaStream_t st) {
  if (a.dtype == DA_F32) return forward<float>(a, st);
  return a.dtype == DA_BF16 ? forward<__nv_bfloat16>(a, st) : forward<__half>(a, st);
}
cudaError_t launch_log_probs_grad(const LpGradArgs& a, cudaStream_t st) {
  if (a.dtype == DA_F32) return backward<float>(a, st);
  return a.dtype == DA_BF16 ? backward<__nv_bfloat16>(a, st) : backward<__half>(a, st);
}

}  // namespace detattn
