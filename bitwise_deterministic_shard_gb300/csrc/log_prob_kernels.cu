// Log probabilities of given tokens, the entropy and the most likely alternatives of each row of logits, and the
// gradient of the first two.
//
//   z = x / temperature;  lse = log sum exp z;  lp = z_target - lse;  H = lse - sum p z,  p = exp(z - lse)
//   dx_v = (a (1[v = target] - p_v) - b p_v (log p_v + H)) / temperature,  a = dL/dlp, b = dL/dH
//
// With c = log2(e) / temperature, m = max x and t_v = (x_v - m) c (the difference first: x may be as large, or as low, as its
// type allows), one pass gives
//   S = sum 2^t,  E = sum 2^t t,  lp = (x_target - m) / temperature - ln S,  H = ln S - ln 2 E / S.
// m, S and H go to the gradient, where dx_v = 2^t (A + B t) + [v = target] a / temperature with A and B of the row: one
// product more than the softmax's own.
//
// What bounds it: HBM; x is read once, and once more and dx written in the gradient.  A step of 4 vectors of 16 bytes a
// thread stays in registers: its maximum, then (the sums moved where that is larger) its terms, while the next step's
// loads are under way.  128256 columns: 4096 f32 rows 302 us (6.96 TB/s), with 5 alternatives 342; 8192 bf16 rows 327 to 343 us (6.13 to 6.43 TB/s;
// issue slots 62 %), with 5 alternatives 440 to 462; the gradient of these 629 us (6.68 TB/s).
//
// Alternatives: each warp keeps the largest few of its lanes' maxima, step by step; the `top`-th of all warps' is a value that at
// least `top` elements of the row reach.  What reaches it is kept in shared memory, some tens of elements of a large row; whenever
// a warp meets such an element it raises the value, so hardly any work is left once a part of the row is read.  A full list is
// shortened by the `top`-th of its parts' largest.  At the end the candidates that still reach the value are ranked by counting,
// equal ones by their index.  No barrier but the first step's and the last; which candidates are kept does not change the
// result.  (A value from each warp's ceil(top / warps)-th largest instead let ten times as many through: 4096 x 128256 f32, 5
// alternatives, 604 us against 312 without alternatives.)
//
// A row is one CTA's of one to eight warps; where few rows would leave SMs idle, a cluster's, whose parts hand their sums and
// lists to the first CTA through distributed shared memory.  The order of the sums depends on the sizes, the type and what
// starts on 16 bytes.
#include <algorithm>

#include "../../include/detattn.h"
#include "decoder_kernels.h"
#include "tc5_tile.cuh"
#include "train_math.cuh"

namespace detattn {
namespace {

using f2::u64;
using tc5::ex2;

constexpr int NV = 4;                  // vectors of a thread in a step
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

struct Sums {   // the largest element, sum of 2^t, sum of 2^t t
  float m, S, E;
  __device__ __forceinline__ void to(float top, float c) {   // top >= m
    if (top == m) return;
    const float d = m == -INFINITY ? 0.f : fmaxf((m - top) * c, FAR), k = ex2(d);
    E = k * __fmaf_rn(d, S, E);   // all are 0 (or NaN, which stays) where no element was above -inf
    S = k * S;
    m = top;
  }
  __device__ __forceinline__ void join(Sums o, float c) {
    const float top = fmaxf(m, o.m);
    to(top, c);
    o.to(top, c);
    S += o.S;
    E += o.E;
  }
};

constexpr int CAP = 256;               // candidates that a warp keeps

template <int W>
struct Shared {
  static constexpr int SEEN = 32 / W;  // of each warp: its largest elements so far that the common value is found from
  u64 cand[W][CAP];
  u64 all[W * CAP];
  u64 best[LP_TOP];
  u64 join[8][LP_TOP];                 // first CTA of a cluster: the parts' lists
  uint32_t seen[32];
  uint32_t reach, total;
};

// The value of rank k (from 0) of one value a lane, largest first.
__device__ __forceinline__ uint32_t of_rank(uint32_t v, int k) {
  const int lane = threadIdx.x & 31;
  if (k == 0) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d; d /= 2) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, d);
      const bool larger = ((lane & size) == 0) == ((lane & d) == 0);   // this lane keeps the larger one
      v = larger ? max(v, o) : min(v, o);
    }
  return __shfl_sync(0xffffffffu, v, k);
}

// The candidates of one warp: elements that reach a value that at least `top` elements of the row do reach.
template <int W>
struct Candidates {
  using Sh = Shared<W>;
  Sh& sh;
  const int top, warp, lane;
  uint32_t own = 0;                    // lane i: the warp's i-th largest of the steps' lanes' maxima, for SEEN lanes
  uint32_t floor = 0x00800000u;        // the value, as it orders; above -inf
  uint32_t passed = 0;                 // the least that this step's cuts left
  float reach = INFINITY;
  int count = 0;

  __device__ __forceinline__ Candidates(Sh& s, int t, int w, int l) : sh(s), top(t), warp(w), lane(l) {}
  __device__ __forceinline__ void raise(uint32_t o) {
    if (o > floor) floor = o;
    reach = value_of(floor);
    if (reach != reach) reach = INFINITY;
  }
  __device__ __forceinline__ void refresh() { raise(*(volatile uint32_t*)&sh.reach); }
  // Takes the largest of a step's lanes' maxima into the warp's: other elements each time.
  __device__ __forceinline__ void see(float big) {
    uint32_t o = ordered(big);
#pragma unroll 1
    for (int j = 0; j < Sh::SEEN; j++) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, o);
      const int place = __popc(__ballot_sync(0xffffffffu, lane < Sh::SEEN && own >= m));
      if (place == Sh::SEEN || m < floor) break;
      const uint32_t up = __shfl_up_sync(0xffffffffu, own, 1);
      own = lane > place ? up : lane == place ? m : own;
      if (lane == __ffs(__ballot_sync(0xffffffffu, o == m)) - 1) o = 0;
    }
    if (lane < Sh::SEEN) ((volatile uint32_t*)sh.seen)[warp * Sh::SEEN + lane] = own;
    __syncwarp();
  }
  // The value that `top` of all warps' do reach.  Reading older ones of other warps only keeps more candidates.
  __device__ __forceinline__ void common() {
    const uint32_t k = of_rank(((volatile uint32_t*)sh.seen)[lane], top - 1);
    if (lane == 0 && k > *(volatile uint32_t*)&sh.reach) atomicMax(&sh.reach, k);
    raise(k);
  }
  __device__ __forceinline__ void begin(float big) {
    see(big);
    if (lane == 0 && warp == 0) sh.reach = sh.total = 0;
    if (warp == 0) sh.best[lane] = 0;
    __syncthreads();
    common();
  }
  // Shortens a full list: to what reaches the `top`-th of the lanes' largest, and if that is still much to its `top` largest.
  __device__ __forceinline__ void cut() {
    __syncwarp();
    u64* const list = sh.cand[warp];
    uint32_t most = 0;
    for (int i = lane; i < count; i += 32) most = max(most, (uint32_t)(list[i] >> 32));
    uint32_t least = of_rank(most, top - 1);
    int left = 0;
#pragma unroll 1
    for (int i = 0; i < count; i += 32) {
      const u64 key = i + lane < count ? list[i + lane] : 0;
      const bool is = key != 0 && (uint32_t)(key >> 32) >= least;
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      if (is) list[left + __popc(m & ((1u << lane) - 1))] = key;   // not past what is read
      left += __popc(m);
      __syncwarp();
    }
    count = left;
    if (count > CAP / 2) {
      u64* const sorted = sh.all + warp * CAP;
#pragma unroll 1
      for (int i = lane; i < count; i += 32) {
        const u64 key = list[i];
        int rank = 0;
        for (int j = 0; j < count; j++) rank += list[j] > key;
        if (rank < top) sorted[rank] = key;
      }
      __syncwarp();
      if (lane < top) list[lane] = sorted[lane];
      __syncwarp();
      count = top;
      least = (uint32_t)(list[top - 1] >> 32);
    }
    raise(least);
    passed = max(passed, least);
  }
  // What reaches the value in a step; big: the lane's largest; at(src, j, index): whether the row has the j-th of lane src's
  // elements, and its index.  They are read again, a lane's by the whole warp: the step's registers may hold the next one's.
  template <int L, typename T, typename At>
  __device__ __forceinline__ void add(const T* row, float big, At at) {
    uint32_t who = __ballot_sync(0xffffffffu, big >= reach);
    passed = 0;
#pragma unroll 1
    while (who) {
      const int src = __ffs(who) - 1;
      who &= who - 1;
      uint32_t index = 0;
      float y = -INFINITY;
      if (lane < L && at(src, lane, index)) y = Elem<T>::get(row[index]);
      if (count > CAP - 32) cut();
      const bool is = y >= reach;                          // above -inf
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      if (is) sh.cand[warp][count + __popc(m & ((1u << lane) - 1))] = key_of(y, index);
      count += __popc(m);
    }
    // elements of later steps have larger indices than the `top` that reach what the list was cut to
    if (passed) raise(passed + 1);
  }
  // The CTA's `top` largest, in order, to sh.best (zeros where there are fewer).
  __device__ __forceinline__ void finish() {
    __syncthreads();
    const uint32_t least = sh.reach;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const u64 key = i0 + lane < count ? sh.cand[warp][i0 + lane] : 0;
      const bool is = key != 0 && (uint32_t)(key >> 32) >= least;
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      uint32_t at = 0;
      if (lane == 0 && m) at = atomicAdd(&sh.total, __popc(m));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1));
      if (is) sh.all[at] = key;
    }
    __syncthreads();
    const int n = (int)sh.total;
    for (int i = threadIdx.x; i < n; i += 32 * W) {
      const u64 key = sh.all[i];
      int rank = 0;
      for (int j = 0; j < n; j++) rank += sh.all[j] > key;
      if (rank < top) sh.best[rank] = key;
    }
    __syncthreads();
  }
};

__device__ __forceinline__ uint32_t leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}

// W warps a CTA; parts: CTAs (a cluster, with 8 warps) of a row
template <typename T, int W, bool TOP>
__global__ void __launch_bounds__(32 * W, W == 1 ? 24 : 32 / W) lp_kernel(const __grid_constant__ LpArgs a, int parts) {
  constexpr int VEC = Elem<T>::VEC, G = 32 * W;
  __shared__ Sums sums[W], joins[8];     // of the warps; of a cluster's parts
  __shared__ std::conditional_t<TOP, Shared<W>, int> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t r = blockIdx.x / (uint32_t)parts;
  const uint32_t part = blockIdx.x % (uint32_t)parts;
  const T* const row = static_cast<const T*>(a.x) + r * a.xs;
  const int64_t target = a.targets[r];
  const float at_target = tid == 0 && target >= 0 && target < (int64_t)a.cols ? Elem<T>::get(row[target]) : 0.f;
  const float c = (float)(1.4426950408889634 / (double)a.temperature);
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");   // the first CTA's memory is there (waited for below)

  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const uint32_t nv = (a.cols + off + VEC - 1) / VEC, per = (nv + parts - 1) / parts;
  const uint32_t v0 = min(nv, part * per), v1 = min(nv, v0 + per);

  float top_x = -INFINITY;                  // this thread's largest element
  u64 S2 = 0, E2 = 0;
  const auto load = [&](Run<T, VEC> (&x)[NV], uint32_t v) {
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t at = v + i * G + tid;
      if (at < v1) {
        load_vector(x[i], row, (int64_t)at * VEC - off, a.cols);
      } else {
        x[i].zero();
#pragma unroll
        for (int e = 0; e < VEC; e++) x[i].put_bits(e, lowest<T>());
      }
    }
  };
  const auto sum = [&](const Run<T, VEC> (&x)[NV], float big) {
    if (big > top_x) {
      float s0, s1, e0, e1;
      f2::unpack(S2, s0, s1);
      f2::unpack(E2, e0, e1);
      Sums lo = {top_x, s0, e0}, hi = {top_x, s1, e1};
      top_x = big;
      lo.to(big, c);
      hi.to(big, c);
      S2 = f2::pack(lo.S, hi.S);
      E2 = f2::pack(lo.E, hi.E);
    }
    const u64 cc = f2::splat(c), mm = f2::splat(top_x == -INFINITY ? 0.f : -top_x);
#pragma unroll
    for (int i = 0; i < NV; i++) {
#pragma unroll
      for (int e = 0; e < VEC / 2; e++) {
        float t0, t1;
        f2::unpack(f2::mul(f2::add(x[i].get2(e), mm), cc), t0, t1);
        t0 = max_nan(t0, FAR);
        t1 = max_nan(t1, FAR);
        const u64 p = f2::pack(ex2(t0), ex2(t1));
        S2 = f2::add(S2, p);
        E2 = f2::fma(p, f2::pack(t0, t1), E2);
      }
    }
  };
  const auto most = [&](const Run<T, VEC> (&x)[NV]) {
    float big = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; i++) big = fmaxf(big, largest(x[i]));
    return big;
  };
  // the loads of one step are under way while the other's elements are worked on
  constexpr uint32_t STEP = NV * G;
  Run<T, VEC> x0[NV], x1[NV];
  load(x0, v0);
  const auto steps = [&](auto begin, auto after) {
    float big[2] = {most(x0), -INFINITY};
    begin(big[0]);
    for (uint32_t v = v0; v < v1; v += 2 * STEP) {
      load(x1, min(v + STEP, v1));
      big[0] = most(x0);
      sum(x0, big[0]);
      load(x0, min(v + 2 * STEP, v1));
      big[1] = most(x1);
      if (v + STEP < v1) sum(x1, big[1]);
      after(v, big);
    }
  };
  if constexpr (TOP) {
    Candidates<W> cand(sh, a.top, warp, lane);
    steps([&](float big) { cand.begin(big); },
          [&](uint32_t v, const float (&big)[2]) {
#pragma unroll 1
            for (int s = 0; s < 2; s++) {
              const float most = s ? big[1] : big[0];
              cand.refresh();
              if (!__any_sync(0xffffffffu, most >= cand.reach)) continue;
              const uint32_t first = v + s * STEP;
              if (first > v0) {
                cand.see(most);
                cand.common();
              }
              cand.template add<NV * VEC>(row, most, [&](int src, int j, uint32_t& index) {
                const uint32_t at = first + (j / VEC) * G + warp * 32 + src;
                const int64_t i = (int64_t)at * VEC - off + j % VEC;
                index = (uint32_t)i;
                return at < v1 && i >= 0 && i < a.cols;
              });
            }
          });
    cand.finish();
  } else {
    steps([](float) {}, [](uint32_t, const float (&)[2]) {});
  }

  float s0, s1, e0, e1;
  f2::unpack(S2, s0, s1);
  f2::unpack(E2, e0, e1);
  Sums m = {top_x, s0 + s1, e0 + e1};
#pragma unroll
  for (int o = 16; o; o >>= 1) {   // the lower lane's sums first, so that both get the same bits
    Sums u = {__shfl_xor_sync(0xffffffffu, m.m, o), __shfl_xor_sync(0xffffffffu, m.S, o), __shfl_xor_sync(0xffffffffu, m.E, o)};
    if (lane & o) {
      const Sums t = m;
      m = u;
      u = t;
    }
    m.join(u, c);
  }
  if (lane == 0) sums[warp] = m;
  __syncthreads();
  if (warp == 0)
    for (int w = 1; w < W; w++) m.join(sums[w], c);
  if (parts > 1) {   // the parts leave their sums and lists with the first CTA
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (warp == 0) {
      const uint32_t at = leader(tc5::smem_addr(&joins[part]));
      __syncwarp();
      if (lane == 0)
        asm volatile("st.shared::cluster.f32 [%0], %1;\n\tst.shared::cluster.f32 [%0 + 4], %2;\n\tst.shared::cluster.f32 [%0 + 8], %3;" ::"r"(at),
                     "f"(m.m), "f"(m.S), "f"(m.E)
                     : "memory");
      if constexpr (TOP)
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(leader(tc5::smem_addr(&sh.join[part][lane]))), "l"(sh.best[lane]) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (part != 0) return;
    if (warp == 0) {
      m = joins[0];
      for (int p = 1; p < parts; p++) m.join(joins[p], c);
    }
    if constexpr (TOP) {
      const u64 key = warp < parts ? sh.join[warp % 8][lane] : 0;   // a warp a part's list
      int rank = 0;
      for (int p = 0; p < parts; p++)
        for (int j = 0; j < a.top; j++) rank += sh.join[p][j] > key;
      if (warp == 0) sh.best[lane] = 0;
      __syncthreads();
      if (key != 0 && rank < a.top) sh.best[rank] = key;
      __syncthreads();
    }
  }
  if (warp != 0) return;
  const bool none = m.S == 0.f;                             // every logit is -inf
  const float log_s = none ? 0.f : logf(m.S);
  // The difference first, which keeps small ones of large logits exact; where it passes the largest finite number its quotient
  // may still be one, and is the difference of the quotients.
  const auto log_prob = [&](float y) {
    if (none || (y == -INFINITY && m.S == m.S)) return -INFINITY;
    const float d = y - m.m;
    return (isfinite(d) ? __fdiv_rn(d, a.temperature) : __fdiv_rn(y, a.temperature) - __fdiv_rn(m.m, a.temperature)) - log_s;
  };
  if (lane == 0) {
    float lp = 0.f;
    if (target >= (int64_t)a.cols) {
      lp = __uint_as_float(0x7fffffffu);
      if (a.status) atomicOr(a.status, DA_STATUS_BAD_TARGET);
    } else if (target >= 0) {
      lp = log_prob(at_target);
    }
    a.lp[r] = lp;
    const float entropy = none ? 0.f : __fmaf_rn(-LN2, m.E / m.S, log_s);
    a.entropy[r] = entropy;
    if (a.stats) {
      a.stats[3 * r] = m.m;
      a.stats[3 * r + 1] = m.S;
      a.stats[3 * r + 2] = entropy;
    }
    if (!isfinite(m.S) && a.status) atomicOr(a.status, DA_STATUS_NONFINITE);
  }
  if constexpr (TOP) {
    u64 key = sh.best[lane];
    int have = __popc(__ballot_sync(0xffffffffu, key != 0));
    for (uint32_t i = 0; have < a.top && i < a.cols; i += 32) {   // few are above -inf: the first of the others
      const bool is = i + lane < a.cols && Elem<T>::get(row[i + lane]) == -INFINITY;
      const uint32_t who = __ballot_sync(0xffffffffu, is);
      const int place = lane - have;                              // this lane takes the place-th of them
      if (place >= 0 && place < __popc(who)) key = key_of(-INFINITY, i + __fns(who, 0, place + 1));
      have += __popc(who);
    }
    if (lane < a.top) {
      const float y = key ? value_of((uint32_t)(key >> 32)) : __uint_as_float(0x7fffffffu);
      a.top_lp[r * a.top + lane] = log_prob(y);
      a.top_index[r * a.top + lane] = min((uint32_t)~(uint32_t)key, a.cols - 1);
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
  const float m = a.stats[3 * r], S = a.stats[3 * r + 1], H = a.stats[3 * r + 2];
  const int64_t target = a.targets[r];
  const float g = a.grad && target >= 0 && target < (int64_t)a.cols ? a.grad[r] : 0.f, h = a.grad_entropy ? a.grad_entropy[r] : 0.f;
  const bool none = S == 0.f;
  const float inv = none ? 0.f : back / S, log_s = none ? 0.f : log2f(S);
  const float A = -(g + h * __fmaf_rn(-LN2, log_s, H)) * inv, B = -h * LN2 * inv;
  const float hit = none ? 0.f : g * back;
  const u64 cc = f2::splat(c), mm = f2::splat(none ? 0.f : -m), aa = f2::splat(A), bb = f2::splat(B);

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
      f2::unpack(f2::mul(f2::add(x[i].get2(e), mm), cc), t0, t1);
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
  // Few rows: parts of a row, as many as keep at most two CTAs an SM and a step's vectors in each (8 x 128256 f32: 6.3 us in 8 parts).
  int parts = 1;
  while (parts < 8 && a.rows * parts * 2 <= 304 && vectors >= (int64_t)parts * 2 * 256 * NV) parts *= 2;
  if (parts > 1) return forward<T, 8>(a, parts, st);
  // Warps of a row: by its length 1 up to 256 vectors, 2 up to 3000, else 4 (fewer leave a warp more steps to one start and end; us of
  // 8192 bf16 rows with 1, 2, 4 and 8 warps, no and 5 alternatives: 2000 columns 14 19 31 59 and 36 40 59 102, 10000 columns
  // 40 39 50 76 and 86 89 105 131); more where there are fewer than 16 warps an SM (300 x 50000: 11 with 4, 10 with 8).
  int warps = vectors <= 256 ? 1 : vectors <= 3000 ? 2 : 4;
  while (warps < 8 && a.rows * warps < 152 * 16 && vectors >= 128 * warps) warps *= 2;
  // More rows than the 1216 CTAs of four warps that fit, and a last round of less than half of them: eight warps, whose rounds are
  // shorter, where a row is long enough for them, up to three rounds (binary32, which waits for memory alone, four); else two
  // warps, which need one round up to 2432 rows.  us with 2, 4 and 8 warps: 1300 x 128256 f32 112 129 117, with 5 alternatives
  // 144 154 136; 1300 x 50000 f32 50 58 56; 2432 x 50000 bf16 48 51 59; 2700 x 262144 f32 509 437 406.
  constexpr int64_t round = 152 * 8;
  if (warps == 4 && a.rows > round) {
    const bool little = (a.rows - 1) % round < round / 2;
    if (little && vectors >= 16000 && a.rows <= (sizeof(T) == 4 ? 4 : 3) * round) warps = 8;
    else if (a.rows <= 2 * round) warps = 2;
  }
  switch (warps) {
    case 1: return forward<T, 1>(a, 1, st);
    case 2: return forward<T, 2>(a, 1, st);
    case 4: return forward<T, 4>(a, 1, st);
    default: return forward<T, 8>(a, 1, st);
  }
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
