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
// What bounds it: HBM; x is read once, and once more and dx written in the gradient.  A step of 4 vectors of 16 bytes a
// thread stays in registers: its maximum, then (the reference moved where that is larger) its terms, while the next step's
// loads are under way.
//
// Alternatives: a value that at least `top` elements of the row reach is found from the first step's maxima of single threads (each of
// the CTA's warps finds its ceil(top / warps)-th largest, the least of them is that value); a warp keeps what reaches it, some
// tens of elements of a large row, in shared memory, and raises the value now and then by its own and the other warps' ceil(top /
// warps)-th best so far.  A full list is cut to its `top` largest.  At the end each warp sorts out its `top`, one
// warp those of all.  Equal values go by their index: a warp meets its elements in order of their indices.  No barrier but the first
// step's, and which candidates are kept does not change the result.
//
// A row is one CTA's; short rows a warp's; where few rows would leave SMs idle, a cluster's, whose parts hand their sums and
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

constexpr int CAP = 256;               // candidates that a warp keeps

template <int W>
struct Shared {
  u64 cand[W][CAP];
  u64 list[W][LP_TOP];
  u64 best[LP_TOP];
  u64 join[8][LP_TOP];                 // first CTA of a cluster: the parts' lists
  uint32_t reached[W];
};

// The largest n of the first `have` keys of `from`, in order, to `to`, zeros behind them; by one whole warp.
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
  __syncwarp();
  scan();
  u64 keep = 0;
  for (int j = 0; j < n; j++) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
    const u64 top = (u64)hi << 32 | lo;
    if (top == 0) break;
    if (lane == j) keep = top;
    if (mine == top) {   // keys differ, so one lane
      from[at] = 0;
      scan();
    }
  }
  __syncwarp();
  if (lane < LP_TOP) to[lane] = keep;
  __syncwarp();
}

// The candidates of one warp: elements that reach `reach`, a value that at least `top` elements of the row do reach.
template <int W>
struct Candidates {
  Shared<W>& sh;
  const int top, warp, lane, need;     // need: elements that each of the W warps has to have above a common value
  float reach = INFINITY;
  int count = 0, next = 0;

  __device__ __forceinline__ Candidates(Shared<W>& s, int t, int w, int l) : sh(s), top(t), warp(w), lane(l), need((t + W - 1) / W) {}
  __device__ __forceinline__ void at_least(uint32_t o) { reach = fmaxf(reach, value_of(max(o, 0x00800000u))); }   // above -inf

  // the first step: from the maxima of the CTA's threads
  __device__ __forceinline__ void begin(float big) {
    uint32_t o = ordered(big), least = 0;
    for (int j = 0; j < need; j++) {
      least = __reduce_max_sync(0xffffffffu, o);
      const uint32_t who = __ballot_sync(0xffffffffu, o == least);
      if (lane == __ffs(who) - 1) o = 0;
    }
    if (lane == 0) sh.reached[warp] = least;
    __syncthreads();
    reach = -INFINITY;
    common();
    next = 24;
  }
  __device__ __forceinline__ void common() {
    const volatile uint32_t* const r = sh.reached;
    at_least(__reduce_min_sync(0xffffffffu, r[lane % W]));
  }
  // The value that `need` of this warp's candidates reach, for all warps; and what all of them have found.  Reading older values of
  // others only keeps more candidates.
  __device__ __forceinline__ void publish() {
    u64 last = ~0ull;
    for (int j = 0; j < need && last; j++) {
      u64 mine = 0;
      for (int i = lane; i < count; i += 32) {
        const u64 k = sh.cand[warp][i];
        if (k < last && k > mine) mine = k;
      }
      const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
      const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
      last = (u64)hi << 32 | lo;
    }
    volatile uint32_t* const mine = &sh.reached[warp];
    if (lane == 0) *mine = max(*mine, (uint32_t)(last >> 32));
    __syncwarp();
    common();
    next = count + 24;
  }
  __device__ __forceinline__ void cut() {   // to the largest `top`; later ones of equal value have larger indices
    select_largest(sh.cand[warp], count, sh.list[warp], top);
    if (lane < top) sh.cand[warp][lane] = sh.list[warp][lane];
    __syncwarp();
    count = top;
    at_least((uint32_t)(sh.list[warp][top - 1] >> 32) + 1);
    publish();
  }
  // the warp's vectors of one load, in order of their indices; big: the lane's largest element
  template <typename T>
  __device__ __forceinline__ void add(const Run<T, Elem<T>::VEC>& x, float big, uint32_t first) {
    constexpr int VEC = Elem<T>::VEC;
    uint32_t who = __ballot_sync(0xffffffffu, big >= reach);
    while (who) {
      const int src = __ffs(who) - 1;
      who &= who - 1;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; i++) w[i] = __shfl_sync(0xffffffffu, x.w[i], src);
      const uint32_t from = __shfl_sync(0xffffffffu, first, src);
      const int e = lane & (VEC - 1), i = VEC == 8 ? e >> 1 : e;
      const uint32_t word = i & 2 ? i & 1 ? w[3] : w[2] : i & 1 ? w[1] : w[0];
      float y;
      if constexpr (VEC == 4) y = __uint_as_float(word);
      else if constexpr (std::is_same<T, __nv_bfloat16>::value) y = __uint_as_float(e & 1 ? word & 0xFFFF0000u : word << 16);
      else y = __half2float(__ushort_as_half((uint16_t)(e & 1 ? word >> 16 : word)));
      if (count > CAP - VEC) cut();
      const bool is = lane < VEC && y >= reach;
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      if (is) sh.cand[warp][count + __popc(m & ((1u << lane) - 1))] = key_of(y, from + e);
      count += __popc(m);
    }
    if (count >= next) {
      __syncwarp();
      publish();
    }
  }
};

__device__ __forceinline__ uint32_t leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}

// W warps a CTA; parts: CTAs (a cluster) of a row
template <typename T, int W, bool TOP>
__global__ void __launch_bounds__(32 * W, W == 8 ? 3 : 16) lp_kernel(const __grid_constant__ LpArgs a, int parts) {
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

  float top_x = -INFINITY, M = -INFINITY;   // this thread's largest element, and its reference
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
  const auto steps = [&](auto each) {
    for (uint32_t v = v0; v < v1; v += 2 * STEP) {
      load(x1, min(v + STEP, v1));
      each(x0, v);
      if (v + STEP >= v1) break;
      load(x0, min(v + 2 * STEP, v1));
      each(x1, v + STEP);
    }
  };
  int count = 0;
  if constexpr (TOP) {
    Candidates<W> cand(sh, a.top, warp, lane);
    cand.begin(most(x0));
    steps([&](const Run<T, VEC> (&x)[NV], uint32_t v) {
      const float big = most(x);
      sum(x, big);
      if (__any_sync(0xffffffffu, big >= cand.reach)) {
#pragma unroll
        for (int i = 0; i < NV; i++) cand.add(x[i], largest(x[i]), (v + i * G + tid) * VEC - off);
      }
    });
    count = cand.count;
  } else {
    steps([&](const Run<T, VEC> (&x)[NV], uint32_t) { sum(x, most(x)); });
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
  if (lane == 0) sums[warp] = m;
  if constexpr (TOP) select_largest(sh.cand[warp], count, sh.list[warp], a.top);
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < W; w++) m.join(sums[w]);
    if constexpr (TOP) select_largest(sh.list[0], W * LP_TOP, sh.best, a.top);
  }
  if (parts > 1) {   // the parts leave their sums and lists with the first CTA
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (warp == 0) {
      const uint32_t at = leader(tc5::smem_addr(&joins[part]));
      __syncwarp();
      if (lane == 0)
        asm volatile("st.shared::cluster.f32 [%0], %1;\n\tst.shared::cluster.f32 [%0 + 4], %2;\n\tst.shared::cluster.f32 [%0 + 8], %3;" ::"r"(at),
                     "f"(m.M), "f"(m.S), "f"(m.E)
                     : "memory");
      if constexpr (TOP)
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(leader(tc5::smem_addr(&sh.join[part][lane]))), "l"(sh.best[lane]) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (part != 0) return;
    if (warp == 0) {
      m = joins[0];
      for (int p = 1; p < parts; p++) m.join(joins[p]);
      if constexpr (TOP) select_largest(sh.join[0], parts * LP_TOP, sh.best, a.top);
    }
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
      a.top_lp[r * a.top + lane] = none || y == -INFINITY ? -INFINITY : (__fmaf_rn(y, c, -m.M) - log_s) * LN2;
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
  if (vectors <= 64 * NV) return forward<T, 1>(a, 1, st);
  // parts of a row: as many as keep at most two CTAs an SM, and a step's vectors in each
  int parts = 1;
  while (parts < 8 && a.rows * parts * 2 <= 304 && vectors >= (int64_t)parts * 2 * 256 * NV) parts *= 2;
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
