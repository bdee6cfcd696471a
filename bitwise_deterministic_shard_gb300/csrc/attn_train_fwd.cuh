// Forward pass of the training attention.
//
//   t = scale q.k;  u = cap tanh(t / cap);  s = u - slope |pos - j|;  hidden keys -inf
//   o = sum exp(s - m) v / sum exp(s - m);  lse = m + log sum exp(s - m)
//
// One CTA holds two tiles of 128 queries and runs over the key tiles once.  Per query tile a group of
// eight warps owns a query row with two threads, each with 64 of the tile's 128 keys: a thread reads its scores
// from TMEM, keeps the row's maximum and its part of the sum in registers, and writes exp2 of the scores as
// 16-bit weights to shared memory, where the second product takes them as its A operand.  One warp
// copies tiles (tensor maps, a ring of key and value tiles), one issues all products as they become possible:
//   S_i = Q_i K_n^T (128 x 128 x D),  O_i += P_i V_n (128 x D x 128).
// TMEM: two score tiles and two output tiles, 2 x 128 + 2 x D columns, 512 for D = 128.  That is why the weights go
// to shared memory: over the scores in TMEM they would hold up the next scores until the second product
// had read them (a group then waited 2450 of the 6300 cycles of a step for its scores).  So the next scores
// are computed while the present ones are worked on.
//
// What bounds it: the softmax's arithmetic (per score 7 to 9 cycles of the FP32 pipe with a cap, 2 without, 4 of the
// special function unit, against 8 of the tensor cores for two products of D = 128) and the latencies
// that four softmax warps a scheduler leave open.  4096 causal, 16 heads, D 128, bf16, cap 30: 80 us, 859 TFLOP/s, 0.45 of the
// measured matrix rate; tensor pipe 40 % and issue slots 54 % of the cycles (one thread a row 107 us; weights over the scores
// in TMEM 108; the products issued by one lane 109; spilling control warps 94; the coefficients in registers 81).
//
// The weights are rounded to the inputs' 16-bit type (the tensor cores take both operands in one
// type); the sum of the weights and the output are binary32.  The output is divided by the sum of the rounded weights where
// a row may have few keys that count: few key tiles, a distance bias (their roundings then largely cancel: 96
// queries, output 2.5e-3 -> 2.0e-3 off) and, as it costs nothing there, the form below; over many keys they do
// not cancel, and the sum costs 1.5 operations a score.  lse is formed from the unrounded sum always.  The maximum is moved only when
// it grows by more than 2^8: until then weights are at most 2^8 too large, which the division by
// their sum undoes exactly, and the output needs no rescaling.  Capped bf16 scores without a bias need no
// maximum: they lie within +-cap, so with a cap of at most 32 (weights of 2^+-46) and values below 2^64 nothing overflows in
// binary32's range, which bf16 shares, with the constant 0 in the maximum's place.
//
// Few queries (Sq * group <= 128): the heads that share a key head are the rows of one tile, so
// a cache is read once; both groups take the same queries and every other key tile, and the key range
// is split over CTAs so that all SMs read.  Each group writes its unnormalised sums, a second
// kernel joins them in a fixed order (8 requests of 32 heads over 8 key heads, 8192 keys: 57 us and 4 for the join, 4.5
// TB/s: each SM keeps at most four key or value tiles in flight).  Without a split of the keys over CTAs the second group hands its sums to the
// first within the CTA; calls with few query tiles take this form too, as twice as many CTAs of half the steps.
#pragma once
#include "../../include/detattn.h"
#include "attn_train.h"
#include "device_once.h"
#include "pack2.cuh"
#include "tc5_tile.cuh"
#include "tile_ring.h"

namespace detattn {
namespace ta {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

using f2::u64;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Scores of a row in log2 units: f tanh(k t) with a cap (k = scale / cap, f = cap log2 e), else f t (f = scale log2 e).
//
// tanh of any argument: 1 - 2 / (1 + e^2x), two operations of the special function unit, 2^-22 absolute.  On
// [-1, 1], where the scores of a capped model nearly always are: x P(x^2), P of degree 5, or of degree 3 on
// [-0.5, 0.5], fitted for the least greatest error (least squares with weights moved toward the largest
// errors), 3.1e-7 and 1.6e-7 absolute with binary32 steps, on the packed multiplier; k and f are folded into the
// coefficients.  The special function unit would otherwise bound the kernels: three of its operations a score
// instead of one.  Scores beyond the cap pay that: 4096 causal, cap 30, forward 118 us against 78, the backward kernels 294
// against 241 (71 and 214 without a cap).
__device__ __forceinline__ float tanh_any(float x) {
  return __fmaf_rn(-2.f, tc5::rcp(1.f + tc5::ex2(x * (2.f * LOG2E))), 1.f);
}
struct Cap {
  const TaCap& c;   // in the kernel's parameters: constant-bank operands, no registers
  __device__ __forceinline__ Cap(const TaArgs& a) : c(a.cap) {}
  __device__ __forceinline__ u64 smaller2(u64 t) const {
    const u64 z = f2::mul(t, t);
    u64 p = f2::fma(c.s[3], z, c.s[2]);
    p = f2::fma(p, z, c.s[1]);
    p = f2::fma(p, z, c.s[0]);
    return f2::mul(t, p);
  }
  __device__ __forceinline__ u64 small2(u64 t) const {
    const u64 z = f2::mul(t, t);
    u64 p = f2::fma(c.c[5], z, c.c[4]);
    p = f2::fma(p, z, c.c[3]);
    p = f2::fma(p, z, c.c[2]);
    p = f2::fma(p, z, c.c[1]);
    p = f2::fma(p, z, c.c[0]);
    return f2::mul(t, p);
  }
  // v <- f tanh(k v) for N scores of each lane.  The warp decides by its scores which form it takes; where they hold padding,
  // whose values may be anything, without a vote the one for any argument (unless that is too far off: 2^-22 of a far cap).
  template <int N>
  __device__ __forceinline__ void apply(float* v, bool clean) const {
    const bool vote = clean || c.far;
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      m[0] = max3_abs(m[0], v[i], v[i + 1]);
      m[1] = max3_abs(m[1], v[i + 2], v[i + 3]);
    }
    const float top = fmaxf(m[0], m[1]);
    if (vote && __all_sync(0xffffffffu, top <= c.least)) {
#pragma unroll
      for (int i = 0; i < N; i += 2) f2::unpack(smaller2(f2::pack(v[i], v[i + 1])), v[i], v[i + 1]);
    } else if (vote && __all_sync(0xffffffffu, top <= c.most)) {
#pragma unroll
      for (int i = 0; i < N; i += 2) f2::unpack(small2(f2::pack(v[i], v[i + 1])), v[i], v[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; i++) v[i] = c.f * tanh_any(v[i] * c.k);
    }
  }
};

// Which key tiles a tile of queries needs.  A whole warp calls it.
__device__ __forceinline__ int2 key_range(const TaArgs& a, int b, int first_pos, int last_pos, int dlo, int dhi) {
  int hi = a.Skv;
  if (a.causal) hi = min(hi, max(last_pos + 1, a.prefix ? a.prefix[b] : 0));
  int n0 = 0, n1 = (max(hi, 0) + TA_TILE - 1) / TA_TILE;
  if (last_pos < first_pos) n1 = 0;
  if (a.docs) {
    const TaBounds* bd = a.bounds + (int64_t)b * a.ktiles;
    int f = n1, l = -1;
    for (int n = threadIdx.x & 31; n < n1; n += 32)
      if (bd[n].lo <= dhi && bd[n].hi >= dlo) {
        f = min(f, n);
        l = max(l, n);
      }
    f = __reduce_min_sync(0xffffffffu, f);
    l = __reduce_max_sync(0xffffffffu, l);
    n0 = f;
    n1 = l + 1;
    if (n1 <= n0) n0 = n1 = 0;
  }
  return make_int2(n0, n1);
}

// The first n of N columns as bits, 32 to a word.
template <int N>
__device__ __forceinline__ void first_bits(uint32_t (&w)[N / 32], int n) {
#pragma unroll
  for (int i = 0; i < N / 32; i++) {
    const int k = n - 32 * i;
    w[i] = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
  }
}
// Keeps of each lane's bits those of columns whose document is its own: other[0, N) are the columns' ids (left of
// them exist), doc the lane's.  A warp's rows hold few documents, so the columns' ids are compared once for
// each of these, a lane a column.  A whole warp calls it.
template <int N>
__device__ __forceinline__ void same_doc(uint32_t (&w)[N / 32], const int* other, int left, int doc) {
  const int lane = threadIdx.x & 31;
  int id[N / 32];
#pragma unroll
  for (int i = 0; i < N / 32; i++) id[i] = 32 * i + lane < left ? other[32 * i + lane] : -1;
  uint32_t todo = __ballot_sync(0xffffffffu, doc >= 0);
  if (doc < 0) {
#pragma unroll
    for (int i = 0; i < N / 32; i++) w[i] = 0;
  }
  while (todo) {
    const int d = __shfl_sync(0xffffffffu, doc, __ffs(todo) - 1);
    const bool mine = doc == d;
#pragma unroll
    for (int i = 0; i < N / 32; i++) {
      const uint32_t same = __ballot_sync(0xffffffffu, id[i] == d);
      if (mine) w[i] &= same;
    }
    todo &= ~__ballot_sync(0xffffffffu, mine);
  }
}

// COLS columns of a TMEM accumulator (plus more times a second one, where more is not 0), times k, to
// 16 bits in a tile's row r (swizzled units); zeros without `some`, which is the same in all lanes (the loads are the
// whole warp's)
template <bool BF, int COLS>
__device__ __forceinline__ void row_out(uint32_t tile, uint32_t taddr, uint32_t taddr2, int r, int c0, float k, float more,
                                        bool some) {
  using namespace tc5;
#pragma unroll
  for (int c = c0; c < c0 + COLS; c += 32) {
    float o[32];
    if (some) {
      ld_x32(taddr + c, o);
      ld_wait();
      if (taddr2 != taddr) {
        float x[32];
        ld_x32(taddr2 + c, x);
        ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e++) o[e] = __fmaf_rn(more, x[e], o[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 32; e++) o[e] = some ? o[e] * k : 0.f;
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int unit = ((c & 63) >> 3) + u;
      const uint32_t at = tile + (c >> 6) * PANEL + r * 128 + ((unit ^ (r & 7)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack16<BF>(o[8 * u], o[8 * u + 1])),
                   "r"(pack16<BF>(o[8 * u + 2], o[8 * u + 3])), "r"(pack16<BF>(o[8 * u + 4], o[8 * u + 5])),
                   "r"(pack16<BF>(o[8 * u + 6], o[8 * u + 7]))
                   : "memory");
    }
  }
}
}  // namespace ta

// Two groups of eight softmax warps and a control group (copies, products, two idle warps).  setmaxnreg moves
// the control group's registers to the softmax threads: 640 x 96 at launch = 128 x 32 + 512 x 112.  The control
// group never takes its registers back: an idle warp's request would be met before the softmax groups'.
constexpr int TA_FWD_THREADS = 640;

template <int DP>
struct TaFwdSmem {
  static constexpr int TILE = DP / 64 * tc5::PANEL, PTILE = 2 * tc5::PANEL;
  // two query tiles, two tiles of weights and a ring of key and value tiles (the split form has one query tile and
  // a stage more), then the rows' maxima
  static constexpr int NST = DP == 128 ? 3 : 7, MOST = NST + 1;   // MOST is a multiple of 4
  static constexpr int Q = 0, P = 2 * TILE, KV = P + 2 * PTILE, MAX = KV + NST * TILE, END = MAX + 2048;
};

// ALT: both groups share a query tile and take every other key tile
template <int DP, bool BF, bool ALT>
__global__ void __launch_bounds__(TA_FWD_THREADS, 1) ta_fwd_kernel(const __grid_constant__ TaArgs a) {
  using namespace tc5;
  using namespace ta;
  using L = TaFwdSmem<DP>;
  constexpr int TILE = L::TILE;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t q_full, kv_full[L::MOST], kv_empty[L::MOST], s_full[2], s_read[2], p_full[2], pv_done[2], gone;
  __shared__ uint32_t tmem_at;
  __shared__ int dead, wdoc[16][3], range[2][2], qdoc[2][3];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  // the rows' maxima in the two halves of the keys, as bf16 rounded up: [turn][tile][half][row]
  uint16_t* const exchange = reinterpret_cast<uint16_t*>(raw + (base - smem_addr(raw)) + L::MAX);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &dead;

  const int NH = a.Hq / a.pack, HB = a.B * NH;
  const int hb = blockIdx.x % HB, b = hb / NH, h = hb % NH;
  const int kh = a.pack > 1 ? h : h / a.group;
  constexpr bool alt = ALT;
  // the last queries first: with causal masking the longest
  const int bt = blockIdx.x / HB, z = alt ? bt % a.splits : 0;
  const int t = alt ? a.qtiles - 1 - bt / a.splits : (int)(gridDim.x / HB) - 1 - bt;
  constexpr int nst = alt ? L::MOST : L::NST;
  // the ring's stages: the split form's last one lies in the second query tile
  const auto stage_at = [&](int s) { return base + (s < L::NST ? L::KV + s * TILE : TILE); };

  // this thread's query row (softmax groups)
  const int wg = warp >> 3, half = (warp >> 2) & 1, r = threadIdx.x & 127;
  const int qt = alt ? t : 2 * t + wg;
  int qi, head;
  if (a.pack > 1) {
    qi = r / a.pack;
    head = h * a.pack + r % a.pack;
  } else {
    qi = qt * TA_TILE + r;
    head = h;
  }
  const bool valid = wg < 2 && qi < a.Sq && (a.pack == 1 || r < a.pack * a.qrows);
  const int off = a.Skv - a.Sq, pos = qi + off;
  int doc = -1;
  if (a.docs && valid && pos >= 0) doc = a.docs[(int64_t)b * a.Skv + pos];

  if (threadIdx.x == 0) {
    dead = 0;
    mbar_init(&q_full, 1);
    mbar_init(&gone, 1);
    for (int s = 0; s < L::MOST; s++) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_read[i], 256);
      mbar_init(&p_full[i], 256);
      mbar_init(&pv_done[i], 1);
    }
    mbar_fence_init();
  }
  if (warp == 17) tmem_alloc(&tmem_at, 512);
  // Rows that the packed heads' query box leaves unfilled (their number need not divide 128): what lies there may not decide
  // the form of the cap.
  if (wg == 0 && half == 0 && a.pack > 1 && r >= a.pack * a.qrows) zero_row<DP>(base + L::Q, r);
  if (wg < 2) {
    const int dl = __reduce_min_sync(0xffffffffu, doc < 0 ? 0x7fffffff : doc), dh = __reduce_max_sync(0xffffffffu, doc);
    const int neg = __any_sync(0xffffffffu, valid && doc < 0);
    if (lane == 0) {
      wdoc[warp][0] = dl;
      wdoc[warp][1] = max(dh, -1);
      wdoc[warp][2] = neg;      // apart: a warp may hold nothing but padding
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (wg < 2 && (warp & 7) == 0) {
    int dl = 0x7fffffff, dh = -1, neg = 0;
    for (int w = warp; w < warp + 4; w++) {
      dl = min(dl, wdoc[w][0]);
      dh = max(dh, wdoc[w][1]);
      neg |= wdoc[w][2];
    }
    const int q0 = (a.pack > 1 ? 0 : qt * TA_TILE) + off;
    const int q1 = (qt >= a.qtiles ? 0 : a.pack > 1 ? a.Sq : min(qt * TA_TILE + TA_TILE, a.Sq)) - 1 + off;   // none: below q0
    const int2 nr = key_range(a, b, q0, q1, dl, dh);
    if (lane == 0) {
      range[wg][0] = nr.x;
      range[wg][1] = nr.y;
      qdoc[wg][0] = dl;
      qdoc[wg][1] = dh;
      qdoc[wg][2] = neg;
    }
  }
  __syncthreads();
  const uint32_t tmem = tmem_at;
  // key tiles of the two groups: [lo, hi[i]), or every other of [lo, hi) from lo + i on
  int lo, hi, hi0, hi1;
  if (alt) {
    const int n = range[0][1] - range[0][0], per = (n + a.splits - 1) / a.splits;
    lo = range[0][0] + min(n, z * per);
    hi = hi0 = hi1 = range[0][0] + min(n, (z + 1) * per);
  } else {
    const bool e0 = range[0][1] <= range[0][0], e1 = range[1][1] <= range[1][0];
    lo = e0 ? range[1][0] : e1 ? range[0][0] : min(range[0][0], range[1][0]);
    hi0 = e0 ? lo : range[0][1];
    hi1 = e1 ? lo : range[1][1];
    hi = max(hi0, hi1);
  }
  const int ntile = hi - lo;

  if (warp >= 16) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 32;" ::: "memory");
  if (warp == 16) {
    // ---- copies: queries once, then keys and values in the order in which the products take them ----
    if (lane == 0 && ntile > 0) {
      const int nq = alt ? 1 : 2;
      const int rows = a.pack > 1 ? a.pack * a.qrows : TA_TILE;
      mbar_expect_tx(&q_full, nq * (DP / 64) * rows * 128);
      for (int i = 0; i < nq; i++)
        for (int p = 0; p < DP / 64; p++) {
          const int at = base + L::Q + i * TILE + p * PANEL;
          if (a.pack > 1) tma_load(at, &a.q, p * 64, 0, 0, h, b, &q_full);   // an empty second tile too
          else tma_load(at, &a.q, p * 64, 0, min(alt ? t : 2 * t + i, a.qtiles - 1) * TA_TILE, h, b, &q_full);
        }
      uint32_t used = 0, odd = 0;                                    // a bit a stage: filled, its last fill's parity
      auto fetch = [&](const CUtensorMap* map, int k, int n) -> bool {
        const int s = k % nst;
        if (k >= nst && !mbar_wait(&kv_empty[s], ((k / nst) - 1) & 1, abort)) return false;
        mbar_expect_tx(&kv_full[s], TILE);
        for (int p = 0; p < DP / 64; p++)
          tma_load(stage_at(s) + p * PANEL, map, p * 64, 0, n * TA_TILE, kh, b, &kv_full[s]);
        used |= 1u << s;
        odd = (odd & ~(1u << s)) | (uint32_t)((k / nst) & 1) << s;
        return true;
      };
      bool ok = fetch(&a.k, key_place<ALT>(0), lo);
      if (ok && lo + 1 < hi) ok = fetch(&a.k, key_place<ALT>(1), lo + 1);
      for (int n = lo; n < hi && ok; n++) {
        ok = fetch(&a.v, value_place<ALT>(n - lo, ntile), n);
        if (ok && n + 2 < hi) ok = fetch(&a.k, key_place<ALT>(n + 2 - lo), n + 2);
      }
      // nothing may be in flight when the CTA ends
#pragma unroll 1
      for (int s = 0; s < nst; s++)
        if (used >> s & 1) mbar_drain(&kv_full[s], odd >> s & 1);
      mbar_drain(&q_full, 0);
    }
  } else if (warp == 17) {
    // ---- products: each as soon as its operands are there ----
    const int first = same(lo), tiles = same(ntile);
    if (tiles > 0) {
      const uint32_t one = elect(), tm = same(tmem);
      const uint32_t id_s = idesc<BF>(128, 128, false), id_o = idesc<BF>(128, DP, true);
      const int step = alt ? 2 : 1;
      const int end[2] = {same(hi0) - first, same(hi1) - first};     // key tiles count from the first one here
      int sn[2] = {0, alt ? 1 : 0}, pn[2] = {0, alt ? 1 : 0};        // next key tile of each group's two products
      int read[2] = {0, 0}, wrote[2] = {0, 0};                       // steps whose products were issued
      uint64_t t0 = 0;
      uint32_t idle = 0;
      bool ok = all_of(mbar_wait(&q_full, 0, abort));
      while (ok && (pn[0] < end[0] || pn[1] < end[1])) {
        bool some = false;
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int n = sn[i];
          if (n < end[i]) {
            const int k = key_place<ALT>(n), st = k % nst;
            if (all_of((read[i] == 0 || mbar_test(&s_read[i], (read[i] - 1) & 1)) && mbar_test(&kv_full[st], (k / nst) & 1))) {
              fence_after();
              const uint32_t q = base + L::Q + (alt ? 0 : i * TILE), kt = stage_at(st);
#pragma unroll
              for (int s = 0; s < DP / 16; s++) mma_ss(tm + i * 128, desc_k(q, s), desc_k(kt, s), id_s, s > 0, one);
              commit_one(&s_full[i], one);
              read[i]++;
              sn[i] += step;
              // only where the copies wait for it: no arrival is left when the CTA ends
              if ((alt || n >= end[i ^ 1] || sn[i ^ 1] > n) && !last_place(k, tiles, nst)) commit_one(&kv_empty[st], one);
              some = true;
            }
          }
          const int m = pn[i];
          if (m < end[i] && m < sn[i]) {
            const int k = value_place<ALT>(m, tiles), st = k % nst;
            if (all_of(mbar_test(&p_full[i], wrote[i] & 1) && mbar_test(&kv_full[st], (k / nst) & 1))) {
              fence_after();
              const uint32_t pt = base + L::P + i * L::PTILE, vt = stage_at(st);
#pragma unroll
              for (int s = 0; s < 8; s++)
                mma_ss(tm + 256 + i * DP, desc_k(pt, s), desc_mn(vt, s), id_o, s > 0 || wrote[i] > 0, one);
              commit_one(&pv_done[i], one);
              wrote[i]++;
              pn[i] += step;
              if ((alt || m >= end[i ^ 1] || pn[i ^ 1] > m) && !last_place(k, tiles, nst)) commit_one(&kv_empty[st], one);
              some = true;
            }
          }
        }
        if (some) {
          idle = 0;
        } else {                                                     // bounded, as every wait
          if (idle++ == 0) t0 = globaltimer();
          if ((idle & 63) == 0 && all_of(*abort || globaltimer() - t0 > WAIT_NS)) {
            ok = false;
            dead = 1;
          }
        }
      }
      if (!ok) {
        commit_one(&gone, one);
        mbar_drain(&gone, 0);
      }
    }
  }
  } else {
    // ---- softmax ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;" ::: "memory");
    const int i = wg, pair = 1 + i * 4 + (warp & 3);         // named barrier of the two warps with this warp's rows
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;      // TMEM lane 32 (w % 4) in bits 16 and up
    const uint32_t ts = tmem + lanes + i * 128, to = tmem + lanes + 256 + i * DP + half * (DP / 2);
    const uint32_t prow = base + L::P + i * L::PTILE + half * PANEL + r * 128;   // this thread's 64 weights: a panel's row
    const bool capped = a.softcap > 0.f;
    const Cap cap(a);
    const float f0 = a.scale * LOG2E;
    const float slope = a.slopes && valid ? a.slopes[head] * LOG2E : 0.f;
    // without cap and bias the scores stay products (of a positive scale) until the exponential
    const bool units = capped || a.slopes != nullptr || !(f0 > 0.f);
    const float f = units ? 1.f : f0, lazy = 8.f / f;
    // capped, unbiased bf16 scores: 0 in the maximum's place
    const bool fixed = BF && capped && a.slopes == nullptr && a.softcap <= 32.f;
    int lim = a.Skv;
    if (a.causal) lim = min(lim, max(pos + 1, a.prefix ? a.prefix[b] : 0));
    const int first_pos = (a.pack > 1 ? 0 : qt * TA_TILE) + off;
    int full = a.Skv;                                        // keys below it are seen by every row, documents apart
    if (a.causal) full = min(full, max(first_pos + 1, a.prefix ? a.prefix[b] : 0));
    float m = fixed ? 0.f : -INFINITY, l = 0.f, lr = 0.f;   // lr: of the rounded weights
    const bool few = alt || ntile <= 4 || a.slopes != nullptr;
    const int step = alt ? 2 : 1, end = i ? hi1 : hi0;
    int cnt = 0;
    // Padding may hold NaN, and 0 NaN is NaN: its value rows become zeros, a row a thread.
    const auto clean = [&](int n) {
      const int k = value_place<ALT>(n - lo, ntile), j = n * TA_TILE + r;
      mbar_wait(&kv_full[k % nst], (k / nst) & 1, abort);
      if (half == 0 && j < a.Skv && a.docs[(int64_t)b * a.Skv + j] < 0) zero_row<DP>(stage_at(k % nst), r);
      __syncwarp();
    };
    // a warp without a query leaves its rows of the weights as they are (the products of a row are its own) and only keeps step
    const bool none = !__any_sync(0xffffffffu, valid);
    // a wait that gives up (dead is set) only spoils values: every barrier below is still passed
    for (int n = lo + (alt ? i : 0); n < end; n += step, cnt++) {
      mbar_wait(&s_full[i], cnt & 1, abort);
      __syncwarp();
      if (none) {
        mbar_arrive(&s_read[i]);
        if (cnt > 0) mbar_wait(&pv_done[i], (cnt - 1) & 1, abort);
        if (a.docs && a.bounds[(int64_t)b * a.ktiles + n].neg) clean(n);
        mbar_arrive(&p_full[i]);
        continue;
      }
      fence_after();
      float v[64];
      ld_x32(ts + half * 64, v);
      ld_x32(ts + half * 64 + 32, v + 32);
      ld_wait();
      fence_before();
      mbar_arrive(&s_read[i]);
      const int j0 = n * TA_TILE + half * 64;
      bool masked = (n + 1) * TA_TILE > full, padded = false, vote = true;   // padded: keys; vote: no padding at all
      if (a.docs) {
        const TaBounds bd = a.bounds[(int64_t)b * a.ktiles + n];
        padded = bd.neg;
        vote = !(bd.neg || qdoc[i][2]);
        masked |= !vote || bd.lo != bd.hi || bd.lo != qdoc[i][0] || bd.lo != qdoc[i][1];
      }
      if (capped) {
        cap.apply<32>(v, vote);
        cap.apply<32>(v + 32, vote);
      } else if (units) {
#pragma unroll
        for (int c = 0; c < 64; c++) v[c] *= f0;
      }
      if (a.slopes) {
        const float d0 = (float)(pos - j0);
#pragma unroll
        for (int c = 0; c < 64; c++) v[c] = __fmaf_rn(-slope, fabsf(d0 - (float)c), v[c]);
      }
      if (masked) {
        uint32_t see[2];
        first_bits<64>(see, lim - j0);
        if (a.docs) same_doc<64>(see, a.docs + (int64_t)b * a.Skv + j0, a.Skv - j0, doc);
#pragma unroll
        for (int c = 0; c < 64; c++)
          if (!(see[c >> 5] & (1u << (c & 31)))) v[c] = -INFINITY;
      }
      if (!fixed) {
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 8)
#pragma unroll
        for (int e = 0; e < 4; e++) top[e] = max3(top[e], v[c + 2 * e], v[c + 2 * e + 1]);
      const float mine = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      // Whether a row's maximum has to move is asked of both threads' maxima as bf16 rounded up, two sets of words by turns, so
      // one barrier does.  That is up to 2^-7 of the score above it, so where it moves the maximum itself passes, through the
      // weights' tile: rows that only these two warps write, free once the product before has read them.
      const bool first = cnt == 0;
      bool grow = first;
      if (!first) {
        uint16_t* const at = exchange + (cnt & 1) * 512 + i * 256 + r;
        at[half * 128] = __bfloat16_as_ushort(__float2bfloat16_ru(mine));
        bar_sync(pair, 64);
        grow = fmaxf(__bfloat162float(__ushort_as_bfloat16(at[0])), __bfloat162float(__ushort_as_bfloat16(at[128]))) > m + lazy;
      }
      if (__any_sync(0xffffffffu, grow)) {   // the same in both warps of these rows
        if (!first) {
          mbar_wait(&pv_done[i], (cnt - 1) & 1, abort);
          __syncwarp();
          fence_after();
        }
        float* const at = reinterpret_cast<float*>(raw + (base - smem_addr(raw)) + L::P + i * L::PTILE + (warp & 3) * 4096) + lane;
        at[half * 32] = mine;
        bar_sync(pair, 64);
        const float mn = grow ? fmaxf(m, fmaxf(at[0], at[32])) : m;
        const float k = mn == m ? 1.f : ex2(m * f - mn * f);   // of the shifts as rounded: the weights were taken with them
        l *= k;
        lr *= k;
        m = mn;
        if (!first) {
#pragma unroll
          for (int c = 0; c < DP / 2; c += 16) {   // 16 at a time: the scores are live
            float o[16];
            uint32_t w[16];
            ld_x16(to + c, o);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; e++) w[e] = __float_as_uint(o[e] * k);
            st_x16(to + c, w);
          }
          st_wait();
        }
        bar_sync(pair, 64);   // both have read the words that the weights take next
      }
      }
      const float mf = m == -INFINITY ? 0.f : m * f;
      u64 sum[2] = {0, 0}, rounded = 0;
      const u64 ff = f2::splat(f), shift = f2::splat(-mf);
      if (cnt > 0) {   // the product before has read the weights' tile
        mbar_wait(&pv_done[i], (cnt - 1) & 1, abort);
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < 8; u += 4) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          f2::unpack(f2::fma(f2::pack(v[8 * u + e], v[8 * u + e + 1]), ff, shift), x, y);
          x = ex2(x);
          y = ex2(y);
          sum[(e >> 1) & 1] = f2::add(sum[(e >> 1) & 1], f2::pack(x, y));
          p[e >> 1] = pack16<BF>(x, y);
        }
        if (few) {
#pragma unroll
          for (int e = 0; e < 16; e++) rounded = f2::add(rounded, unpack16<BF>(p[e]));
        }
#pragma unroll
        for (int w = 0; w < 4; w++)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + (((u + w) ^ (r & 7)) << 4)), "r"(p[4 * w]),
                       "r"(p[4 * w + 1]), "r"(p[4 * w + 2]), "r"(p[4 * w + 3])
                       : "memory");
      }
      {
        float x, y;
        f2::unpack(f2::add(sum[0], sum[1]), x, y);
        l += x + y;
        f2::unpack(rounded, x, y);
        lr += x + y;
      }
      if (padded) clean(n);
      fence_async_smem();
      fence_before();
      mbar_arrive(&p_full[i]);
    }
    if (cnt > 0) mbar_wait(&pv_done[i], (cnt - 1) & 1, abort);
    if (ntile > 0) mbar_wait(&q_full, 0, abort);   // a group without key tiles still reuses its query tile below
    __syncwarp();
    fence_after();
    {   // the row's sum, by way of the weights' tile, which is no longer read
      float* const at = reinterpret_cast<float*>(raw + (base - smem_addr(raw)) + L::P + i * L::PTILE) + r;
      bar_sync(9 + i, 256);
      at[half * 128] = l;
      at[256 + half * 128] = lr;
      bar_sync(pair, 64);
      l = at[0] + at[128];
      lr = few ? at[256] + at[384] : l;
    }
    if (valid && !isfinite(l) && half == 0 && a.status) atomicOr(a.status, DA_STATUS_NONFINITE);
    __syncwarp();
    float lse = l > 0.f ? (m * f + log2f(l)) * LN2 : l == 0.f ? -INFINITY : l;
    if (alt && a.splits == 1) {
      // one CTA holds all keys: the second group hands its sums to the first through the weights' tiles
      unsigned char* const room = raw + (base - smem_addr(raw)) + L::P;
      float4* const stat = reinterpret_cast<float4*>(exchange);
      const auto at = [&](int c) { return reinterpret_cast<float4*>(room + r * (DP * 4) + (((half * (DP / 2) + c) >> 2) ^ (r & 7)) * 16); };
      bar_sync(11, 512);
      if (i == 1) {
        if (half == 0) stat[r] = make_float4(m * f, l, lr, 0.f);
        if (cnt > 0) {
#pragma unroll 1
          for (int c = 0; c < DP / 2; c += 16) {
            float x[16];
            ld_x16(to + c, x);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; e += 4) *at(c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
        }
      }
      bar_sync(11, 512);
      if (i == 0) {
        const float4 other = stat[r];
        const float m0 = m * f, top = fmaxf(l != 0.f ? m0 : -INFINITY, other.y != 0.f ? other.x : -INFINITY);
        const float k0 = l != 0.f ? ex2(m0 - top) : 0.f, k1 = other.y != 0.f ? ex2(other.x - top) : 0.f;
        const float all = l * k0 + other.y * k1, by = lr * k0 + other.z * k1, inv = by > 0.f ? 1.f / by : by;
        lse = all > 0.f ? (top + log2f(all)) * LN2 : all == 0.f ? -INFINITY : all;
        const bool more = ntile > 1;
        const uint32_t tile = base + L::Q;
#pragma unroll 1
        for (int c = 0; c < DP / 2; c += 16) {
          float x[16];
          if (cnt > 0) {
            ld_x16(to + c, x);
            ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (more && k1 > 0.f) y = *at(c + e);
            const float o[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int w = 0; w < 4; w++) x[e + w] = (cnt > 0 ? __fmaf_rn(x[e + w], k0, o[w] * k1) : 0.f) * inv;
          }
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const int col = half * (DP / 2) + c + 8 * u;
            const uint32_t to_smem = tile + (col >> 6) * PANEL + r * 128 + ((((col & 63) >> 3) ^ (r & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to_smem), "r"(pack16<BF>(x[8 * u], x[8 * u + 1])),
                         "r"(pack16<BF>(x[8 * u + 2], x[8 * u + 3])), "r"(pack16<BF>(x[8 * u + 4], x[8 * u + 5])),
                         "r"(pack16<BF>(x[8 * u + 6], x[8 * u + 7]))
                         : "memory");
          }
        }
      }
    } else if (!alt) {
      const uint32_t tile = base + L::Q + i * TILE;
      row_out<BF, DP / 2>(tile, tmem + lanes + 256 + i * DP, tmem + lanes + 256 + i * DP, r, half * (DP / 2),
                          lr > 0.f ? 1.f / lr : lr, 0.f, cnt > 0);   // a row that sees nothing: zeros times zero
    }
    if (!alt || a.splits == 1) {
      const bool mine = qt < a.qtiles && !(alt && i == 1);
      fence_async_smem();
      bar_sync(9 + i, 256);
      if (r == 0 && half == 0 && mine && !dead) {
        const uint32_t tile = base + L::Q + (alt ? 0 : i * TILE);
        for (int p = 0; p < DP / 64; p++)
          if (p * 64 < a.D) {
            if (a.pack > 1) tma_store(&a.o, tile + p * PANEL, p * 64, 0, 0, h, b);
            else tma_store(&a.o, tile + p * PANEL, p * 64, 0, qt * TA_TILE, h, b);
          }
        tma_store_commit();
        tma_store_wait();
      }
      if (a.lse && half == 0 && valid && mine) a.lse[((int64_t)b * a.Hq + head) * a.Sq + qi] = lse;
    } else {
      const int64_t row = ((int64_t)(2 * z + i) * HB + hb) * TA_TILE + r;
      float* o = a.part + row * DP + half * (DP / 2);
      float4* stat = reinterpret_cast<float4*>(a.part + (int64_t)2 * a.splits * HB * TA_TILE * DP) + row;
      if (valid && half == 0) *stat = make_float4(m * f, l, lr, 0.f);
#pragma unroll 1
      for (int c = 0; c < DP / 2; c += 16) {
        float x[16];
        if (cnt > 0) {
          ld_x16(to + c, x);
          ld_wait();
        }
        if (valid && cnt > 0) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(o + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
      }
    }
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;" ::: "memory");   // as the control group, for what follows
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x == 0 && dead && a.status) atomicOr(a.status, DA_STATUS_TIMEOUT);
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// Joins the key ranges of the split forward: one warp a query row, the ranges in their order.
template <int DP, bool BF>
__global__ void __launch_bounds__(128) ta_join_kernel(const __grid_constant__ TaArgs a) {
  using namespace tc5;
  const int NH = a.Hq / a.pack, HB = a.B * NH, np = 2 * a.splits;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (int64_t)HB * a.pack * a.Sq) return;
  const int rows = a.pack * a.Sq, hb = (int)(w / rows), r = (int)(w % rows);
  const int b = hb / NH, qi = r / a.pack, head = hb % NH * a.pack + r % a.pack;
  const float4* ml = reinterpret_cast<const float4*>(a.part + (int64_t)np * HB * TA_TILE * DP);
  float top = -INFINITY;
  for (int p = lane; p < np; p += 32) top = fmaxf(top, ml[((int64_t)p * HB + hb) * TA_TILE + r].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  constexpr int E = DP / 32;
  float sum[E] = {}, l = 0.f, lr = 0.f;
#pragma unroll 4
  for (int p = 0; p < np; p++) {
    const int64_t row = ((int64_t)p * HB + hb) * TA_TILE + r;
    const float4 x = ml[row];
    const bool some = x.y != 0.f;                 // a range without visible keys wrote no sums
    const float k = some ? ex2(x.x - top) : 0.f;
    l = __fmaf_rn(x.y, k, l);
    lr = __fmaf_rn(x.z, k, lr);
#pragma unroll
    for (int e = 0; e < E; e++) {
      const float o = some ? a.part[row * DP + lane * E + e] : 0.f;
      sum[e] = __fmaf_rn(o, k, sum[e]);
    }
  }
  const float inv = lr > 0.f ? 1.f / lr : lr;     // NaN stays
  uint16_t* out = (uint16_t*)a.out + b * a.os[0] + head * a.os[1] + qi * a.os[2];
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const uint32_t x = pack16<BF>(sum[e] * inv, sum[e + 1] * inv);
    if (lane * E + e < a.D) *reinterpret_cast<uint32_t*>(out + lane * E + e) = x;   // D is even
  }
  if (a.lse && lane == 0)
    a.lse[((int64_t)b * a.Hq + head) * a.Sq + qi] = l > 0.f ? (top + log2f(l)) * ta::LN2 : l == 0.f ? -INFINITY : l;
}

// Dynamic shared memory of a kernel with `tiles` bytes of 1024-byte aligned tiles: with up to 1024 bytes of static shared
// memory before them the tiles are aligned within the 227 KB of a CTA.  One object a kernel.
class TileSmem {
  DeviceOnce once;
  std::atomic<int> fixed{-1};   // bytes of static shared memory: the kernel's, on every device

 public:
  template <typename K>
  cudaError_t ready(K kernel, int tiles, int* bytes) {
    int before = fixed.load(std::memory_order_relaxed);
    if (before < 0) {
      cudaFuncAttributes at;
      const cudaError_t e = cudaFuncGetAttributes(&at, kernel);
      if (e != cudaSuccess) return e;
      if (at.sharedSizeBytes > 1024) return cudaErrorInvalidConfiguration;
      fixed.store(before = (int)at.sharedSizeBytes, std::memory_order_relaxed);
    }
    *bytes = tiles + 1024 - before;
    return allow_smem(once, kernel, *bytes);
  }
};

template <int DP, bool BF>
cudaError_t ta_forward(const TaArgs& a, cudaStream_t st) {
  using L = TaFwdSmem<DP>;
  static TileSmem smem[2];
  const bool alt = a.splits > 0;
  int bytes;
  const auto kernel = alt ? ta_fwd_kernel<DP, BF, true> : ta_fwd_kernel<DP, BF, false>;
  if (const cudaError_t e = smem[alt].ready(kernel, L::END, &bytes)) return e;
  const int HB = a.B * (a.Hq / a.pack);
  const unsigned grid = (unsigned)HB * (alt ? a.splits * a.qtiles : (a.qtiles + 1) / 2);
  kernel<<<grid, TA_FWD_THREADS, bytes, st>>>(a);
  if (a.splits > 1) {
    const int64_t rows = (int64_t)HB * a.pack * a.Sq;
    ta_join_kernel<DP, BF><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace detattn
