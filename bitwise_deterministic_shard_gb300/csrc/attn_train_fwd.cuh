// Forward pass of the training attention.
//
//   t = scale q.k;  u = cap tanh(t / cap);  s = u - slope |pos - j|;  hidden keys -inf
//   o = sum exp(s - m) v / sum exp(s - m);  lse = m + log sum exp(s - m)
//
// One CTA holds two tiles of 128 queries and runs over the key tiles once.  Per query tile a group of
// four warps owns one query row a thread: it reads its scores from TMEM, keeps the row's running
// maximum and sum in registers, and writes exp2 of the scores back to TMEM as 16-bit weights,
// over the scores they came from, where the second product takes them as its A operand.  The two
// groups alternate on the tensor cores: while one computes weights, the other's products run.  One
// warp copies tiles (tensor maps, a ring of key and value tiles), one issues all products:
//   S_i = Q_i K_n^T (128 x 128 x D),  O_i += P_i V_n (128 x D x 128).
// TMEM: two score tiles and two output tiles, 2 x 128 + 2 x D columns.
//
// The weights are rounded to the inputs' 16-bit type (the tensor cores take both operands in one
// type); the sum of the weights and the output are binary32.  The maximum is moved only when
// it grows by more than 2^8: until then weights are at most 2^8 too large, which the division by
// their sum undoes exactly, and the output needs no rescaling.
//
// Few queries (Sq * group <= 128): the heads that share a key head are the rows of one tile, so
// a cache is read once; both groups take the same queries and every other key tile, and the key range
// is split over CTAs so that all SMs read.  Each group writes its unnormalised sums, a second
// kernel joins them in a fixed order.
#pragma once
#include "../../include/detattn.h"
#include "attn_train.h"
#include "pack2.cuh"
#include "tc5_tile.cuh"

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

// tanh.  Any argument: 1 - 2 / (1 + e^2x), two operations of the special function unit, 2^-22 absolute.  On
// [-1, 1], where the scores of a capped model nearly always are: x P(x^2), P of degree 5 fitted for the least
// greatest error (least squares with weights moved toward the largest errors), 3.1e-7 absolute with
// binary32 steps, on the packed multiplier.  The special function unit would otherwise bound the kernel:
// three of its operations a score instead of one (forward 169 -> see above).
__device__ __forceinline__ float tanh_any(float x) {
  return __fmaf_rn(-2.f, tc5::rcp(1.f + tc5::ex2(x * (2.f * LOG2E))), 1.f);
}
__device__ __forceinline__ u64 tanh_small2(u64 x) {
  const u64 z = f2::mul(x, x);
  u64 p = f2::fma(f2::splat(-0x1.742c6ap-9f), z, f2::splat(0x1.0803b2p-6f));
  p = f2::fma(p, z, f2::splat(-0x1.a191cep-5f));
  p = f2::fma(p, z, f2::splat(0x1.0f6ea4p-3f));
  p = f2::fma(p, z, f2::splat(-0x1.553ce0p-2f));
  p = f2::fma(p, z, f2::splat(0x1.ffff96p-1f));
  return f2::mul(x, p);
}
// v <- tanh(k v) for N scores of each lane; the warp decides which form it takes
template <int N>
__device__ __forceinline__ void tanh_row(float* v, float k) {
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    m[0] = max3_abs(m[0], v[c], v[c + 1]);
    m[1] = max3_abs(m[1], v[c + 2], v[c + 3]);
  }
  if (__any_sync(0xffffffffu, !(fmaxf(m[0], m[1]) * fabsf(k) <= 1.f))) {
#pragma unroll
    for (int c = 0; c < N; c++) v[c] = tanh_any(v[c] * k);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 2)
      f2::unpack(tanh_small2(f2::mul(f2::pack(v[c], v[c + 1]), f2::splat(k))), v[c], v[c + 1]);
  }
}

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

}  // namespace ta

// Two softmax groups and a control group (copies, products, two idle warps).  setmaxnreg moves the control group's
// registers to the softmax threads, which hold a row's 128 scores: 384 x 168 at launch = 128 x 56 + 256 x 224.  The
// control group never takes its registers back: an idle warp's request would be met before the softmax groups'.
constexpr int TA_FWD_THREADS = 384;

template <int DP>
struct TaFwdSmem {
  static constexpr int TILE = DP / 64 * tc5::PANEL;
  static constexpr int NST = DP == 128 ? 5 : 8;
  static constexpr int Q = 0, KV = 2 * TILE, END = KV + NST * TILE;
  static constexpr int BYTES = END + 1024;
};

template <int DP, bool BF>
__global__ void __launch_bounds__(TA_FWD_THREADS, 1) ta_fwd_kernel(const __grid_constant__ TaArgs a) {
  using namespace tc5;
  using namespace ta;
  using L = TaFwdSmem<DP>;
  constexpr int NST = L::NST, TILE = L::TILE;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t q_full, kv_full[NST], kv_empty[NST], s_full[2], p_full[2], o_full[2], gone;
  __shared__ uint32_t tmem_at;
  __shared__ int dead, wdoc[8][2], range[2][2], qdoc[2][3];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &dead;

  const int NH = a.Hq / a.pack, HB = a.B * NH;
  const int hb = blockIdx.x % HB, b = hb / NH, h = hb % NH;
  const int kh = a.pack > 1 ? h : h / a.group;
  const bool alt = a.splits > 0;
  const int t = alt ? 0 : (int)(gridDim.x / HB) - 1 - blockIdx.x / HB;   // the last queries first: with causal masking the longest
  const int z = alt ? blockIdx.x / HB : 0;

  // this thread's query row (softmax groups)
  const int wg = warp >> 2, r = threadIdx.x & 127;
  const int qt = alt ? 0 : 2 * t + wg;
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
    for (int s = 0; s < NST; s++) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(&tmem_at, 512);
  if (wg < 2) {
    const int dl = __reduce_min_sync(0xffffffffu, doc < 0 ? 0x7fffffff : doc), dh = __reduce_max_sync(0xffffffffu, doc);
    const int neg = __any_sync(0xffffffffu, valid && doc < 0);
    if (lane == 0) {
      wdoc[warp][0] = dl;
      wdoc[warp][1] = neg ? -2 - dh : dh;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (wg < 2 && (warp & 3) == 0) {
    int dl = 0x7fffffff, dh = -1, neg = 0;
    for (int w = warp; w < warp + 4; w++) {
      int x = wdoc[w][1];
      if (x < -1) {
        neg = 1;
        x = -2 - x;
      }
      dl = min(dl, wdoc[w][0]);
      dh = max(dh, x);
    }
    const int q0 = (a.pack > 1 ? 0 : qt * TA_TILE) + off;
    const int q1 = (a.pack > 1 ? a.Sq : min(qt * TA_TILE + TA_TILE, a.Sq)) - 1 + off;
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

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");
  if (warp == 8) {
    // ---- copies: queries once, then keys and values in the order in which the products take them ----
    if (lane == 0 && ntile > 0) {
      const int nq = alt ? 1 : 2;
      const int rows = a.pack > 1 ? a.pack * a.qrows : TA_TILE;
      mbar_expect_tx(&q_full, nq * (DP / 64) * rows * 128);
      for (int i = 0; i < nq; i++)
        for (int p = 0; p < DP / 64; p++) {
          const int at = base + L::Q + i * TILE + p * PANEL;
          if (a.pack > 1) tma_load(at, &a.q, p * 64, 0, 0, h, b, &q_full);
          else tma_load(at, &a.q, p * 64, 0, min(2 * t + i, a.qtiles - 1) * TA_TILE, h, b, &q_full);
        }
      int it = 0;
      auto fetch = [&](const CUtensorMap* map, int n) -> bool {
        const int s = it % NST;
        if (it >= NST && !mbar_wait(&kv_empty[s], ((it / NST) - 1) & 1, abort)) return false;
        mbar_expect_tx(&kv_full[s], TILE);
        for (int p = 0; p < DP / 64; p++)
          tma_load(base + L::KV + s * TILE + p * PANEL, map, p * 64, 0, n * TA_TILE, kh, b, &kv_full[s]);
        it++;
        return true;
      };
      bool ok = fetch(&a.k, lo);
      if (alt && ok && lo + 1 < hi) ok = fetch(&a.k, lo + 1);
      const int ahead = alt ? 2 : 1;
      for (int n = lo; n < hi && ok; n++) {
        ok = fetch(&a.v, n);
        if (ok && n + ahead < hi) ok = fetch(&a.k, n + ahead);
      }
      // nothing may be in flight when the CTA ends
      for (int k = max(0, it - NST); k < it; k++) mbar_drain(&kv_full[k % NST], (k / NST) & 1);
      mbar_drain(&q_full, 0);
    }
  } else if (warp == 9) {
    // ---- products ----
    if (lane == 0 && ntile > 0) {
      const uint32_t id_s = idesc<BF>(128, 128, false), id_o = idesc<BF>(128, DP, true);
      int it = 0;
      auto wait_kv = [&](uint32_t& at) -> bool {
        const int s = it % NST;
        at = base + L::KV + s * TILE;
        return mbar_wait(&kv_full[s], (it / NST) & 1, abort);
      };
      auto scores = [&](int i, uint32_t ktile) {
        const uint32_t q = base + L::Q + (alt ? 0 : i * TILE);
#pragma unroll
        for (int s = 0; s < DP / 16; s++) mma_bf16(tmem + i * 128, desc_k(q, s), desc_k(ktile, s), id_s, s > 0);
        commit(&s_full[i]);
      };
      auto values = [&](int i, uint32_t vtile, bool first) {
#pragma unroll
        for (int s = 0; s < 8; s++)
          mma_ts(tmem + 256 + i * DP, tmem + i * 128 + 8 * s, desc_mn(vtile, s), id_o, s > 0 || !first);
      };
      uint32_t kt, vt;
      bool ok = mbar_wait(&q_full, 0, abort) && wait_kv(kt);
      fence_after();
      if (!alt) {
        if (ok) {
          if (lo < hi0) scores(0, kt);
          if (lo < hi1) scores(1, kt);
          commit(&kv_empty[it % NST]);
          it++;
        }
        for (int n = lo; n < hi && ok; n++) {
          ok = wait_kv(vt);
          if (!ok) break;
          const int vs = it++ % NST;
          bool have_k = false;
          for (int i = 0; i < 2 && ok; i++) {
            const int end = i ? hi1 : hi0;
            if (n < end) {
              ok = mbar_wait(&p_full[i], (n - lo) & 1, abort);
              if (!ok) break;
              fence_after();
              values(i, vt, n == lo);
              if (n + 1 == end) commit(&o_full[i]);
            }
            if (n + 1 < end) {
              if (!have_k) ok = wait_kv(kt);
              if (!ok) break;
              have_k = true;
              scores(i, kt);
            }
          }
          if (!ok) break;
          commit(&kv_empty[vs]);
          if (have_k) commit(&kv_empty[it++ % NST]);
        }
      } else {
        for (int i = 0; i < 2 && ok && lo + i < hi; i++) {
          if (i) ok = wait_kv(kt);
          if (!ok) break;
          scores(i, kt);
          commit(&kv_empty[it++ % NST]);
        }
        for (int n = lo; n < hi && ok; n++) {
          const int i = (n - lo) & 1;
          ok = wait_kv(vt) && mbar_wait(&p_full[i], ((n - lo) >> 1) & 1, abort);
          if (!ok) break;
          fence_after();
          values(i, vt, n - lo < 2);
          if (n + 2 >= hi) commit(&o_full[i]);
          commit(&kv_empty[it++ % NST]);
          if (n + 2 < hi) {
            ok = wait_kv(kt);
            if (!ok) break;
            scores(i, kt);
            commit(&kv_empty[it++ % NST]);
          }
        }
      }
      if (!ok) {
        commit(&gone);
        mbar_drain(&gone, 0);
      }
    }
  }
  } else {
    // ---- softmax ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;" ::: "memory");
    const int i = wg;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;      // TMEM lane 32 (w % 4) in bits 16 and up
    const uint32_t ts = tmem + lanes + i * 128, to = tmem + lanes + 256 + i * DP;
    const bool cap = a.softcap > 0.f;
    const float capx = cap ? a.scale / a.softcap : 0.f;
    const float f0 = (cap ? a.softcap : a.scale) * LOG2E;    // scores' units -> log2 units
    const float slope = a.slopes && valid ? a.slopes[head] * LOG2E : 0.f;
    const bool biased = a.slopes != nullptr || !(f0 > 0.f);  // applied before the maximum
    const float f = biased ? 1.f : f0;
    const float lazy = 8.f / f;
    int lim = a.Skv;
    if (a.causal) lim = min(lim, max(pos + 1, a.prefix ? a.prefix[b] : 0));
    const int first_pos = (a.pack > 1 ? 0 : qt * TA_TILE) + off;
    int full = a.Skv;                                        // keys below it are seen by every row, documents apart
    if (a.causal) full = min(full, max(first_pos + 1, a.prefix ? a.prefix[b] : 0));
    float m = -INFINITY, l = 0.f;
    const int step = alt ? 2 : 1, end = i ? hi1 : hi0;
    int cnt = 0;
    bool ok = true;
    for (int n = lo + (alt ? i : 0); n < end; n += step, cnt++) {
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[i], cnt & 1, abort));
      if (!ok) break;
      fence_after();
      float v[128];
#pragma unroll
      for (int c = 0; c < 4; c++) ld_x32(ts + 32 * c, v + 32 * c);
      ld_wait();
      const int j0 = n * TA_TILE;
      bool masked = j0 + TA_TILE > full, padded = false;
      if (a.docs) {
        const TaBounds bd = a.bounds[(int64_t)b * a.ktiles + n];
        padded = bd.neg;
        masked |= bd.neg || bd.lo != bd.hi || bd.lo != qdoc[i][0] || bd.lo != qdoc[i][1] || qdoc[i][2];
      }
      if (cap) {
#pragma unroll
        for (int c = 0; c < 4; c++) tanh_row<32>(v + 32 * c, capx);
      }
      if (biased) {
        const float d0 = (float)(pos - j0);
#pragma unroll
        for (int c = 0; c < 128; c++) v[c] = __fmaf_rn(v[c], f0, -slope * fabsf(d0 - (float)c));
      }
      if (masked) {
        if (a.docs) {
          const int* dj = a.docs + (int64_t)b * a.Skv + j0;
          const int left = a.Skv - j0;
#pragma unroll
          for (int c = 0; c < 128; c++) {
            const int d = c < left ? dj[c] : -1;
            if (j0 + c >= lim || d != doc || doc < 0) v[c] = -INFINITY;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 128; c++)
            if (j0 + c >= lim) v[c] = -INFINITY;
        }
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; c += 8)
#pragma unroll
        for (int e = 0; e < 4; e++) top[e] = max3(top[e], v[c + 2 * e], v[c + 2 * e + 1]);
      const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      const bool grow = cnt == 0 || mx > m + lazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? fmaxf(m, mx) : m;
        const float k = mn == m ? 1.f : ex2((m - mn) * f);
        l *= k;
        m = mn;
        if (cnt > 0) {
#pragma unroll
          for (int c = 0; c < DP / 32; c++) {
            float o[32];
            ld_x32(to + 32 * c, o);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] *= k;
            st_x32(to + 32 * c, o);
          }
        }
      }
      const float mf = m == -INFINITY ? 0.f : m * f;
      u64 sum[2] = {0, 0};
      const u64 ff = f2::splat(f), shift = f2::splat(-mf);
#pragma unroll
      for (int c = 0; c < 4; c++) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          f2::unpack(f2::fma(f2::pack(v[32 * c + e], v[32 * c + e + 1]), ff, shift), x, y);
          x = ex2(x);
          y = ex2(y);
          sum[(e >> 1) & 1] = f2::add(sum[(e >> 1) & 1], f2::pack(x, y));
          p[e >> 1] = pack16<BF>(x, y);
        }
        st_x16(ts + 16 * c, p);
      }
      {
        float x, y;
        f2::unpack(f2::add(sum[0], sum[1]), x, y);
        l += x + y;
      }
      if (padded) {   // padding may hold NaN, and 0 NaN is NaN: its value rows become zeros
        const int d = n - lo, k = alt ? min(ntile, d + 2) + d : 1 + 2 * d;   // this value tile in the order of the copies
        mbar_wait(&kv_full[k % NST], (k / NST) & 1, abort);
        if (j0 + r < a.Skv && a.docs[(int64_t)b * a.Skv + j0 + r] < 0) zero_row<DP>(base + L::KV + (k % NST) * TILE, r);
        __syncwarp();
      }
      st_wait();
      fence_before();
      mbar_arrive(&p_full[i]);
    }
    if (cnt > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(&o_full[i], 0, abort));
    if (ntile > 0) mbar_wait(&q_full, 0, abort);   // a group without key tiles still reuses its query tile below
    fence_after();
    if (valid && !isfinite(l) && a.status) atomicOr(a.status, DA_STATUS_NONFINITE);
    if (!alt) {
      const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
      const uint32_t tile = base + L::Q + i * TILE;
#pragma unroll
      for (int c = 0; c < DP / 32; c++) {
        float o[32];
        if (cnt > 0) {
          ld_x32(to + 32 * c, o);
          ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; e++) o[e] = cnt > 0 && l != 0.f ? o[e] * inv : 0.f;
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const int unit = (c & 1) * 4 + u;
          const uint32_t at = tile + (c >> 1) * PANEL + r * 128 + ((unit ^ (r & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack16<BF>(o[8 * u], o[8 * u + 1])),
                       "r"(pack16<BF>(o[8 * u + 2], o[8 * u + 3])), "r"(pack16<BF>(o[8 * u + 4], o[8 * u + 5])),
                       "r"(pack16<BF>(o[8 * u + 6], o[8 * u + 7]))
                       : "memory");
        }
      }
      fence_async_smem();
      bar_sync(1 + i, 128);
      if (r == 0 && qt < a.qtiles && ok) {
        for (int p = 0; p < DP / 64; p++)
          if (p * 64 < a.D) {
            if (a.pack > 1) {
              if (i == 0) tma_store(&a.o, tile + p * PANEL, p * 64, 0, 0, h, b);
            } else {
              tma_store(&a.o, tile + p * PANEL, p * 64, 0, qt * TA_TILE, h, b);
            }
          }
        tma_store_commit();
        tma_store_wait();
      }
      if (a.lse && valid && qt < a.qtiles)
        a.lse[((int64_t)b * a.Hq + head) * a.Sq + qi] = l > 0.f ? (m * f + log2f(l)) * LN2 : l == 0.f ? -INFINITY : l;
    } else {
      const int64_t row = ((int64_t)(2 * z + i) * HB + hb) * TA_TILE + r;
      float* o = a.part + row * DP;
      float2* ml = reinterpret_cast<float2*>(a.part + (int64_t)2 * a.splits * HB * TA_TILE * DP) + row;
      if (valid) *ml = make_float2(m * f, l);
#pragma unroll
      for (int c = 0; c < DP / 32; c++) {
        float x[32];
        if (cnt > 0) {
          ld_x32(to + 32 * c, x);
          ld_wait();
        }
        if (valid && cnt > 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(o + 32 * c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
      }
    }
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");   // as the control group, for what follows
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x == 0 && dead && a.status) atomicOr(a.status, DA_STATUS_TIMEOUT);
  if (warp == 9) tmem_dealloc(tmem, 512);
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
  const float2* ml = reinterpret_cast<const float2*>(a.part + (int64_t)np * HB * TA_TILE * DP);
  float top = -INFINITY;
  for (int p = lane; p < np; p += 32) top = fmaxf(top, ml[((int64_t)p * HB + hb) * TA_TILE + r].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  constexpr int E = DP / 32;
  float sum[E] = {}, l = 0.f;
#pragma unroll 4
  for (int p = 0; p < np; p++) {
    const int64_t row = ((int64_t)p * HB + hb) * TA_TILE + r;
    const float2 x = ml[row];
    const bool some = x.y != 0.f;                 // a range without visible keys wrote no sums
    const float k = some ? ex2(x.x - top) : 0.f;
    l = __fmaf_rn(x.y, k, l);
#pragma unroll
    for (int e = 0; e < E; e++) {
      const float o = some ? a.part[row * DP + lane * E + e] : 0.f;
      sum[e] = __fmaf_rn(o, k, sum[e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : l;        // NaN stays
  uint16_t* out = (uint16_t*)a.out + b * a.os[0] + head * a.os[1] + qi * a.os[2];
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const uint32_t x = pack16<BF>(sum[e] * inv, sum[e + 1] * inv);
    if (lane * E + e < a.D) *reinterpret_cast<uint32_t*>(out + lane * E + e) = x;   // D is even
  }
  if (a.lse && lane == 0)
    a.lse[((int64_t)b * a.Hq + head) * a.Sq + qi] = l > 0.f ? (top + log2f(l)) * ta::LN2 : l == 0.f ? -INFINITY : l;
}

template <int DP, bool BF>
cudaError_t ta_forward(const TaArgs& a, cudaStream_t st) {
  using L = TaFwdSmem<DP>;
  static const cudaError_t ready =
      cudaFuncSetAttribute(ta_fwd_kernel<DP, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (ready != cudaSuccess) return ready;
  const int HB = a.B * (a.Hq / a.pack);
  const unsigned grid = (unsigned)HB * (a.splits > 0 ? a.splits : (a.qtiles + 1) / 2);
  ta_fwd_kernel<DP, BF><<<grid, TA_FWD_THREADS, L::BYTES, st>>>(a);
  if (a.splits > 0) {
    const int64_t rows = (int64_t)HB * a.pack * a.Sq;
    ta_join_kernel<DP, BF><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace detattn
