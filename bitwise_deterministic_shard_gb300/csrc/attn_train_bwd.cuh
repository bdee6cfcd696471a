// Backward passes of the training attention.
//
//   p = exp(s - lse);  dp = grad.v;  ds = p (dp - delta) (1 - tanh^2);  delta = grad.out
//   dv_j = sum_i p_ij grad_i;  dk_j = scale sum_i ds_ij q_i;  dq_i = scale sum_j ds_ij k_j
//
// delta from the rounded output is off by the output's rounding, and where a row's weight lies on few keys
// ds is a small difference that this spoils (dq 5e-3 off, four times the rounding of the result).  The
// kernel that runs over a query's keys therefore also sums D = sum p dp and E = sum p (1 - tanh^2) k,
// corrects dq by (delta - D) E, and hands D to the other kernel, which runs after it.
//
// Two kernels, so that every sum has one owner and a fixed order without atomics: one keeps a tile of
// 128 keys and runs over the queries (and the query heads that share the key head), one keeps a
// tile of 128 queries and runs over the keys.  That is eight products a tile pair (seven without
// E) instead of the five of a single kernel whose dq would be added by atomics in any order.
//
// Eight warps compute: a TMEM lane (tile row) has two threads, each with 64 of the 128 columns.
// One warp copies, one issues the products:
//   keys kept:    S^T = K Q^T;  dP^T = V G^T;  dV += P^T G;  dK += dS^T Q      TMEM 2 x 128 + 2 x D
//   queries kept: S = Q K^T;    dP = G V^T;    E += P K;      dQ += dS K       TMEM 2 x 128 + 2 x D
// P and dS overwrite, as 16-bit A operands, the scores and products they came from.  The tensor cores run
// the products of a step in the shadow of the other half of it: dV or E and the next S while dS is
// computed, dK or dQ and the next dP while the next P is.  P and dS are rounded to the inputs' type, the sums
// are binary32.
#pragma once
#include "../../include/detattn.h"
#include "attn_train.h"
#include "attn_train_fwd.cuh"

namespace detattn {

// Query tiles [lo, hi) that may see the key tile n.  A whole warp calls it.
namespace ta {
__device__ __forceinline__ int2 query_range(const TaArgs& a, int b, int n) {
  const int j0 = n * TA_TILE, off = a.Skv - a.Sq;
  int q0 = 0, q1 = a.qtiles;
  if (a.causal && !(a.prefix && j0 < a.prefix[b])) q0 = max(0, j0 - off) / TA_TILE;
  if (a.docs) {
    const TaBounds kb = a.bounds[(int64_t)b * a.ktiles + n];
    const TaBounds* qb = a.qbounds + (int64_t)b * a.qtiles;
    int f = q1, l = -1;
    for (int q = q0 + (threadIdx.x & 31); q < q1; q += 32)
      if (qb[q].lo <= kb.hi && qb[q].hi >= kb.lo) {
        f = min(f, q);
        l = max(l, q);
      }
    q0 = __reduce_min_sync(0xffffffffu, f);
    q1 = __reduce_max_sync(0xffffffffu, l) + 1;
    if (q1 <= q0) q0 = q1 = 0;
  }
  return make_int2(q0, max(q0, q1));
}

}  // namespace ta

template <int DP>
struct TaBwdSmem {
  static constexpr int TILE = DP / 64 * tc5::PANEL;
  static constexpr int NST = 2;
  // two kept tiles, then stages of two tiles and 128 (lse, delta) pairs
  static constexpr int KEEP = 0, ST = 2 * TILE, STAGE = 2 * TILE + 1024, END = ST + NST * STAGE;
  static constexpr int BYTES = END + 1024;
};

// ---- keys kept: dK and dV ----
template <int DP, bool BF>
__global__ void __launch_bounds__(320, 1) ta_dkv_kernel(const __grid_constant__ TaArgs a) {
  using namespace tc5;
  using namespace ta;
  using L = TaBwdSmem<DP>;
  constexpr int NST = L::NST, TILE = L::TILE;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t kv_full, q_full[NST], q_empty[NST], s_full, dp_full, p_full, ds_full, done, gone;
  __shared__ uint32_t tmem_at;
  __shared__ int dead, range[2];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  unsigned char* const gen = raw + (base - smem_addr(raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &dead;
  const int HB = a.B * a.Hkv, hb = blockIdx.x % HB, b = hb / a.Hkv, kh = hb % a.Hkv;
  const int n = blockIdx.x / HB;                 // the first keys first: with causal masking the longest
  const int off = a.Skv - a.Sq;

  if (threadIdx.x == 0) {
    dead = 0;
    mbar_init(&kv_full, 1);
    for (int s = 0; s < NST; s++) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&p_full, 256);
    mbar_init(&ds_full, 256);
    mbar_init(&done, 1);
    mbar_init(&gone, 1);
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(&tmem_at, 512);
  if (warp == 8) {
    const int2 r = query_range(a, b, n);
    if (lane == 0) {
      range[0] = r.x;
      range[1] = r.y;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_at;
  const int q0 = range[0], nq = range[1] - q0, total = nq * a.group;

  if (warp == 8) {
    if (lane == 0 && total > 0) {
      mbar_expect_tx(&kv_full, 2 * TILE);
      for (int p = 0; p < DP / 64; p++) {
        tma_load(base + L::KEEP + p * PANEL, &a.k, p * 64, 0, n * TA_TILE, kh, b, &kv_full);
        tma_load(base + L::KEEP + TILE + p * PANEL, &a.v, p * 64, 0, n * TA_TILE, kh, b, &kv_full);
      }
      bool ok = true;
      int it = 0;
      for (; it < total; it++) {
        const int s = it % NST, h = kh * a.group + it / nq, q = q0 + it % nq;
        if (it >= NST) ok = mbar_wait(&q_empty[s], ((it / NST) - 1) & 1, abort);
        if (!ok) break;
        const uint32_t at = base + L::ST + s * L::STAGE;
        mbar_expect_tx(&q_full[s], 2 * TILE + 1024);
        for (int p = 0; p < DP / 64; p++) {
          tma_load(at + p * PANEL, &a.q, p * 64, 0, q * TA_TILE, h, b, &q_full[s]);
          tma_load(at + TILE + p * PANEL, &a.go, p * 64, 0, q * TA_TILE, h, b, &q_full[s]);
        }
        bulk_g2s(gen + L::ST + s * L::STAGE + 2 * TILE, a.rows + (((int64_t)b * a.Hq + h) * a.qtiles + q) * TA_TILE, 1024,
                 &q_full[s]);
      }
      for (int k = max(0, it - NST); k < it; k++) mbar_drain(&q_full[k % NST], (k / NST) & 1);
      mbar_drain(&kv_full, 0);
    }
  } else if (warp == 9) {
    const int steps = same(total);
    if (steps > 0) {
      const uint32_t one = elect(), tm = same(tmem);
      const uint32_t id_s = idesc<BF>(128, 128, false), id_o = idesc<BF>(128, DP, true);
      const uint32_t ts = tm, tp = tm + 128, tv = tm + 256, tk = tm + 256 + DP;
      const uint32_t ktile = base + L::KEEP, vtile = ktile + TILE;
      auto stage = [&](int it) { return base + L::ST + (it % NST) * L::STAGE; };
      auto scores = [&](int it) {
#pragma unroll
        for (int s = 0; s < DP / 16; s++) mma_ss(ts, desc_k(ktile, s), desc_k(stage(it), s), id_s, s > 0, one);
        commit_one(&s_full, one);
      };
      auto grads = [&](int it) {
#pragma unroll
        for (int s = 0; s < DP / 16; s++) mma_ss(tp, desc_k(vtile, s), desc_k(stage(it) + TILE, s), id_s, s > 0, one);
        commit_one(&dp_full, one);
      };
      bool ok = all_of(mbar_wait(&kv_full, 0, abort) && mbar_wait(&q_full[0], 0, abort));
      if (ok) {
        fence_after();
        scores(0);
        grads(0);
      }
      for (int it = 0; it < steps && ok; it++) {
        ok = all_of(mbar_wait(&p_full, it & 1, abort));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int s = 0; s < 8; s++) mma_ts(tv, ts + 8 * s, desc_mn(stage(it) + TILE, s), id_o, s > 0 || it > 0, one);
        if (it + 1 < steps) {
          ok = all_of(mbar_wait(&q_full[(it + 1) % NST], ((it + 1) / NST) & 1, abort));
          if (!ok) break;
          scores(it + 1);
        }
        ok = all_of(mbar_wait(&ds_full, it & 1, abort));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int s = 0; s < 8; s++) mma_ts(tk, tp + 8 * s, desc_mn(stage(it), s), id_o, s > 0 || it > 0, one);
        commit_one(&q_empty[it % NST], one);
        if (it + 1 < steps) grads(it + 1);
      }
      commit_one(&done, one);
      if (!ok) {
        commit_one(&gone, one);
        mbar_drain(&gone, 0);
      }
    }
  } else {
    const int r = threadIdx.x & 127, half = threadIdx.x >> 7, j = n * TA_TILE + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + lanes, tp = ts + 128;
    const bool cap = a.softcap > 0.f;
    const float capx = cap ? a.scale / a.softcap : 0.f;
    const float f0 = (cap ? a.softcap : a.scale) * LOG2E;
    const bool free_key = !a.causal || (a.prefix && j < a.prefix[b]);
    const int doc = a.docs && j < a.Skv ? a.docs[(int64_t)b * a.Skv + j] : -1;
    TaBounds kb{};
    if (a.docs) kb = a.bounds[(int64_t)b * a.ktiles + n];
    const int free_below = a.causal && a.prefix ? a.prefix[b] : a.causal ? 0 : 0x7fffffff;
    // a wait that gives up (dead is set) only spoils values: every barrier below is still passed
    for (int it = 0; it < total; it++) {
      const int q = q0 + it % nq, h = kh * a.group + it / nq;
      const int pos0 = q * TA_TILE + off;
      const float slope = a.slopes ? a.slopes[h] * LOG2E : 0.f;
      bool padded = false, masked = (n + 1) * TA_TILE > a.Skv || ((n + 1) * TA_TILE - 1 > pos0 && (n + 1) * TA_TILE > free_below);
      if (a.docs) {
        const TaBounds qb = a.qbounds[(int64_t)b * a.qtiles + q];
        padded = kb.neg || qb.neg;
        masked |= padded || kb.lo != kb.hi || qb.lo != qb.hi || kb.lo != qb.lo;
      }
      const float4* rows = reinterpret_cast<const float4*>(gen + L::ST + (it % NST) * L::STAGE + 2 * TILE) + half * 32;
      mbar_wait(&s_full, it & 1, abort);
      mbar_wait(&q_full[it % NST], (it / NST) & 1, abort);
      __syncwarp();
      fence_after();
      float v[64];
      ld_x32(ts + half * 64, v);
      ld_x32(ts + half * 64 + 32, v + 32);
      ld_wait();
      // P may be written over the scores once both halves of the row have been read
      bar_sync(1 + (warp & 3), 64);
      const float d0 = (float)(pos0 + half * 64 - j);
      const int cmin = free_key ? -1 : j - pos0 - half * 64;   // the columns below it are hidden
      const int* dq = a.docs + (a.docs ? (int64_t)b * a.Skv + pos0 + half * 64 : 0);
      const int left = a.Sq - q * TA_TILE - half * 64;
#pragma unroll
      for (int g = 0; g < 2; g++) {
        uint32_t p16[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int c = 32 * g + e;
          const float4 row = rows[c >> 1];        // lse, delta of two queries
          float pp[2];
#pragma unroll
          for (int k = 0; k < 2; k++) {
            float x = v[c + k], dc = 1.f;
            if (cap) {
              x = tanh_any(x * capx);
              dc = __fmaf_rn(-x, x, 1.f);
            }
            float s = __fmaf_rn(x, f0, -(k ? row.z : row.x));
            if (a.slopes) s = __fmaf_rn(-slope, fabsf(d0 + (float)(c + k)), s);
            float p = ex2(s);
            dc *= p;
            if (masked) {
              bool see = c + k >= cmin && j < a.Skv;
              if (a.docs) see = see && c + k < left && doc >= 0 && dq[c + k] == doc;
              p = see ? p : 0.f;
              dc = see ? dc : 0.f;
            }
            pp[k] = p;
            v[c + k] = dc;
          }
          p16[e >> 1] = pack16<BF>(pp[0], pp[1]);
        }
        st_x16(ts + half * 32 + 16 * g, p16);
      }
      if (padded) {   // padding may hold NaN, and 0 NaN is NaN: its query and gradient rows become zeros
        const int i = q * TA_TILE + r;
        if (i < a.Sq && a.docs[(int64_t)b * a.Skv + i + off] < 0)
          zero_row<DP>(base + L::ST + (it % NST) * L::STAGE + half * TILE, r);
        __syncwarp();
      }
      st_wait();
      fence_before();
      mbar_arrive(&p_full);
      mbar_wait(&dp_full, it & 1, abort);
      __syncwarp();
      fence_after();
      float w[64];
      ld_x32(tp + half * 64, w);
      ld_x32(tp + half * 64 + 32, w + 32);
      ld_wait();
      bar_sync(1 + (warp & 3), 64);
      if (padded) {
#pragma unroll
        for (int c = 0; c < 64; c++) w[c] = v[c] == 0.f ? 0.f : w[c];
      }
#pragma unroll
      for (int g = 0; g < 2; g++) {
        uint32_t d16[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int c = 32 * g + e;
          const float4 row = rows[c >> 1];
          d16[e >> 1] = pack16<BF>(v[c] * (w[c] - row.y), v[c + 1] * (w[c + 1] - row.w));
        }
        st_x16(tp + half * 32 + 16 * g, d16);
      }
      st_wait();
      fence_before();
      mbar_arrive(&ds_full);
    }
    if (total > 0) mbar_wait(&done, 0, abort);
    __syncwarp();
    fence_after();
    // dK over the keys' tile, dV over the values': both are no longer read
    const uint32_t kt = base + L::KEEP, vt = kt + TILE;
    row_out<BF, DP / 2>(vt, tmem + lanes + 256, tmem + lanes + 256, r, half * (DP / 2), 1.f, 0.f, total > 0);
    row_out<BF, DP / 2>(kt, tmem + lanes + 256 + DP, tmem + lanes + 256 + DP, r, half * (DP / 2), a.scale, 0.f, total > 0);
    fence_async_smem();
    bar_sync(5, 256);
    if (threadIdx.x == 0 && !dead) {
      for (int p = 0; p < DP / 64; p++)
        if (p * 64 < a.D) {
          tma_store(&a.dk, kt + p * PANEL, p * 64, 0, n * TA_TILE, kh, b);
          tma_store(&a.dv, vt + p * PANEL, p * 64, 0, n * TA_TILE, kh, b);
        }
      tma_store_commit();
      tma_store_wait();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x == 0 && dead && a.status) atomicOr(a.status, DA_STATUS_TIMEOUT);
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---- queries kept: dQ ----
template <int DP, bool BF>
__global__ void __launch_bounds__(320, 1) ta_dq_kernel(const __grid_constant__ TaArgs a) {
  using namespace tc5;
  using namespace ta;
  using L = TaBwdSmem<DP>;
  constexpr int NST = L::NST, TILE = L::TILE;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t q_full, kv_full[NST], kv_empty[NST], s_full, dp_full, p_full, ds_full, done, gone;
  __shared__ uint32_t tmem_at;
  __shared__ int dead, range[2];
  __shared__ float delta_sum[2][128];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &dead;
  const int HB = a.B * a.Hq, hb = blockIdx.x % HB, b = hb / a.Hq, h = hb % a.Hq, kh = h / a.group;
  const int q = a.qtiles - 1 - blockIdx.x / HB, off = a.Skv - a.Sq, pos0 = q * TA_TILE + off;

  if (threadIdx.x == 0) {
    dead = 0;
    mbar_init(&q_full, 1);
    for (int s = 0; s < NST; s++) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&p_full, 256);
    mbar_init(&ds_full, 256);
    mbar_init(&done, 1);
    mbar_init(&gone, 1);
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(&tmem_at, 512);
  if (warp == 8) {
    TaBounds qb{};
    if (a.docs) qb = a.qbounds[(int64_t)b * a.qtiles + q];
    const int2 r = key_range(a, b, pos0, min(pos0 + TA_TILE, a.Skv) - 1, qb.lo, qb.hi);
    if (lane == 0) {
      range[0] = r.x;
      range[1] = r.y;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_at;
  const int n0 = range[0], total = range[1] - n0;

  if (warp == 8) {
    if (lane == 0 && total > 0) {
      mbar_expect_tx(&q_full, 2 * TILE);
      for (int p = 0; p < DP / 64; p++) {
        tma_load(base + L::KEEP + p * PANEL, &a.q, p * 64, 0, q * TA_TILE, h, b, &q_full);
        tma_load(base + L::KEEP + TILE + p * PANEL, &a.go, p * 64, 0, q * TA_TILE, h, b, &q_full);
      }
      bool ok = true;
      int it = 0;
      for (; it < total; it++) {
        const int s = it % NST;
        if (it >= NST) ok = mbar_wait(&kv_empty[s], ((it / NST) - 1) & 1, abort);
        if (!ok) break;
        const uint32_t at = base + L::ST + s * L::STAGE;
        mbar_expect_tx(&kv_full[s], 2 * TILE);
        for (int p = 0; p < DP / 64; p++) {
          tma_load(at + p * PANEL, &a.k, p * 64, 0, (n0 + it) * TA_TILE, kh, b, &kv_full[s]);
          tma_load(at + TILE + p * PANEL, &a.v, p * 64, 0, (n0 + it) * TA_TILE, kh, b, &kv_full[s]);
        }
      }
      for (int k = max(0, it - NST); k < it; k++) mbar_drain(&kv_full[k % NST], (k / NST) & 1);
      mbar_drain(&q_full, 0);
    }
  } else if (warp == 9) {
    const int steps = same(total);
    if (steps > 0) {
      const uint32_t one = elect(), tm = same(tmem);
      const uint32_t id_s = idesc<BF>(128, 128, false), id_o = idesc<BF>(128, DP, true);
      const uint32_t ts = tm, tp = tm + 128, tq = tm + 256, te = tm + 256 + DP;
      const uint32_t qtile = base + L::KEEP, gtile = qtile + TILE;
      auto stage = [&](int it) { return base + L::ST + (it % NST) * L::STAGE; };
      auto scores = [&](int it) {
#pragma unroll
        for (int s = 0; s < DP / 16; s++) mma_ss(ts, desc_k(qtile, s), desc_k(stage(it), s), id_s, s > 0, one);
        commit_one(&s_full, one);
      };
      auto grads = [&](int it) {
#pragma unroll
        for (int s = 0; s < DP / 16; s++) mma_ss(tp, desc_k(gtile, s), desc_k(stage(it) + TILE, s), id_s, s > 0, one);
        commit_one(&dp_full, one);
      };
      bool ok = all_of(mbar_wait(&q_full, 0, abort) && mbar_wait(&kv_full[0], 0, abort));
      if (ok) {
        fence_after();
        scores(0);
        grads(0);
      }
      for (int it = 0; it < steps && ok; it++) {
        ok = all_of(mbar_wait(&p_full, it & 1, abort));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int s = 0; s < 8; s++) mma_ts(te, ts + 8 * s, desc_mn(stage(it), s), id_o, s > 0 || it > 0, one);
        if (it + 1 < steps) {
          ok = all_of(mbar_wait(&kv_full[(it + 1) % NST], ((it + 1) / NST) & 1, abort));
          if (!ok) break;
          scores(it + 1);
        }
        ok = all_of(mbar_wait(&ds_full, it & 1, abort));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int s = 0; s < 8; s++) mma_ts(tq, tp + 8 * s, desc_mn(stage(it), s), id_o, s > 0 || it > 0, one);
        commit_one(&kv_empty[it % NST], one);
        if (it + 1 < steps) grads(it + 1);
      }
      commit_one(&done, one);
      if (!ok) {
        commit_one(&gone, one);
        mbar_drain(&gone, 0);
      }
    }
  } else {
    const int r = threadIdx.x & 127, half = threadIdx.x >> 7, qi = q * TA_TILE + r, pos = pos0 + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + lanes, tp = ts + 128;
    const bool cap = a.softcap > 0.f;
    const float capx = cap ? a.scale / a.softcap : 0.f;
    const float f0 = (cap ? a.softcap : a.scale) * LOG2E;
    const float slope = a.slopes ? a.slopes[h] * LOG2E : 0.f;
    float2* const my_row = a.rows + ((int64_t)b * a.Hq + h) * a.qtiles * TA_TILE + qi;
    const float2 row = *my_row;
    float delta[4] = {0.f, 0.f, 0.f, 0.f};
    const int doc = a.docs && qi < a.Sq ? a.docs[(int64_t)b * a.Skv + pos] : -1;
    TaBounds qb{};
    if (a.docs) qb = a.qbounds[(int64_t)b * a.qtiles + q];
    int lim = a.Skv, full = a.Skv;
    if (a.causal) {
      const int pre = a.prefix ? a.prefix[b] : 0;
      lim = min(lim, max(pos + 1, pre));
      full = min(full, max(pos0 + 1, pre));
    }
    for (int it = 0; it < total; it++) {   // a wait that gives up only spoils values, as above
      const int n = n0 + it, j0 = n * TA_TILE + half * 64;
      bool padded = false, masked = (n + 1) * TA_TILE > full;
      if (a.docs) {
        const TaBounds kb = a.bounds[(int64_t)b * a.ktiles + n];
        padded = kb.neg || qb.neg;
        masked |= padded || kb.lo != kb.hi || qb.lo != qb.hi || kb.lo != qb.lo;
      }
      mbar_wait(&s_full, it & 1, abort);
      __syncwarp();
      fence_after();
      float v[64];
      ld_x32(ts + half * 64, v);
      ld_x32(ts + half * 64 + 32, v + 32);
      ld_wait();
      bar_sync(1 + (warp & 3), 64);
      const float d0 = (float)(pos - j0);
      const int* dj = a.docs + (a.docs ? (int64_t)b * a.Skv + j0 : 0);
      const int left = a.Skv - j0;
      uint32_t hidden[2] = {0, 0};
      if (masked) {
#pragma unroll
        for (int c = 0; c < 64; c++) {
          bool see = j0 + c < lim;
          if (a.docs) see = see && c < left && doc >= 0 && dj[c] == doc;
          hidden[c >> 5] |= (see ? 0u : 1u) << (c & 31);
        }
      }
      float p[64];
#pragma unroll
      for (int g = 0; g < 2; g++) {
        uint32_t p16[16];
#pragma unroll
        for (int e = 0; e < 32; e++) {
          const int c = 32 * g + e;
          float x = v[c], dc = 1.f;
          if (cap) {
            x = tanh_any(x * capx);
            dc = __fmaf_rn(-x, x, 1.f);
          }
          float y = __fmaf_rn(x, f0, -row.x);
          if (a.slopes) y = __fmaf_rn(-slope, fabsf(d0 - (float)c), y);
          p[c] = ex2(y);
          v[c] = p[c] * dc;
          if (masked && (hidden[g] >> e & 1)) p[c] = v[c] = 0.f;
          if (e & 1) p16[e >> 1] = pack16<BF>(v[c - 1], v[c]);
        }
        st_x16(ts + half * 32 + 16 * g, p16);
      }
      if (padded) {   // padding may hold NaN: its key rows become zeros before a product sums over them
        const int j = n * TA_TILE + r;
        if (half == 0 && j < a.Skv && a.docs[(int64_t)b * a.Skv + j] < 0) zero_row<DP>(base + L::ST + (it % NST) * L::STAGE, r);
        __syncwarp();
      }
      st_wait();
      fence_before();
      mbar_arrive(&p_full);
      mbar_wait(&dp_full, it & 1, abort);
      __syncwarp();
      fence_after();
      float w[64];
      ld_x32(tp + half * 64, w);
      ld_x32(tp + half * 64 + 32, w + 32);
      ld_wait();
      bar_sync(1 + (warp & 3), 64);
      if (padded) {
#pragma unroll
        for (int c = 0; c < 64; c++) w[c] = p[c] == 0.f ? 0.f : w[c];
      }
#pragma unroll
      for (int c = 0; c < 64; c++) delta[c & 3] = __fmaf_rn(p[c], w[c], delta[c & 3]);
#pragma unroll
      for (int g = 0; g < 2; g++) {
        uint32_t d16[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int c = 32 * g + e;
          d16[e >> 1] = pack16<BF>(v[c] * (w[c] - row.y), v[c + 1] * (w[c + 1] - row.y));
        }
        st_x16(tp + half * 32 + 16 * g, d16);
      }
      st_wait();
      fence_before();
      mbar_arrive(&ds_full);
    }
    if (total > 0) mbar_wait(&done, 0, abort);
    __syncwarp();
    fence_after();
    // The sums were taken with delta from the rounded output; with D = sum p dp the gradient is
    // scale (sum ds k - (D - delta) sum p (1 - tanh^2) k).  D goes to the other kernel too.
    delta_sum[half][r] = (delta[0] + delta[1]) + (delta[2] + delta[3]);
    bar_sync(5, 256);
    const float exact = delta_sum[0][r] + delta_sum[1][r];
    if (half == 0 && !dead) my_row->y = exact;
    const uint32_t qt = base + L::KEEP;
    row_out<BF, DP / 2>(qt, tmem + lanes + 256, tmem + lanes + 256 + DP, r, half * (DP / 2), a.scale, row.y - exact, total > 0);
    fence_async_smem();
    bar_sync(5, 256);
    if (threadIdx.x == 0 && !dead) {
      for (int p = 0; p < DP / 64; p++)
        if (p * 64 < a.D) tma_store(&a.dq, qt + p * PANEL, p * 64, 0, q * TA_TILE, h, b);
      tma_store_commit();
      tma_store_wait();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x == 0 && dead && a.status) atomicOr(a.status, DA_STATUS_TIMEOUT);
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int DP, bool BF>
cudaError_t ta_dkv(const TaArgs& a, cudaStream_t st) {
  using L = TaBwdSmem<DP>;
  static const cudaError_t ready =
      cudaFuncSetAttribute(ta_dkv_kernel<DP, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (ready != cudaSuccess) return ready;
  ta_dkv_kernel<DP, BF><<<(unsigned)(a.B * a.Hkv) * a.ktiles, 320, L::BYTES, st>>>(a);
  return cudaGetLastError();
}

template <int DP, bool BF>
cudaError_t ta_dq(const TaArgs& a, cudaStream_t st) {
  using L = TaBwdSmem<DP>;
  static const cudaError_t ready =
      cudaFuncSetAttribute(ta_dq_kernel<DP, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (ready != cudaSuccess) return ready;
  if (a.qtiles == 0) return cudaSuccess;
  ta_dq_kernel<DP, BF><<<(unsigned)(a.B * a.Hq) * a.qtiles, 320, L::BYTES, st>>>(a);
  return cudaGetLastError();
}

}  // namespace detattn
