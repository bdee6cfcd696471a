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
// Sixteen warps compute: a TMEM lane (tile row) has four threads, each with 32 of the 128 columns.
// One warp copies, one issues the products:
//   keys kept:    S^T = K Q^T;  dP^T = V G^T;  dV += P^T G;  dK += dS^T Q      TMEM 2 x 128 + 2 x D
//   queries kept: S = Q K^T;    dP = G V^T;    E += P K;      dQ += dS K       TMEM 2 x 128 + 2 x D
// P (times the cap's derivative for E) goes to shared memory as an A operand, so the next scores are computed as soon
// as the present ones are read (over the scores in TMEM it held them up by 1200 of 4500 cycles a step).  dS
// overwrites, as 16-bit A operand, the products it came from: each thread's 32 columns become the first 16 of the
// same 32, so no thread writes what another still reads; the next dP follows dK or dQ in the shadow of the next P.
// P and dS are rounded to the inputs' type, the sums are binary32.
//
// What bounds it: four products a tile pair in each kernel (2048 cycles; their shared-memory operands with the copies and
// P take about 2500) beside 1700 cycles of FP32 arithmetic with a cap, in steps of 3900 cycles: sixteen warps that pass the
// same phases together.  4096 causal, 16 heads, D 128, bf16, cap 30: dq 120 us, dk and dv 126 us (tensor pipe 52 and 50 %, issue
// slots 56 and 55 % of the cycles); eight warps of 64 columns with tanh from the special function unit took 341 each.
// Many CTAs of few steps (packed documents) pay about 3 us each for their start and end, and with shared key heads the
// longest of the dk and dv kernel's few CTAs set its end.
#pragma once
#include "../../include/detattn.h"
#include "attn_train.h"
#include "attn_train_fwd.cuh"
#include "train_math.cuh"

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

constexpr int TA_BWD_THREADS = 640;   // registers: 640 x 96 at launch = 128 x 32 + 512 x 112

template <int DP>
struct TaBwdSmem {
  static constexpr int TILE = DP / 64 * tc5::PANEL;
  static constexpr int NST = 2;
  // two kept tiles, stages of two tiles and 128 (-lse), 128 (-delta) of the queries, a tile of weights
  static constexpr int KEEP = 0, ST = 2 * TILE, STAGE = 2 * TILE + 1024, P = ST + NST * STAGE, END = P + 2 * tc5::PANEL;
};

namespace ta {
// the columns of a 16-deep step of the second products' A operand, within its 128 columns of TMEM
__device__ __forceinline__ uint32_t a_at(int s) { return (s >> 1) * 32 + (s & 1) * 8; }

template <int DP, bool BF>
struct Products {
  uint32_t ts, tp, t1, t2, one;           // scores, products with the gradient; the two sums
  uint32_t id_s, id_o;
  __device__ __forceinline__ void first(uint32_t d, uint32_t a, uint32_t b, uint64_t* bar) const {
    using namespace tc5;
#pragma unroll
    for (int s = 0; s < DP / 16; s++) mma_ss(d, desc_k(a, s), desc_k(b, s), id_s, s > 0, one);
    commit_one(bar, one);
  }
  __device__ __forceinline__ void weights(uint32_t a, uint32_t b, bool sum, uint64_t* bar) const {
    using namespace tc5;
#pragma unroll
    for (int s = 0; s < 8; s++) mma_ss(t1, desc_k(a, s), desc_mn(b, s), id_o, s > 0 || sum, one);
    commit_one(bar, one);
  }
  __device__ __forceinline__ void grads(uint32_t b, bool sum) const {
    using namespace tc5;
#pragma unroll
    for (int s = 0; s < 8; s++) mma_ts(t2, tp + a_at(s), desc_mn(b, s), id_o, s > 0 || sum, one);
  }
};

// A thread's 32 weights of row r: half a panel's row
template <bool BF>
__device__ __forceinline__ void put_weights(uint32_t tile, int r, int part, const float* p) {
  using namespace tc5;
  const uint32_t row = tile + (part >> 1) * PANEL + r * 128;
#pragma unroll
  for (int u = 0; u < 4; u++)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((((part & 1) * 4 + u) ^ (r & 7)) << 4)),
                 "r"(pack16<BF>(p[8 * u], p[8 * u + 1])), "r"(pack16<BF>(p[8 * u + 2], p[8 * u + 3])),
                 "r"(pack16<BF>(p[8 * u + 4], p[8 * u + 5])), "r"(pack16<BF>(p[8 * u + 6], p[8 * u + 7]))
                 : "memory");
}

// What turns a product of a query and a key into a score in log2 units, and that into the cap's derivative
// 1 - tanh^2 = 1 + inv2 score^2.
struct Scores {
  Cap cap;
  float f0, inv2;         // without a cap; minus one over the square of the cap's factor
  bool capped;
  __device__ __forceinline__ Scores(const TaArgs& a)
      : cap(a), f0(a.scale * LOG2E), capped(a.softcap > 0.f) {
    inv2 = -1.f / (a.cap.f * a.cap.f);
  }
};
}  // namespace ta

// ---- keys kept: dK and dV ----
template <int DP, bool BF>
__global__ void __launch_bounds__(TA_BWD_THREADS, 1) ta_dkv_kernel(const __grid_constant__ TaArgs a) {
  using namespace tc5;
  using namespace ta;
  using L = TaBwdSmem<DP>;
  constexpr int NST = L::NST, TILE = L::TILE;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t kv_full, q_full[NST], q_empty[NST], g_full[NST], g_empty[NST], s_full, s_read, dp_full, p_full, p_read, ds_full, done, gone;
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
      mbar_init(&g_full[s], 1);
      mbar_init(&g_empty[s], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&s_read, 512);
    mbar_init(&p_read, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&p_full, 512);
    mbar_init(&ds_full, 512);
    mbar_init(&done, 1);
    mbar_init(&gone, 1);
    mbar_fence_init();
  }
  if (warp == 17) tmem_alloc(&tmem_at, 512);
  if (warp == 16) {
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

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;" ::: "memory");
    if (warp == 16) {
      if (lane == 0 && total > 0) {
        mbar_expect_tx(&kv_full, 2 * TILE);
        for (int p = 0; p < DP / 64; p++) {
          tma_load(base + L::KEEP + p * PANEL, &a.k, p * 64, 0, n * TA_TILE, kh, b, &kv_full);
          tma_load(base + L::KEEP + TILE + p * PANEL, &a.v, p * 64, 0, n * TA_TILE, kh, b, &kv_full);
        }
        // a query tile stays until its second product, a gradient tile goes after its first and dV: apart, so that the next
        // scores only wait for the former
        const auto query = [&](int it) -> bool {
          const int s = it % NST, h = kh * a.group + it / nq, q = q0 + it % nq;
          if (it >= NST && !mbar_wait(&q_empty[s], ((it / NST) - 1) & 1, abort)) return false;
          const uint32_t at = base + L::ST + s * L::STAGE;
          mbar_expect_tx(&q_full[s], TILE + 1024);
          for (int p = 0; p < DP / 64; p++) tma_load(at + p * PANEL, &a.q, p * 64, 0, q * TA_TILE, h, b, &q_full[s]);
          bulk_g2s(gen + L::ST + s * L::STAGE + 2 * TILE, a.rows + (((int64_t)b * a.Hq + h) * a.qtiles + q) * 256, 1024,
                   &q_full[s]);
          return true;
        };
        const auto gradient = [&](int it) -> bool {
          const int s = it % NST, h = kh * a.group + it / nq, q = q0 + it % nq;
          if (it >= NST && !mbar_wait(&g_empty[s], ((it / NST) - 1) & 1, abort)) return false;
          const uint32_t at = base + L::ST + s * L::STAGE + TILE;
          mbar_expect_tx(&g_full[s], TILE);
          for (int p = 0; p < DP / 64; p++) tma_load(at + p * PANEL, &a.go, p * 64, 0, q * TA_TILE, h, b, &g_full[s]);
          return true;
        };
        int nqt = 0, ngt = 0;
        if (query(0)) nqt++;
        while (ngt < total && gradient(ngt)) {
          ngt++;
          if (nqt < total && !query(nqt)) break;
          if (nqt < total) nqt++;
        }
        for (int k = max(0, nqt - NST); k < nqt; k++) mbar_drain(&q_full[k % NST], (k / NST) & 1);
        for (int k = max(0, ngt - NST); k < ngt; k++) mbar_drain(&g_full[k % NST], (k / NST) & 1);
        mbar_drain(&kv_full, 0);
      }
    } else if (warp == 17) {
      const int steps = same(total);
      if (steps > 0) {
        const uint32_t tm = same(tmem);
        const Products<DP, BF> go{tm, tm + 128, tm + 256, tm + 256 + DP, elect(), idesc<BF>(128, 128, false), idesc<BF>(128, DP, true)};
        const uint32_t ktile = base + L::KEEP, vtile = ktile + TILE, st0 = base + L::ST;
        bool ok = all_of(mbar_wait(&kv_full, 0, abort) && mbar_wait(&q_full[0], 0, abort));
        if (ok) {
          fence_after();
          go.first(go.ts, ktile, st0, &s_full);
          ok = all_of(mbar_wait(&g_full[0], 0, abort));
          if (ok) go.first(go.tp, vtile, st0 + TILE, &dp_full);
        }
        for (int it = 0; it < steps && ok; it++) {
          const uint32_t st = st0 + (it % NST) * L::STAGE, next = st0 + ((it + 1) % NST) * L::STAGE;
          if (it + 1 < steps) {
            ok = all_of(mbar_wait(&s_read, it & 1, abort) && mbar_wait(&q_full[(it + 1) % NST], ((it + 1) / NST) & 1, abort));
            if (!ok) break;
            fence_after();
            go.first(go.ts, ktile, next, &s_full);
          }
          ok = all_of(mbar_wait(&p_full, it & 1, abort));
          if (!ok) break;
          fence_after();
          go.weights(base + L::P, st + TILE, it > 0, &p_read);
          if (it + NST < steps) commit_one(&g_empty[it % NST], go.one);   // only where the copies wait for it, as below
          ok = all_of(mbar_wait(&ds_full, it & 1, abort));
          if (!ok) break;
          fence_after();
          go.grads(st, it > 0);
          if (it + NST < steps) commit_one(&q_empty[it % NST], go.one);
          if (it + 1 < steps) {
            ok = all_of(mbar_wait(&g_full[(it + 1) % NST], ((it + 1) / NST) & 1, abort));
            if (ok) go.first(go.tp, vtile, next + TILE, &dp_full);
          }
        }
        commit_one(&done, go.one);
        if (!ok) {
          commit_one(&gone, go.one);
          mbar_drain(&gone, 0);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;" ::: "memory");
    const int r = threadIdx.x & 127, part = threadIdx.x >> 7, j = n * TA_TILE + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + lanes + part * 32, tp = ts + 128;
    const Scores sc(a);
    const bool free_key = !a.causal || (a.prefix && j < a.prefix[b]);
    const int doc = a.docs && j < a.Skv ? a.docs[(int64_t)b * a.Skv + j] : -1;
    TaBounds kb{};
    if (a.docs) kb = a.bounds[(int64_t)b * a.ktiles + n];
    const int free_below = a.causal && a.prefix ? a.prefix[b] : a.causal ? 0 : 0x7fffffff;
    // a wait that gives up (dead is set) only spoils values
    for (int it = 0; it < total; it++) {
      const int q = q0 + it % nq, h = kh * a.group + it / nq;
      const int pos0 = q * TA_TILE + off;
      bool padded = false, masked = (n + 1) * TA_TILE > a.Skv || ((n + 1) * TA_TILE - 1 > pos0 && (n + 1) * TA_TILE > free_below);
      if (a.docs) {
        const TaBounds qb = a.qbounds[(int64_t)b * a.qtiles + q];
        padded = kb.neg || qb.neg;
        masked |= padded || kb.lo != kb.hi || qb.lo != qb.hi || kb.lo != qb.lo;
      }
      const float* rows = reinterpret_cast<const float*>(gen + L::ST + (it % NST) * L::STAGE + 2 * TILE) + part * 32;
      mbar_wait(&q_full[it % NST], (it / NST) & 1, abort);
      mbar_wait(&s_full, it & 1, abort);
      __syncwarp();
      fence_after();
      float v[32];
      ld_x32(ts, v);
      ld_wait();
      fence_before();
      mbar_arrive(&s_read);
      uint32_t see[1] = {0xffffffffu};
      if (masked) {
        if (!free_key) {
          first_bits<32>(see, j - pos0 - part * 32);   // the columns before it are hidden
          see[0] = ~see[0];
        }
        if (j >= a.Skv) see[0] = 0;
        if (a.docs) same_doc<32>(see, a.docs + (int64_t)b * a.Skv + pos0 + part * 32, a.Sq - q * TA_TILE - part * 32, doc);
      }
      if (sc.capped) {
        sc.cap.apply<32>(v, !padded);
      } else {
#pragma unroll
        for (int c = 0; c < 32; c += 2) f2::unpack(f2::mul(f2::pack(v[c], v[c + 1]), f2::splat(sc.f0)), v[c], v[c + 1]);
      }
      float p[32];
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const ulonglong2 shift = *reinterpret_cast<const ulonglong2*>(rows + c);   // -lse of four queries
        f2::unpack(f2::add(f2::pack(v[c], v[c + 1]), shift.x), p[c], p[c + 1]);
        f2::unpack(f2::add(f2::pack(v[c + 2], v[c + 3]), shift.y), p[c + 2], p[c + 3]);
      }
      if (a.slopes) {
        const float slope = a.slopes[h] * LOG2E, d0 = (float)(pos0 + part * 32 - j);
#pragma unroll
        for (int c = 0; c < 32; c++) p[c] = __fmaf_rn(-slope, fabsf(d0 + (float)c), p[c]);
      }
#pragma unroll
      for (int c = 0; c < 32; c++) p[c] = ex2(p[c]);
      if (sc.capped) {
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const u64 y = f2::pack(v[c], v[c + 1]);
          f2::unpack(f2::mul(f2::pack(p[c], p[c + 1]), f2::fma(f2::mul(y, y), f2::splat(sc.inv2), f2::splat(1.f))), v[c], v[c + 1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 32; c++) v[c] = p[c];
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < 32; c++)
          if (!(see[0] & (1u << c))) p[c] = v[c] = 0.f;
      }
      if (it > 0) mbar_wait(&p_read, (it - 1) & 1, abort);
      put_weights<BF>(base + L::P, r, part, p);
      if (padded) {   // padding may hold NaN, and 0 NaN is NaN: its query and gradient rows become zeros
        const int i = q * TA_TILE + r;
        mbar_wait(&g_full[it % NST], (it / NST) & 1, abort);   // the scores only needed the query tile
        if (part < 2 && i < a.Sq && a.docs[(int64_t)b * a.Skv + i + off] < 0)
          zero_row<DP>(base + L::ST + (it % NST) * L::STAGE + part * TILE, r);
        __syncwarp();
      }
      fence_async_smem();
      mbar_arrive(&p_full);
      mbar_wait(&dp_full, it & 1, abort);
      __syncwarp();
      fence_after();
      float w[32];
      ld_x32(tp, w);
      ld_wait();
      if (padded) {
#pragma unroll
        for (int c = 0; c < 32; c++) w[c] = v[c] == 0.f ? 0.f : w[c];
      }
      {
        uint32_t d[16];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const ulonglong2 less = *reinterpret_cast<const ulonglong2*>(rows + 128 + c);   // -delta of four queries
          float x, y;
          f2::unpack(f2::mul(f2::pack(v[c], v[c + 1]), f2::add(f2::pack(w[c], w[c + 1]), less.x)), x, y);
          d[c >> 1] = pack16<BF>(x, y);
          f2::unpack(f2::mul(f2::pack(v[c + 2], v[c + 3]), f2::add(f2::pack(w[c + 2], w[c + 3]), less.y)), x, y);
          d[(c >> 1) + 1] = pack16<BF>(x, y);
        }
        st_x16(tp, d);
      }
      st_wait();
      fence_before();
      mbar_arrive(&ds_full);
    }
    if (total > 0) {   // every product is done and no arrival is left when the CTA ends
      mbar_wait(&p_read, (total - 1) & 1, abort);
      mbar_wait(&done, 0, abort);
    }
    __syncwarp();
    fence_after();
    // dK over the keys' tile, dV over the values': both are no longer read
    const uint32_t kt = base + L::KEEP, vt = kt + TILE, acc = tmem + lanes + 256;
    constexpr int HALF = DP / 2;
    if (part < 2) row_out<BF, HALF>(vt, acc, acc, r, part * HALF, 1.f, 0.f, total > 0);
    else row_out<BF, HALF>(kt, acc + DP, acc + DP, r, (part - 2) * HALF, a.scale, 0.f, total > 0);
    fence_async_smem();
    bar_sync(5, 512);
    if (threadIdx.x == 0 && !dead) {
      for (int p = 0; p < DP / 64; p++)
        if (p * 64 < a.D) {
          tma_store(&a.dk, kt + p * PANEL, p * 64, 0, n * TA_TILE, kh, b);
          tma_store(&a.dv, vt + p * PANEL, p * 64, 0, n * TA_TILE, kh, b);
        }
      tma_store_commit();
      tma_store_wait();
    }
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;" ::: "memory");   // as the control group, for what follows
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x == 0 && dead && a.status) atomicOr(a.status, DA_STATUS_TIMEOUT);
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// ---- queries kept: dQ ----
template <int DP, bool BF>
__global__ void __launch_bounds__(TA_BWD_THREADS, 1) ta_dq_kernel(const __grid_constant__ TaArgs a) {
  using namespace tc5;
  using namespace ta;
  using L = TaBwdSmem<DP>;
  constexpr int NST = L::NST, TILE = L::TILE;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t q_full, k_full[NST], k_empty[NST], v_full[NST], v_empty[NST], s_full, s_read, dp_full, p_full, p_read, ds_full, done, gone;
  __shared__ uint32_t tmem_at;
  __shared__ int dead, range[2];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &dead;
  const int HB = a.B * a.Hq, hb = blockIdx.x % HB, b = hb / a.Hq, h = hb % a.Hq, kh = h / a.group;
  const int q = a.qtiles - 1 - blockIdx.x / HB, off = a.Skv - a.Sq, pos0 = q * TA_TILE + off;

  if (threadIdx.x == 0) {
    dead = 0;
    mbar_init(&q_full, 1);
    for (int s = 0; s < NST; s++) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&s_read, 512);
    mbar_init(&p_read, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&p_full, 512);
    mbar_init(&ds_full, 512);
    mbar_init(&done, 1);
    mbar_init(&gone, 1);
    mbar_fence_init();
  }
  if (warp == 17) tmem_alloc(&tmem_at, 512);
  if (warp == 16) {
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

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;" ::: "memory");
    if (warp == 16) {
      if (lane == 0 && total > 0) {
        mbar_expect_tx(&q_full, 3 * TILE);
        for (int p = 0; p < DP / 64; p++) {
          tma_load(base + L::KEEP + p * PANEL, &a.q, p * 64, 0, q * TA_TILE, h, b, &q_full);
          tma_load(base + L::KEEP + TILE + p * PANEL, &a.go, p * 64, 0, q * TA_TILE, h, b, &q_full);
          tma_load(base + L::P + p * PANEL, &a.o, p * 64, 0, q * TA_TILE, h, b, &q_full);
        }
        const auto fetch = [&](const CUtensorMap* map, int it, int at, uint64_t* full, uint64_t* empty) -> bool {
          const int s = it % NST;
          if (it >= NST && !mbar_wait(&empty[s], ((it / NST) - 1) & 1, abort)) return false;
          mbar_expect_tx(&full[s], TILE);
          for (int p = 0; p < DP / 64; p++)
            tma_load(base + L::ST + s * L::STAGE + at + p * PANEL, map, p * 64, 0, (n0 + it) * TA_TILE, kh, b, &full[s]);
          return true;
        };
        int nk = 0, nv = 0;
        if (fetch(&a.k, 0, 0, k_full, k_empty)) nk++;
        while (nv < total && fetch(&a.v, nv, TILE, v_full, v_empty)) {
          nv++;
          if (nk < total && !fetch(&a.k, nk, 0, k_full, k_empty)) break;
          if (nk < total) nk++;
        }
        for (int k = max(0, nk - NST); k < nk; k++) mbar_drain(&k_full[k % NST], (k / NST) & 1);
        for (int k = max(0, nv - NST); k < nv; k++) mbar_drain(&v_full[k % NST], (k / NST) & 1);
        mbar_drain(&q_full, 0);
      }
    } else if (warp == 17) {
      const int steps = same(total);
      if (steps > 0) {
        const uint32_t tm = same(tmem);
        const Products<DP, BF> go{tm, tm + 128, tm + 256 + DP, tm + 256, elect(), idesc<BF>(128, 128, false), idesc<BF>(128, DP, true)};
        const uint32_t qtile = base + L::KEEP, gtile = qtile + TILE, st0 = base + L::ST;
        bool ok = all_of(mbar_wait(&q_full, 0, abort) && mbar_wait(&k_full[0], 0, abort));
        if (ok) {
          fence_after();
          go.first(go.ts, qtile, st0, &s_full);
          ok = all_of(mbar_wait(&v_full[0], 0, abort));
          if (ok) {
            go.first(go.tp, gtile, st0 + TILE, &dp_full);
            if (NST < steps) commit_one(&v_empty[0], go.one);   // only where the copies wait for it, as below
          }
        }
        for (int it = 0; it < steps && ok; it++) {
          const uint32_t st = st0 + (it % NST) * L::STAGE, next = st0 + ((it + 1) % NST) * L::STAGE;
          if (it + 1 < steps) {
            ok = all_of(mbar_wait(&s_read, it & 1, abort) && mbar_wait(&k_full[(it + 1) % NST], ((it + 1) / NST) & 1, abort));
            if (!ok) break;
            fence_after();
            go.first(go.ts, qtile, next, &s_full);
          }
          ok = all_of(mbar_wait(&p_full, it & 1, abort));
          if (!ok) break;
          fence_after();
          go.weights(base + L::P, st, it > 0, &p_read);
          ok = all_of(mbar_wait(&ds_full, it & 1, abort));
          if (!ok) break;
          fence_after();
          go.grads(st, it > 0);
          if (it + NST < steps) commit_one(&k_empty[it % NST], go.one);
          if (it + 1 < steps) {
            ok = all_of(mbar_wait(&v_full[(it + 1) % NST], ((it + 1) / NST) & 1, abort));
            if (!ok) break;
            go.first(go.tp, gtile, next + TILE, &dp_full);
            if (it + 1 + NST < steps) commit_one(&v_empty[(it + 1) % NST], go.one);
          }
        }
        commit_one(&done, go.one);
        if (!ok) {
          commit_one(&gone, go.one);
          mbar_drain(&gone, 0);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;" ::: "memory");
    const int r = threadIdx.x & 127, part = threadIdx.x >> 7, qi = q * TA_TILE + r, pos = pos0 + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + lanes + part * 32, tp = ts + 128;
    const Scores sc(a);
    const float slope = a.slopes ? a.slopes[h] * LOG2E : 0.f;
    float* const my_row = a.rows + (((int64_t)b * a.Hq + h) * a.qtiles + q) * 256 + r;
    float* const sums = reinterpret_cast<float*>(raw + (base - smem_addr(raw)) + L::P);   // the weights' tile, when it is free
    // -lse and, from the rounded output, -delta: a quarter of the row's dimensions a thread.  The output's tile was copied
    // to the weights'; its words are read, then the quarters' sums take its place.
    float shift = -INFINITY, less;
    {
      using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
      if (qi < a.Sq) {
        const float l = a.lse[((int64_t)b * a.Hq + h) * a.Sq + qi];
        if (l != -INFINITY) shift = -l * LOG2E;
      }
      float s = 0.f;
      if (total > 0) {
        mbar_wait(&q_full, 0, abort);
        const unsigned char* const o = raw + (base - smem_addr(raw)) + L::P;
        const unsigned char* const g = raw + (base - smem_addr(raw)) + L::KEEP + TILE;
#pragma unroll
        for (int k = 0; k < DP / 32; k++) {
          const int u = part * (DP / 32) + k, at = (u >> 3) * PANEL + r * 128 + (((u & 7) ^ (r & 7)) << 4);
          Run<T, 8> x, y;
          x.load((const T*)(o + at));
          y.load((const T*)(g + at));
#pragma unroll
          for (int e = 0; e < 8; e++) s = __fmaf_rn(x.get(e), y.get(e), s);
        }
      }
      __syncwarp();
      bar_sync(5, 512);
      sums[part * 128 + r] = s;
      bar_sync(5, 512);
      less = shift == -INFINITY ? 0.f : -((sums[r] + sums[128 + r]) + (sums[256 + r] + sums[384 + r]));
      bar_sync(5, 512);
    }
    const int doc = a.docs && qi < a.Sq ? a.docs[(int64_t)b * a.Skv + pos] : -1;
    TaBounds qb{};
    if (a.docs) qb = a.qbounds[(int64_t)b * a.qtiles + q];
    int lim = a.Skv, full = a.Skv;
    if (a.causal) {
      const int pre = a.prefix ? a.prefix[b] : 0;
      lim = min(lim, max(pos + 1, pre));
      full = min(full, max(pos0 + 1, pre));
    }
    u64 delta[2] = {0, 0};
    for (int it = 0; it < total; it++) {   // a wait that gives up only spoils values, as above
      const int n = n0 + it, j0 = n * TA_TILE + part * 32;
      bool padded = false, masked = (n + 1) * TA_TILE > full;
      if (a.docs) {
        const TaBounds kb = a.bounds[(int64_t)b * a.ktiles + n];
        padded = kb.neg || qb.neg;
        masked |= padded || kb.lo != kb.hi || qb.lo != qb.hi || kb.lo != qb.lo;
      }
      mbar_wait(&s_full, it & 1, abort);
      __syncwarp();
      fence_after();
      float v[32];
      ld_x32(ts, v);
      ld_wait();
      fence_before();
      mbar_arrive(&s_read);
      uint32_t see[1] = {0xffffffffu};
      if (masked) {
        first_bits<32>(see, lim - j0);
        if (a.docs) same_doc<32>(see, a.docs + (int64_t)b * a.Skv + j0, a.Skv - j0, doc);
      }
      float p[32];
      const u64 sh = f2::splat(shift);
      if (sc.capped) {
        sc.cap.apply<32>(v, !padded);
#pragma unroll
        for (int c = 0; c < 32; c += 2) f2::unpack(f2::add(f2::pack(v[c], v[c + 1]), sh), p[c], p[c + 1]);
      } else {
#pragma unroll
        for (int c = 0; c < 32; c += 2) f2::unpack(f2::fma(f2::pack(v[c], v[c + 1]), f2::splat(sc.f0), sh), p[c], p[c + 1]);
      }
      if (a.slopes) {
        const float d0 = (float)(pos - j0);
#pragma unroll
        for (int c = 0; c < 32; c++) p[c] = __fmaf_rn(-slope, fabsf(d0 - (float)c), p[c]);
      }
#pragma unroll
      for (int c = 0; c < 32; c++) p[c] = ex2(p[c]);
      if (sc.capped) {
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const u64 y = f2::pack(v[c], v[c + 1]);
          f2::unpack(f2::mul(f2::pack(p[c], p[c + 1]), f2::fma(f2::mul(y, y), f2::splat(sc.inv2), f2::splat(1.f))), v[c], v[c + 1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 32; c++) v[c] = p[c];
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < 32; c++)
          if (!(see[0] & (1u << c))) p[c] = v[c] = 0.f;
      }
      if (it > 0) mbar_wait(&p_read, (it - 1) & 1, abort);
      put_weights<BF>(base + L::P, r, part, v);
      if (padded) {   // padding may hold NaN: its key rows become zeros before a product sums over them
        const int j = n * TA_TILE + r;
        if (part == 0 && j < a.Skv && a.docs[(int64_t)b * a.Skv + j] < 0) zero_row<DP>(base + L::ST + (it % NST) * L::STAGE, r);
        __syncwarp();
      }
      fence_async_smem();
      mbar_arrive(&p_full);
      mbar_wait(&dp_full, it & 1, abort);
      __syncwarp();
      fence_after();
      uint32_t d[16];
#pragma unroll
      for (int g = 0; g < 2; g++) {      // 16 at a time: weights and factors are live
        float w[16];
        ld_x16(tp + 16 * g, w);
        ld_wait();
        if (padded) {
#pragma unroll
          for (int c = 0; c < 16; c++) w[c] = p[16 * g + c] == 0.f ? 0.f : w[c];
        }
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const int k = 16 * g + c;
          const u64 x = f2::pack(w[c], w[c + 1]);
          delta[(c >> 1) & 1] = f2::fma(f2::pack(p[k], p[k + 1]), x, delta[(c >> 1) & 1]);
          float y, z;
          f2::unpack(f2::mul(f2::pack(v[k], v[k + 1]), f2::add(x, f2::splat(less))), y, z);
          d[k >> 1] = pack16<BF>(y, z);
        }
      }
      st_x16(tp, d);
      st_wait();
      fence_before();
      mbar_arrive(&ds_full);
    }
    if (total > 0) {   // every product is done and no arrival is left when the CTA ends
      mbar_wait(&p_read, (total - 1) & 1, abort);
      mbar_wait(&done, 0, abort);
    }
    __syncwarp();
    fence_after();
    // The sums were taken with delta from the rounded output; with D = sum p dp the gradient is
    // scale (sum ds k - (D - delta) sum p (1 - tanh^2) k).  D goes to the other kernel too.
    {
      float x, y;
      f2::unpack(f2::add(delta[0], delta[1]), x, y);
      sums[part * 128 + r] = x + y;
    }
    bar_sync(5, 512);
    const float exact = (sums[r] + sums[128 + r]) + (sums[256 + r] + sums[384 + r]);
    if (part == 0 && !dead) {
      my_row[0] = shift;
      my_row[128] = -exact;
    }
    __syncwarp();
    const uint32_t qt = base + L::KEEP, acc = tmem + lanes + 256;
    if (DP == 128) row_out<BF, 32>(qt, acc, acc + DP, r, part * 32, a.scale, -less - exact, total > 0);
    else if (part < 2) row_out<BF, 32>(qt, acc, acc + DP, r, part * 32, a.scale, -less - exact, total > 0);
    fence_async_smem();
    bar_sync(5, 512);
    if (threadIdx.x == 0 && !dead) {
      for (int p = 0; p < DP / 64; p++)
        if (p * 64 < a.D) tma_store(&a.dq, qt + p * PANEL, p * 64, 0, q * TA_TILE, h, b);
      tma_store_commit();
      tma_store_wait();
    }
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x == 0 && dead && a.status) atomicOr(a.status, DA_STATUS_TIMEOUT);
  if (warp == 17) tmem_dealloc(tmem, 512);
}

template <int DP, bool BF>
cudaError_t ta_dkv(const TaArgs& a, cudaStream_t st) {
  using L = TaBwdSmem<DP>;
  static TileSmem smem;
  int bytes;
  if (const cudaError_t e = smem.ready(ta_dkv_kernel<DP, BF>, L::END, &bytes)) return e;
  ta_dkv_kernel<DP, BF><<<(unsigned)(a.B * a.Hkv) * a.ktiles, TA_BWD_THREADS, bytes, st>>>(a);
  return cudaGetLastError();
}

template <int DP, bool BF>
cudaError_t ta_dq(const TaArgs& a, cudaStream_t st) {
  using L = TaBwdSmem<DP>;
  static TileSmem smem;
  int bytes;
  if (const cudaError_t e = smem.ready(ta_dq_kernel<DP, BF>, L::END, &bytes)) return e;
  if (a.qtiles == 0) return cudaSuccess;
  ta_dq_kernel<DP, BF><<<(unsigned)(a.B * a.Hq) * a.qtiles, TA_BWD_THREADS, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace detattn
