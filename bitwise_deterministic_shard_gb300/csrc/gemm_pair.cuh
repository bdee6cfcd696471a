// Matrix products on pairs of SMs (tcgen05, cta_group::2) for the gated feed-forward operator:
// tiles of 256 x 256 (or 256 x 128) of the result, one pair a tile at a time, fed by tensor-map copies.
//
// A cluster of two CTAs works on one tile: each CTA holds 128 of the rows of A and half of the rows of B for a step of 64 of
// the contracted dimension, the leader's products read both CTAs' shared memory and write 128 rows of binary32 sums into each
// CTA's TMEM.  Per SM and step of a 256 x 256 tile that is 32 KB of copies for 512 cycles of the tensor cores: a single SM with a
// tile of its own of 128 x 256 would need 48 KB, more than its share of the L2's rate.  The narrow tile is for results of so few
// tiles that the last round of wide ones would leave many pairs idle.
//
// One warp copies (a ring of steps), one of the leader issues the products, eight warps take the finished sums from TMEM.
// Two tiles of sums fit, so a tile's results are taken while the next one's products run.  The grid is as
// many pairs as the GPU holds; which tiles a pair takes is a function of the sizes.  All sums of a result are one chain of
// products in the order of the contracted dimension: no split, no atomics.
//
// Operands lie in shared memory as the 128-byte swizzle writes them: contracted over the contiguous dimension (K-major: rows of
// 64 elements) or over the rows (MN-major: panels of 64 rows of 64 elements), so no operand is ever transposed.  All copies are boxes
// of 64 x 64 elements: 8 KB, a panel, or 64 rows of a K-major operand.
#pragma once
#include "device_once.h"
#include "tc5_tile.cuh"

namespace detattn {
namespace pair {

constexpr int BK = 64;                    // contracted elements of a step
constexpr int BOX = 64 * BK * 2;          // bytes of a copy
constexpr int TAKERS = 8;                 // warps that take results
constexpr int THREADS = (TAKERS + 2) * 32;

// TN: columns of a tile (rows of B); EXTRA: bytes of shared memory beside the ring
template <int TN, int EXTRA>
struct Ring {
  static constexpr int A = 2 * BOX, B = TN / 128 * BOX, STAGE = A + B;
  static constexpr int STAGES = (227 * 1024 - 1024 - 512 - EXTRA) / STAGE;
  static constexpr int SMEM = STAGES * STAGE + EXTRA + 1024;
};

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the leader's address of a place in this CTA's shared memory
__device__ __forceinline__ uint32_t at_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// A bounded wait.  Arrivals may come from the other CTA; what they stand for (copies, products, sums taken from TMEM) is not plain
// memory, so the wait takes no scope beyond the CTA.
// A whole warp calls it; the answer is the same in all lanes.
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (tc5::all_of(tc5::mbar_try(bar, parity))) return true;
  const uint64_t t0 = tc5::globaltimer();
  for (uint32_t it = 1; it < (1u << 30); it++) {
    if (tc5::all_of(tc5::mbar_try(bar, parity))) return true;
    if ((it & 15) == 0 && tc5::all_of(*abort || tc5::globaltimer() - t0 > tc5::WAIT_NS)) break;
  }
  *abort = 1;
  return false;
}

__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {   // one whole warp of each CTA of the pair
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc5::smem_addr(dst)), "r"(ncols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols));
}
// box of a rank-2 tensor map -> this CTA's shared memory, completion counted on a barrier of the leader; by the one lane of a warp
// that runs it together (tc5_tile.cuh: operands in uniform registers)
__device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t leader_bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(leader_bar), "r"(one)
      : "memory");
}
__device__ __forceinline__ void expect_one(uint64_t* bar, uint32_t bytes, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(tc5::smem_addr(bar)),
      "r"(bytes), "r"(one)
      : "memory");
}
// D[tmem of both] (+)= A[both CTAs' smem] * B[both CTAs' smem]; issued by one lane of the leader
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                    uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one));
}
// arrive on bar in both CTAs once every product issued so far has completed
__device__ __forceinline__ void commit_both(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b16 m;\n\tsetp.ne.u32 q, %1, 0;\n\tmov.b16 m, 3;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          tc5::smem_addr(bar)),
      "r"(one)
      : "memory");
}

// products of a type, 256 x TN x 16, either operand MN-major
template <bool BF, int TN>
__device__ __forceinline__ uint32_t idesc(bool a_mn, bool b_mn) {
  return (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
}
// low word of the descriptor of an operand's contracted elements [0, 16), and what 16 further on adds
__device__ __forceinline__ uint32_t desc_lo(uint32_t tile, bool mn) { return (tile >> 4) + (mn ? BOX >> 4 << 16 : 1 << 16); }
__device__ __forceinline__ uint32_t desc_step(bool mn) { return mn ? 2048 / 16 : 32 / 16; }

constexpr int MOST_STAGES = 10;
struct Shared {   // beside the ring
  uint64_t full[MOST_STAGES], empty[MOST_STAGES], done[2], taken[2];
  uint32_t tmem;
  int dead;
};

struct Tile {
  int kind, m, n, steps;   // steps 0: no more tiles
};
// tile t of mt x nt: runs of 8 tile rows, column after column, so that the pairs at work at one time read few rows of both
// operands
__device__ __forceinline__ Tile tile_of(int t, int mt, int nt, int kind, int steps) {
  const int g = t / (8 * nt), r = t - g * 8 * nt, rows = min(8, mt - 8 * g);
  return {kind, 8 * g + r % rows, r / rows, steps};
}

// The products of this pair's tiles.
//   tile(j): the pair's j-th Tile
//   load(tile, step, a, b, leader_bar, one): copies this CTA's halves of a step (2 and TN / 128 boxes) to the addresses a and b; a
//     whole warp calls it, `one` in the lane that is to issue them
//   take(tile, columns, extra, release): takes a tile's sums; columns: TMEM address of this warp's lanes; extra: address of the
//     shared memory beside the ring; calls release() when it has read them
// a_mn(kind): whether A is MN-major; B is with B_MN.
template <bool BF, int TN, int EXTRA, bool B_MN, typename Next, typename Major, typename Load, typename Take>
__device__ __forceinline__ void run(Shared& sh, unsigned char* raw, int32_t* status, Next tile, Major a_mn, Load load, Take take) {
  using namespace tc5;
  using R = Ring<TN, EXTRA>;
  constexpr int STAGES = R::STAGES;
  static_assert(STAGES <= MOST_STAGES, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  volatile int* abort = &sh.dead;

  if (threadIdx.x == 0) {
    sh.dead = 0;
    for (int s = 0; s < STAGES; s++) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&sh.done[i], 1);
      mbar_init(&sh.taken[i], 2 * TAKERS);
    }
    mbar_fence_init();
  }
  if (warp == TAKERS + 1) tmem_alloc(&sh.tmem, 512);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = sh.tmem;
  after_previous();

  if (warp == TAKERS) {
    const uint32_t one = elect(), first = one && rank == 0, ring = same(base), bars = same(at_leader(smem_addr(&sh.full[0])));
    int s = 0, used = 0;       // the stage and how many are in use; round: the fills of the present stage before
    uint32_t round = 0;
    bool ok = true;
    for (int j = 0; ok; j++) {
      const Tile t = tile(j);
      const int steps = same(t.steps);
      if (steps == 0) break;
      for (int n = 0; n < steps; n++) {
        if (round > 0 && !(ok = wait_pair(&sh.empty[s], (round - 1) & 1, abort))) break;
        const uint32_t at = ring + s * R::STAGE;
        expect_one(&sh.full[s], 2 * R::STAGE, first);
        load(t, n, at, at + R::A, bars + s * 8, one);
        if (++s == STAGES) {
          s = 0;
          round++;
        }
        used = round > 0 ? STAGES : s;
      }
    }
    // every step's products are done, so nothing is in flight when the CTA ends; given up: what was copied arrives at the leader
    for (int j = 0; j < used; j++) {
      const uint32_t last = (round - (j >= s)) & 1;   // of the stage's last fill
      if (ok) ok = wait_pair(&sh.empty[j], last, abort);
      if (!ok && rank == 0) mbar_drain(&sh.full[j], last);
    }
  } else if (warp == TAKERS + 1) {
    if (rank == 0) {
      const uint32_t one = elect(), tm = same(tmem), ring = same(base);
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; i++) {
        const Tile t = tile(i);
        const int steps = same(t.steps);
        if (steps == 0) break;
        const bool mn = a_mn(same(t.kind));
        const uint32_t id = idesc<BF, TN>(mn, B_MN), sa = desc_step(mn), sb = desc_step(B_MN), d = tm + (i & 1) * TN;
        if (i >= 2 && !(ok = wait_pair(&sh.taken[i & 1], ((i >> 1) - 1) & 1, abort))) break;
        fence_after();
        for (int n = 0; n < steps; n++) {
          if (!(ok = wait_pair(&sh.full[s], phase, abort))) break;
          fence_after();
          const uint32_t at = ring + s * R::STAGE, da = desc_lo(at, mn), db = desc_lo(at + R::A, B_MN);
#pragma unroll
          for (int j = 0; j < BK / 16; j++) mma(d, desc_of(da + j * sa), desc_of(db + j * sb), id, n > 0 || j > 0, one);
          commit_both(&sh.empty[s], one);
          if (++s == STAGES) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok) commit_both(&sh.done[i & 1], one);
      }
    }
  } else {
    for (int i = 0;; i++) {
      const Tile t = tile(i);
      if (t.steps == 0 || !wait_pair(&sh.done[i & 1], (i >> 1) & 1, abort)) break;
      fence_after();
      const uint32_t bar = at_leader(smem_addr(&sh.taken[i & 1]));
      take(t, tmem + ((uint32_t)(warp & 3) << 21) + (i & 1) * TN, base + STAGES * R::STAGE, [&] {
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(bar);
      });
    }
  }
  __syncwarp();
  fence_before();
  cluster_sync();   // the leader's products have read the other CTA's shared memory, all sums are taken
  fence_after();
  if (warp == TAKERS + 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && sh.dead && status) atomicOr(status, DA_STATUS_TIMEOUT);
}

}  // namespace pair
}  // namespace detattn
