// Tiles of 128 rows x 64 or 128 16-bit columns in shared memory for the training attention:
// tensor-map copies, tcgen05.mma with the A operand in shared memory or in TMEM, and wide
// TMEM loads and stores.
//
// A tile is one or two panels of 128 rows x 64 columns.  A panel row is 128 bytes, its 16-byte units
// exchanged by the 128-byte swizzle (unit u of row r lies at u ^ (r % 8)), which is what a tensor
// map with that swizzle writes.  The same tile serves as an operand contracted over its
// columns (K-major) and as one contracted over its rows (MN-major): no operand is ever
// transposed or copied.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tc5.cuh"

namespace detattn {
namespace tc5 {

constexpr int PANEL = 128 * 128;   // bytes

// The descriptor's high word: groups of 8 rows are 1024 bytes apart, descriptor version, 128-byte swizzle.  Its low word is
// the address in 16-byte units (under 2^14) and the leading offset, so a step is one 32-bit addition.
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return ((uint64_t)DESC_HI << 32) | lo; }

// columns [16 s, 16 s + 16) of a tile, contracted over the columns
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int s) {
  return desc_of((tile >> 4) + (uint32_t)(((s >> 2) * PANEL + (s & 3) * 32) / 16 + (1 << 16)));
}
// rows [16 s, 16 s + 16), contracted over the rows: panels PANEL apart
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int s) {
  return desc_of((tile >> 4) + (uint32_t)(s * 2048 / 16 + ((PANEL >> 4) << 16)));
}

template <bool BF>
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool b_mn) {
  return BF ? idesc_bf16(m, n, b_mn) : idesc_f16(m, n, b_mn);
}

// Products and commits are issued by whole warps with one elected lane.  A tcgen05.mma takes its descriptors from uniform
// registers: in code that only one lane runs the compiler has to move every one of them there (measured 79 to
// 160 cycles a product of 128 x 128 x 16); in code that the warp runs together, on values it can tell are the same in
// all lanes, they are computed there (64 cycles, the tensor cores' rate).  same() makes a value such a one.
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ int same(int x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ uint32_t same(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ bool all_of(bool x) { return __all_sync(0xffffffffu, x); }

// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                       uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one));
}
// D[tmem] (+)= A[tmem] * B[smem], A 16-bit elements, two in a 32-bit column
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one));
}
__device__ __forceinline__ void commit_one(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(one)
      : "memory");
}

// box of a rank-5 tensor map -> shared memory; completion counted on bar
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3, int c4) {
  asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];" ::"l"(map),
               "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
               : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Whether the phase of that parity is complete; never suspends the thread.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait for a copy or commit of this thread whatever became of the rest of the CTA: a CTA that gives up
// still ends with nothing in flight.  Bounded (20 ms) like every wait.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try(bar, parity) && globaltimer() - t0 < 20000000ull) __nanosleep(100);
}

// 32 consecutive 32-bit columns of this thread's TMEM lane
__device__ __forceinline__ void ld_x32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int e = 0; e < 32; e++) v[e] = __uint_as_float(r[e]);
}
__device__ __forceinline__ void ld_x16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
#pragma unroll
  for (int e = 0; e < 16; e++) v[e] = __uint_as_float(r[e]);
}
__device__ __forceinline__ void st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {   // two 16-bit floats, rounded to nearest even
  uint32_t d;
  if constexpr (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <bool BF>
__device__ __forceinline__ unsigned long long unpack16(uint32_t w) {   // the packed binary32 pair of two 16-bit floats
  float2 f;
  if constexpr (BF) f = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  unsigned long long d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(f.x), "f"(f.y));
  return d;
}
__device__ __forceinline__ float ex2(float x) {   // 2^x, 2^-inf = 0; error 2^-22 relative
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// zeros over row r of a tile (any thread; the reader is a product that waits for this thread)
template <int DP>
__device__ __forceinline__ void zero_row(uint32_t tile, int r) {
#pragma unroll
  for (int p = 0; p < DP / 64; p++)
#pragma unroll
    for (int u = 0; u < 8; u++)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + p * PANEL + r * 128 + u * 16), "r"(0) : "memory");
  fence_async_smem();
}

}  // namespace tc5
}  // namespace detattn
