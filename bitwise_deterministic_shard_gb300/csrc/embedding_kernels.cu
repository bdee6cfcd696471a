// Embedding lookup with scaling and its gradient by sorted tokens.
//
//   y[i] = scale w[id_i];   dw[v] = scale (sum over i with id_i = v, in order of i, of dy[i])
//
// What bounds both: HBM.  The lookup reads the named rows and writes one a token; the gradient reads dy once and writes every
// row of dw, most of them zeros for a large vocabulary.
//
// Gradient: the tokens are sorted by id, stably, by counting digits of up to 9 bits from the lowest on (two passes below 2^18
// rows).  Up to 4096 tokens one CTA does that in shared memory; longer ones take two launches a pass (three past 32768), each of
// which starts as the one before it ends.  dw's zeros wait for nothing and are written beside all of these.  A token's place among those of its digit comes
// from ballots over the warp and the warp's counters, so the order never depends on which thread came first.  Then a chunk of up to 32 tokens of a row is one
// chain of binary32 additions for each column, in order of the tokens; rows of more leave their chunks' sums in the
// workspace, and a last kernel adds these, eight runs of chunks in order and then the eight.  So a row's bits depend on its own
// tokens alone, and no atomics add values (the lists of chunks are filled by atomics: their order is that of the work, not
// of a sum).
//
// A warp takes a short chunk's 1024 16-bit columns at once (its loads are independent), a long one's 256 with eight tokens'
// loads under way: with one column width for all, 16384 tokens of width 2048 took 64 us instead of 22.  16384 tokens, 128256 rows of
// 2048 bf16: lookup 12 us, gradient 109, of which 78 are the zeros (6.7 TB/s); 3001 tokens, 20011 rows of 1003 f32: 5 and 24.
#include <algorithm>

#include "../../include/detattn.h"
#include "decoder_kernels.h"
#include "device_once.h"
#include "train_math.cuh"

namespace detattn {
namespace {

__device__ __forceinline__ int64_t id_at(const EmArgs& a, int64_t i) {
  return a.wide ? static_cast<const int64_t*>(a.ids)[i] : (int64_t) static_cast<const int32_t*>(a.ids)[i];
}

// ---- lookup: a warp LOOKUP_RUNS runs (of 16 bytes or one element a lane) of a token ----
constexpr int LOOKUP_RUNS = 4;
template <typename T, bool AL>
__global__ void __launch_bounds__(256) em_lookup_kernel(const __grid_constant__ EmArgs a, uint32_t pieces) {
  constexpr int VEC = AL ? Elem<T>::VEC : 1, U = LOOKUP_RUNS;
  const int lane = threadIdx.x & 31;
  const uint64_t w = ((uint64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int64_t i = w / pieces, c0 = (int64_t)(w % pieces) * 32 * VEC * U;
  if (i >= a.n) return;
  const int64_t id = id_at(a, i);
  const bool known = id >= 0 && id < a.rows;
  if (!known && lane == 0 && c0 == 0 && a.status) atomicOr(a.status, DA_STATUS_BAD_TARGET);
  const T* const from = static_cast<const T*>(a.w) + (known ? id : 0) * a.ws;
  T* const to = static_cast<T*>(a.y) + i * a.ys;
  if constexpr (AL) {
    Run<T, VEC> r[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t c = c0 + (u * 32 + lane) * VEC;
      r[u].zero();
      if (known && c < a.cols) r[u].load(from + c);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t c = c0 + (u * 32 + lane) * VEC;
      if (a.scale != 1.f) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e++) v[e] = r[u].get(e) * a.scale;
        r[u].set(v);
      }
      if (c < a.cols) r[u].store(to + c);
    }
  } else {
    T r[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t c = c0 + u * 32 + lane;
      r[u] = known && c < a.cols ? from[c] : Elem<T>::put(0.f);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t c = c0 + u * 32 + lane;
      if (c < a.cols) to[c] = a.scale == 1.f ? r[u] : Elem<T>::put(Elem<T>::get(r[u]) * a.scale);
    }
  }
}

// ---- sort ----
__device__ __forceinline__ uint32_t key_at(const EmArgs& a, int64_t i) {   // rows: gives no gradient
  const int64_t id = id_at(a, i);
  if (id < 0 || id >= a.rows) {
    if (a.status) atomicOr(a.status, DA_STATUS_BAD_TARGET);
    return (uint32_t)a.rows;
  }
  return id == a.padding ? (uint32_t)a.rows : (uint32_t)id;
}
// Zeros over a contiguous dw, which wait for nothing: they run beside the sort.  Part `part` of `parts` of it, by CTAs of a launch.
struct Fill {
  uint32_t part, parts;
};
__device__ __forceinline__ void fill_zeros(const EmArgs& a, uint32_t cta, uint32_t ctas, Fill f) {
  const int64_t bytes = a.rows * a.cols * (a.dtype == DA_F32 ? 4 : 2);
  unsigned char* const p = static_cast<unsigned char*>(a.dw);
  const int64_t head = min(bytes, (int64_t)(-reinterpret_cast<intptr_t>(p) & 15)), body = (bytes - head) / 16;
  const int64_t end = body / f.parts * (f.part + 1) + (f.part + 1 == f.parts ? body % f.parts : 0);
  for (int64_t i = body / f.parts * f.part + (int64_t)cta * blockDim.x + threadIdx.x; i < end; i += (int64_t)ctas * blockDim.x)
    reinterpret_cast<uint4*>(p + head)[i] = make_uint4(0, 0, 0, 0);
  if (f.part == 0 && cta == 0 && threadIdx.x < 32) {
    if (threadIdx.x < head) p[threadIdx.x] = 0;
    const int64_t tail = head + body * 16 + threadIdx.x;
    if (tail < bytes) p[tail] = 0;
  }
}
// Beside the kernel before it, which it does not depend on; it ends after that one, so what follows may take both as done.
__global__ void __launch_bounds__(256) em_fill_kernel(const __grid_constant__ EmArgs a) {
  next_may_start();
  fill_zeros(a, blockIdx.x, gridDim.x, Fill{0, 1});
  after_previous();
}

// Places of a warp's tokens among those of the same digit, in their order: what the counters held and, of this step's, how many lower
// lanes have it.  A lane without a token has a digit of its own, EM_BINS.  By ballots over the digit's bits.
__device__ __forceinline__ uint32_t count_digit(uint32_t digit, int bits, uint32_t* hist) {
  const uint32_t lane = threadIdx.x & 31;
  const bool live = digit < EM_BINS;
  uint32_t same = __ballot_sync(0xffffffffu, live);
  for (int b = 0; b < bits; b++) {
    const bool bit = digit >> b & 1;
    const uint32_t who = __ballot_sync(0xffffffffu, bit);
    same &= bit ? who : ~who;
  }
  const uint32_t before = live ? hist[digit] : 0, rank = __popc(same & ((1u << lane) - 1));
  __syncwarp();
  if (live && same >> lane == 1) hist[digit] = before + rank + 1;   // the last of them
  __syncwarp();
  return before + rank;
}

// One CTA sorts up to EM_SMALL tokens.
constexpr int SORT_THREADS = 1024, SORT_WARPS = 32, SORT_RUN = EM_SMALL / SORT_WARPS;
struct SortSmall {
  uint32_t key[EM_SMALL];
  uint16_t pos[2][EM_SMALL];
  uint32_t hist[SORT_WARPS][EM_BINS];   // in the end the sorted keys lie here
  uint32_t base[EM_BINS], warps[32];
  EmUnits found;
};
static_assert(SORT_WARPS * EM_BINS >= EM_SMALL, "room for the sorted keys");

// What starts at place i of the sorted keys: a chunk of a row's tokens, or nothing.  Called by whole warps; the counters are atomics.
__device__ __forceinline__ void find_chunk(const EmArgs& a, const uint32_t* key, int64_t i, int64_t n, EmUnits* found) {
  uint32_t k = (uint32_t)a.rows, len = 0;
  bool more = false, start = false;
  int64_t end = i;
  if (i < n) k = key[i];
  if (k < a.rows) {
    int64_t first = i;
    bool is = true;
    if (i > 0 && key[i - 1] == k) {
      is = i >= EM_CHUNK && key[i - EM_CHUNK] == k;   // else within the first chunk
      if (is) {                                       // the first place of k
        int64_t lo = 0;
        while (lo < first) {
          const int64_t mid = (lo + first) >> 1;
          if (key[mid] < k) lo = mid + 1;
          else first = mid;
        }
        is = (i - first) % EM_CHUNK == 0;
      }
    }
    if (is) {
      start = i == first;
      int64_t lo = i + 1;
      end = min(n, i + EM_CHUNK);
      more = !start || (i + EM_CHUNK < n && key[i + EM_CHUNK] == k);
      while (lo < end) {   // the first place past k, at most a chunk on
        const int64_t mid = (lo + end) >> 1;
        if (key[mid] == k) lo = mid + 1;
        else end = mid;
      }
      len = (uint32_t)(end - i);
    }
  }
  const int lane = threadIdx.x & 31;
  const auto place = [&](bool mine, uint32_t* counter) {   // of this lane's entry
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    uint32_t at = 0;
    if (lane == 0 && who) at = atomicAdd(counter, __popc(who));
    return __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
  };
  const bool few = len > 0 && len <= EM_FEW && !more, many = len > 0 && !few;
  const uint32_t f = place(few, &found->few), m = place(many, &found->many), r = place(many && more && start, &found->rows);
  const uint4 unit = make_uint4((uint32_t)i, len | (more ? EM_MORE : 0), k, 0);
  if (few) a.unit[f] = unit;
  if (many) a.unit[n - 1 - m] = unit;
  if (many && more && start) {
    int64_t lo = i + EM_CHUNK, hi = n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (key[mid] == k) lo = mid + 1;
      else hi = mid;
    }
    a.row[r] = make_uint4((uint32_t)i, (uint32_t)hi, k, 0);
  }
}

__global__ void __launch_bounds__(SORT_THREADS, 1) em_sort_kernel(const __grid_constant__ EmArgs a, int passes, int bits) {
  next_may_start();
  extern __shared__ unsigned char raw[];
  SortSmall& s = *reinterpret_cast<SortSmall*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = (int)a.n;
  constexpr int K = SORT_RUN / 32;
  const int i0 = warp * SORT_RUN + lane, used = (n + SORT_RUN - 1) / SORT_RUN;   // a warp's run of places; warps that have one
  for (int i = tid; i < n; i += SORT_THREADS) s.key[i] = key_at(a, i);
  __syncthreads();
  for (int p = 0; p < passes; p++) {
    const int shift = p * bits;
    const uint32_t mask = (1u << bits) - 1;
    const uint16_t* const from = s.pos[(p + 1) & 1];
    uint16_t* const to = s.pos[p & 1];
    int token[K];
    uint32_t digit[K], place[K];
#pragma unroll
    for (int k = 0; k < K; k++) token[k] = i0 + 32 * k < n ? p ? from[i0 + 32 * k] : i0 + 32 * k : -1;
#pragma unroll
    for (int k = 0; k < K; k++) digit[k] = token[k] < 0 ? EM_BINS : s.key[token[k]] >> shift & mask;
    for (int b = lane; b <= (int)mask; b += 32) s.hist[warp][b] = 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < K; k++) place[k] = count_digit(digit[k], bits, s.hist[warp]);
    __syncthreads();
    // places before each digit, and within it before each warp
    uint32_t total = 0;
    if (tid <= (int)mask)
#pragma unroll 8
      for (int w = 0; w < used; w++) {
        const uint32_t c = s.hist[w][tid];
        s.hist[w][tid] = total;
        total += c;
      }
    uint32_t sum = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) s.warps[warp] = sum;
    __syncthreads();
    if (tid <= (int)mask) {
      uint32_t before = sum - total;
      for (int w = 0; w < warp; w++) before += s.warps[w];
      s.base[tid] = before;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; k++)
      if (token[k] >= 0) to[s.base[digit[k]] + s.hist[warp][digit[k]] + place[k]] = (uint16_t)token[k];
    __syncthreads();
  }
  const uint16_t* const done = s.pos[(passes - 1) & 1];
  uint32_t* const sorted = &s.hist[0][0];
  if (tid == 0) s.found = {0, 0, 0};
  for (int i = tid; i < n; i += SORT_THREADS) {
    a.pos[0][i] = done[i];
    sorted[i] = s.key[done[i]];
  }
  __syncthreads();
  for (int i = warp * 32; i < n; i += SORT_THREADS) find_chunk(a, sorted, i + lane, n, &s.found);
  __syncthreads();
  if (tid == 0) *a.found = s.found;
}

// ---- a pass over longer ones; CTAs past a kernel's own fill their part of the zeros ----
constexpr int RADIX_THREADS = 256, RADIX_WARPS = 8;
// counts of a block's digits (the first pass: from the ids), as [blocks][EM_BINS] where the next kernel adds them up itself, else as
// [bins][blocks]
__global__ void __launch_bounds__(RADIX_THREADS) em_count_kernel(const __grid_constant__ EmArgs a, uint32_t blocks, int block, bool by_block, int from, int shift,
                                                                 int bits, Fill fill) {
  next_may_start();
  if (blockIdx.x >= blocks) {
    fill_zeros(a, blockIdx.x - blocks, gridDim.x - blocks, fill);
    return;
  }
  __shared__ uint32_t hist[EM_BINS];
  const uint32_t mask = (1u << bits) - 1;
  for (int b = threadIdx.x; b < EM_BINS; b += RADIX_THREADS) hist[b] = 0;
  __syncthreads();
  after_previous();
  if (from < 0 && blockIdx.x == 0 && threadIdx.x == 0) *a.found = {0, 0, 0};
  const int64_t i0 = (int64_t)blockIdx.x * block, i1 = min(a.n, i0 + block);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += RADIX_THREADS)
    atomicAdd(&hist[(from < 0 ? key_at(a, i) : a.key[from][i]) >> shift & mask], 1u);
  __syncthreads();
  if (by_block)
    for (int b = threadIdx.x; b < EM_BINS; b += RADIX_THREADS) a.count[(size_t)blockIdx.x * EM_BINS + b] = hist[b];
  else
    for (uint32_t b = threadIdx.x; b <= mask; b += RADIX_THREADS) a.count[(size_t)b * blocks + blockIdx.x] = hist[b];
}
// places before each (digit, block): one CTA, a run of counts a thread
__global__ void __launch_bounds__(1024) em_scan_kernel(const __grid_constant__ EmArgs a, int64_t n, Fill fill) {
  next_may_start();
  if (blockIdx.x > 0) {
    fill_zeros(a, blockIdx.x - 1, gridDim.x - 1, fill);
    return;
  }
  __shared__ uint32_t warps[32];
  after_previous();
  uint32_t* const count = a.count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t per = (n + 4095) / 4096, i0 = min(n / 4, tid * per), i1 = min(n / 4, i0 + per);   // n is a multiple of 4: so are the bins
  uint4* const four = reinterpret_cast<uint4*>(count);
  uint32_t total = 0;
#pragma unroll 4
  for (int64_t i = i0; i < i1; i++) {
    const uint4 c = four[i];
    total += c.x + c.y + c.z + c.w;
  }
  uint32_t sum = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) warps[warp] = sum;
  __syncthreads();
  uint32_t before = sum - total;
  for (int w = 0; w < warp; w++) before += warps[w];
#pragma unroll 4
  for (int64_t i = i0; i < i1; i++) {
    const uint4 c = four[i];
    four[i] = make_uint4(before, before + c.x, before + c.x + c.y, before + c.x + c.y + c.z);
    before += c.x + c.y + c.z + c.w;
  }
}
// K: steps of a warp, blocks of 256 K tokens.  ADD: this kernel adds up the blocks' counts (a thread two neighbouring digits), else
// em_scan_kernel has: a launch less, as long as there are few blocks to read (5000 tokens, 1000 rows of 64: 29 us instead of 35; 32768,
// 50000 rows of 512, 32 blocks of 1024: 47.6 and 48.4; but 65536, 30000 rows of 64, 32 blocks of 2048: 52 and 46).
static_assert(EM_BINS == 2 * RADIX_THREADS, "two digits a thread");
template <int K, bool ADD>
__global__ void __launch_bounds__(RADIX_THREADS) em_scatter_kernel(const __grid_constant__ EmArgs a, uint32_t blocks, int from, int to, int shift, int bits,
                                                                   Fill fill) {
  next_may_start();
  if (blockIdx.x >= blocks) {
    fill_zeros(a, blockIdx.x - blocks, gridDim.x - blocks, fill);
    return;
  }
  __shared__ uint32_t hist[RADIX_WARPS][EM_BINS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t mask = (1u << bits) - 1;
  const int64_t i0 = ((int64_t)blockIdx.x * RADIX_WARPS + warp) * 32 * K + lane;
  uint32_t key[K], pos[K], place[K];
  for (int b = lane; b < EM_BINS; b += 32) hist[warp][b] = 0;
  after_previous();
#pragma unroll
  for (int k = 0; k < K; k++) {
    const int64_t i = i0 + k * 32;
    key[k] = i < a.n ? from < 0 ? key_at(a, i) : a.key[from][i] : 0;
    pos[k] = i < a.n && from >= 0 ? a.pos[from][i] : (uint32_t)i;
  }
  __shared__ uint32_t base[ADD ? EM_BINS : 1], warps[RADIX_WARPS];
  if constexpr (ADD) {
    uint2 all = make_uint2(0, 0), earlier = make_uint2(0, 0);
    const uint2* const count = reinterpret_cast<const uint2*>(a.count) + tid;
#pragma unroll 8
    for (uint32_t b = 0; b < blocks; b++) {
      const uint2 c = count[(size_t)b * RADIX_THREADS];
      if (b == blockIdx.x) earlier = all;
      all.x += c.x;
      all.y += c.y;
    }
    uint32_t sum = all.x + all.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    uint32_t before = sum - all.x - all.y;
    for (int w = 0; w < warp; w++) before += warps[w];
    base[2 * tid] = before + earlier.x;
    base[2 * tid + 1] = before + all.x + earlier.y;
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < K; k++) place[k] = count_digit(i0 + k * 32 < a.n ? key[k] >> shift & mask : EM_BINS, bits, hist[warp]);
  __syncthreads();
  for (uint32_t b = tid; b <= mask; b += RADIX_THREADS) {
    uint32_t before = ADD ? base[ADD ? b : 0] : a.count[(size_t)b * blocks + blockIdx.x];
#pragma unroll
    for (int w = 0; w < RADIX_WARPS; w++) {
      const uint32_t c = hist[w][b];
      hist[w][b] = before;
      before += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; k++)
    if (i0 + k * 32 < a.n) {
      const uint32_t at = hist[warp][key[k] >> shift & mask] + place[k];
      a.key[to][at] = key[k];
      a.pos[to][at] = pos[k];
    }
}
__global__ void __launch_bounds__(256) em_chunk_kernel(const __grid_constant__ EmArgs a, uint32_t blocks, int from, Fill fill) {
  next_may_start();
  if (blockIdx.x >= blocks) {
    fill_zeros(a, blockIdx.x - blocks, gridDim.x - blocks, fill);
    return;
  }
  after_previous();
  find_chunk(a, a.key[from], (int64_t)blockIdx.x * 256 + threadIdx.x, a.n, a.found);
}
// Where a chunk of several leaves its sum: full ones start at least a chunk apart, and so do the last ones of their rows.
__device__ __forceinline__ int64_t slot_of(const EmArgs& a, int64_t i, uint32_t len) {
  return i / EM_CHUNK + (len < EM_CHUNK ? a.n / EM_CHUNK + 1 : 0);
}

// ---- sums ----
// AL: runs of 16 bytes a lane; else of 4 single elements, neighbouring lanes' beside each other.  C runs of a chunk, R tokens' loads
// under way.
template <typename T, bool AL, int C, int R>
__device__ __forceinline__ void sum_chunk(const EmArgs& a, uint4 unit, int64_t c0, int from) {
  constexpr int VEC = AL ? Elem<T>::VEC : 4, STRIDE = AL ? 1 : 32;
  const int lane = threadIdx.x & 31;
  const uint32_t len = unit.y & ~EM_MORE;
  const uint32_t* const pos = a.pos[from] + unit.x;
  uint32_t token[EM_CHUNK / 32];
#pragma unroll
  for (int i = 0; i < EM_CHUNK / 32; i++) token[i] = i * 32 + lane < len ? pos[i * 32 + lane] : 0;
  c0 += AL ? lane * VEC : lane;
  const T* const dy = static_cast<const T*>(a.dy) + c0;
  const auto inside = [&](int c, int e) { return c0 + c * 32 * VEC + (AL ? 0 : 32 * e) < a.cols; };
  float sum[C][VEC];
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int e = 0; e < VEC; e++) sum[c][e] = 0.f;
  for (uint32_t j = 0; j < len; j += R) {
    const T* at[R];
#pragma unroll
    for (int u = 0; u < R; u++) {
      const uint32_t t = j + u;
      at[u] = dy + (int64_t)__shfl_sync(0xffffffffu, EM_CHUNK == 32 || t < 32 ? token[0] : token[EM_CHUNK / 32 - 1], t & 31) * a.ys;
    }
    if constexpr (AL) {
      Run<T, VEC> r[R][C];
#pragma unroll
      for (int u = 0; u < R; u++)
#pragma unroll
        for (int c = 0; c < C; c++)
          if (j + u < len && inside(c, 0)) r[u][c].load(at[u] + c * 32 * VEC);
          else r[u][c].zero();
#pragma unroll
      for (int u = 0; u < R; u++)
        if (j + u < len) {
#pragma unroll
          for (int c = 0; c < C; c++)
#pragma unroll
            for (int e = 0; e < VEC; e++) sum[c][e] += r[u][c].get(e);
        }
    } else {
      T r[R][C][VEC];
#pragma unroll
      for (int u = 0; u < R; u++)
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
          for (int e = 0; e < VEC; e++) r[u][c][e] = j + u < len && inside(c, e) ? at[u][c * 128 + 32 * e] : Elem<T>::put(0.f);
#pragma unroll
      for (int u = 0; u < R; u++)
        if (j + u < len) {
#pragma unroll
          for (int c = 0; c < C; c++)
#pragma unroll
            for (int e = 0; e < VEC; e++) sum[c][e] += Elem<T>::get(r[u][c][e]);
        }
    }
  }
  static_assert(EM_CHUNK == 32 || EM_CHUNK == 64, "one or two words of tokens a lane");
  if (unit.y & EM_MORE) {
    float* const to = a.part + slot_of(a, unit.x, len) * a.cols + c0;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int e = 0; e < VEC; e++)
        if (inside(c, e)) to[c * 32 * VEC + e * STRIDE] = sum[c][e];
    return;
  }
  T* const to = static_cast<T*>(a.dw) + (int64_t)unit.z * a.ws + c0;
#pragma unroll
  for (int c = 0; c < C; c++) {
#pragma unroll
    for (int e = 0; e < VEC; e++) sum[c][e] *= a.scale;
    if constexpr (AL) {
      Run<T, VEC> o;
      o.set(sum[c]);
      if (inside(c, 0)) o.store(to + c * 32 * VEC);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; e++)
        if (inside(c, e)) to[c * 128 + 32 * e] = Elem<T>::put(sum[c][e]);
    }
  }
}
constexpr int SUM_CTAS = 152 * 3;   // as many as fit
template <typename T, bool AL>
__global__ void __launch_bounds__(256, 3) em_sum_kernel(const __grid_constant__ EmArgs a, int from) {
  constexpr int RUN = 32 * (AL ? Elem<T>::VEC : 4), WIDE = 4;
  after_previous();
  next_may_start();
  const EmUnits found = *a.found;
  const int64_t narrow = (a.cols + RUN - 1) / RUN, wide = (a.cols + WIDE * RUN - 1) / (WIDE * RUN);
  const int64_t many = found.many * narrow, all = many + found.few * wide, warps = (int64_t)gridDim.x * 8;
  for (int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5; w < all; w += warps) {   // the long ones first
    if (w < many) sum_chunk<T, AL, 1, 8>(a, a.unit[a.n - 1 - w / narrow], (w % narrow) * RUN, from);
    else sum_chunk<T, AL, WIDE, 2>(a, a.unit[(w - many) / wide], ((w - many) % wide) * (WIDE * RUN), from);
  }
}

// ---- rows of several chunks: a CTA 128 columns of one, its eight warps a run of the chunks each ----
template <typename T>
__global__ void __launch_bounds__(256) em_join_kernel(const __grid_constant__ EmArgs a) {
  __shared__ float sums[8][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_previous();
  const int64_t pieces = (a.cols + 127) / 128, all = a.found->rows * pieces;
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    const uint4 row = a.row[w / pieces];
    const int64_t c0 = (w % pieces) * 128 + lane, first = row.x, end = row.y;
    const int64_t chunks = (end - first + EM_CHUNK - 1) / EM_CHUNK, per = (chunks + 7) / 8;
    const int64_t q0 = min(chunks, warp * per), q1 = min(chunks, q0 + per);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t q = q0; q < q1; q += 4) {
      float v[4][4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int64_t i = first + (q + u) * EM_CHUNK;
        const float* const at = a.part + slot_of(a, i, (uint32_t)min((int64_t)EM_CHUNK, end - i)) * a.cols + c0;
#pragma unroll
        for (int e = 0; e < 4; e++) v[u][e] = q + u < q1 && c0 + 32 * e < a.cols ? at[32 * e] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; u++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (q + u < q1) sum[e] += v[u][e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; e++) sums[warp][32 * e + lane] = sum[e];
    __syncthreads();
    const int64_t c = (w % pieces) * 128 + threadIdx.x;
    if (threadIdx.x < 128 && c < a.cols) {
      float total = sums[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < 8; k++) total += sums[k][threadIdx.x];
      static_cast<T*>(a.dw)[(int64_t)row.z * a.ws + c] = Elem<T>::put(total * a.scale);
    }
  }
}

bool rows_aligned(const void* p, int64_t stride, int64_t cols, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0 && cols * es % 16 == 0;
}

template <typename T, bool AL>
cudaError_t lookup(const EmArgs& a, cudaStream_t st) {
  const int64_t run = 32 * LOOKUP_RUNS * (AL ? Elem<T>::VEC : 1), pieces = (a.cols + run - 1) / run;
  em_lookup_kernel<T, AL><<<(unsigned)((a.n * pieces + 7) / 8), 256, 0, st>>>(a, (uint32_t)pieces);
  return cudaGetLastError();
}
template <typename T, bool AL>
cudaError_t sums(const EmArgs& a, int from, cudaStream_t st) {
  constexpr int RUN = 32 * (AL ? Elem<T>::VEC : 4);
  const int64_t most = a.n * ((a.cols + RUN - 1) / RUN);   // warps' items
  const cudaError_t e = launch_early(em_sum_kernel<T, AL>, dim3((unsigned)std::min<int64_t>(SUM_CTAS, (most + 7) / 8)), 256, 0, st, a, from);
  if (e != cudaSuccess || a.n <= EM_CHUNK) return e;
  return launch_early(em_join_kernel<T>, dim3((unsigned)std::min<int64_t>(152 * 2, a.n / EM_CHUNK * ((a.cols + 127) / 128))), 256, 0, st, a);
}
template <typename T>
cudaError_t gradient(const EmArgs& a, int from, cudaStream_t st) {
  return rows_aligned(a.dy, a.ys, a.cols, sizeof(T)) && rows_aligned(a.dw, a.ws, a.cols, sizeof(T)) ? sums<T, true>(a, from, st)
                                                                                                  : sums<T, false>(a, from, st);
}

}  // namespace

cudaError_t launch_embedding(const EmArgs& a, cudaStream_t st) {
  const int es = a.dtype == DA_F32 ? 4 : 2;
  const bool al = rows_aligned(a.w, a.ws, a.cols, es) && rows_aligned(a.y, a.ys, a.cols, es);
  if (a.dtype == DA_F32) return al ? lookup<float, true>(a, st) : lookup<float, false>(a, st);
  if (a.dtype == DA_BF16) return al ? lookup<__nv_bfloat16, true>(a, st) : lookup<__nv_bfloat16, false>(a, st);
  return al ? lookup<__half, true>(a, st) : lookup<__half, false>(a, st);
}

cudaError_t launch_embedding_grad(const EmArgs& a, cudaStream_t st) {
  const int es = a.dtype == DA_F32 ? 4 : 2;
  const bool flat = a.rows <= 1 || a.ws == a.cols;
  cudaError_t e = cudaSuccess;
  if (!flat || a.n == 0) e = cudaMemset2DAsync(a.dw, (size_t)a.ws * es, 0, (size_t)a.cols * es, (size_t)a.rows, st);
  if (e != cudaSuccess || a.n == 0) return e;
  int need = 1, from = 0;
  while (need < 32 && ((uint64_t)1 << need) <= (uint64_t)a.rows) need++;   // bits of the keys 0 .. rows
  const int passes = (need + 8) / 9, bits = std::max(2, (need + passes - 1) / passes);
  const int64_t bytes = flat ? a.rows * a.cols * es : 0;
  const auto fillers = [&](int64_t part, int threads) {   // CTAs for so many bytes of zeros
    return (unsigned)std::min<int64_t>(152 * 1024 / threads, (part + 128 * threads - 1) / (128 * threads));
  };
  if (a.n <= EM_SMALL) {
    static DeviceOnce once;
    if ((e = allow_smem(once, em_sort_kernel, (int)sizeof(SortSmall))) != cudaSuccess) return e;
    em_sort_kernel<<<1, SORT_THREADS, sizeof(SortSmall), st>>>(a, passes, bits);
    if ((e = cudaGetLastError()) == cudaSuccess && flat) e = launch_early(em_fill_kernel, dim3(fillers(bytes, 256)), 256, 0, st, a);
  } else {
    const int block = em_block(a.n);
    const uint32_t blocks = (uint32_t)((a.n + block - 1) / block), chunks = (uint32_t)((a.n + 255) / 256);
    const bool add = block == 1024;   // 32 blocks at most
    const uint32_t each = add ? 2 : 3, parts = each * passes + 1;   // launches of a pass
    const int64_t part = (bytes + parts - 1) / parts;   // rounded up: where there are fewer bytes than parts, one CTA still writes the ends
    const unsigned f = fillers(part, 256), g = fillers(part, 1024);
    for (int p = 0; p < passes && e == cudaSuccess; p++) {
      const int src = p ? (p + 1) & 1 : -1, dst = p & 1, shift = p * bits;
      const auto fill = [&](uint32_t k) { return Fill{each * p + k, parts}; };
      if (p == 0) {   // after everything before it; the others only wait for each other
        em_count_kernel<<<blocks + f, RADIX_THREADS, 0, st>>>(a, blocks, block, add, src, shift, bits, fill(0));
        e = cudaGetLastError();
      } else {
        e = launch_early(em_count_kernel, dim3(blocks + f), RADIX_THREADS, 0, st, a, blocks, block, add, src, shift, bits, fill(0));
      }
      if (e == cudaSuccess && !add) e = launch_early(em_scan_kernel, dim3(1 + g), 1024, 0, st, a, (int64_t)blocks << bits, fill(1));
      const auto scatter = add ? em_scatter_kernel<4, true> : em_scatter_kernel<8, false>;
      if (e == cudaSuccess)
        e = launch_early(scatter, dim3(blocks + f), RADIX_THREADS, 0, st, a, blocks, src, dst, shift, bits, fill(each - 1));
      from = dst;
    }
    if (e == cudaSuccess) e = launch_early(em_chunk_kernel, dim3(chunks + f), 256, 0, st, a, chunks, from, Fill{parts - 1, parts});
  }
  if (e != cudaSuccess) return e;
  if (a.dtype == DA_F32) return gradient<float>(a, from, st);
  return a.dtype == DA_BF16 ? gradient<__nv_bfloat16>(a, from, st) : gradient<__half>(a, from, st);
}

}  // namespace detattn
