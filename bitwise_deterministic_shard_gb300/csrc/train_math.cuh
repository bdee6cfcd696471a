// Element types of the training operators: loads and stores of 16-bit and 32-bit floats as
// binary32, each store rounded once to nearest even.
#pragma once
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pack2.cuh"

namespace detattn {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int VEC = 4;   // elements of 16 bytes
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<__half> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};

// A run of N elements moved by one access of 8 or 16 bytes, kept as 32-bit words: two 16-bit elements are taken from
// and put into a word by one or two instructions (element-wise structures of 16-bit types are not).
template <typename T, int N>
struct Run {
  static constexpr int WORDS = sizeof(T) * N / 4;
  static_assert(WORDS == 2 || WORDS == 4, "8 or 16 bytes");
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (WORDS == 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (WORDS == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; i++) w[i] = 0;
  }
  // The words stay words: without this the compiler keeps the binary32 elements of one pass over
  // a row for the next (twice the registers of the 16-bit words, and spills).
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int i = 0; i < WORDS; i++) asm volatile("" : "+r"(w[i]));
  }
  // the bits of element e (the run starts from zero)
  __device__ __forceinline__ void put_bits(int e, T x) {
    if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(*reinterpret_cast<const float*>(&x));
    else w[e >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(&x) << (16 * (e & 1));
  }
  __device__ __forceinline__ T bits(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else {
      const uint16_t x = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      return *reinterpret_cast<const T*>(&x);
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e >> 1]));
      return e & 1 ? f.y : f.x;
    }
  }
  // elements 2 i and 2 i + 1 as a packed pair
  __device__ __forceinline__ f2::u64 get2(int i) const { return f2::pack(get(2 * i), get(2 * i + 1)); }
  __device__ __forceinline__ void set2(int i, f2::u64 x) {
    float a, b;
    f2::unpack(x, a, b);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(a);
      w[2 * i + 1] = __float_as_uint(b);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
    } else {
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
    }
  }
  __device__ __forceinline__ void set(const float* x) {   // all N elements, rounded to nearest even
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < WORDS; i++) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < WORDS; i++) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        else
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
      }
    }
  }
};

__device__ __forceinline__ float warp_sum(float x) {   // the same tree, and so the same bits, in every lane
#pragma unroll
  for (int o = 16; o; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

}  // namespace detattn
