// Element types of the training operators: loads and stores of 16-bit and 32-bit floats as
// binary32, each store rounded once to nearest even.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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

// N elements moved by one access of N * sizeof(T) bytes
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T e[N];
};

__device__ __forceinline__ float warp_sum(float x) {   // the same tree, and so the same bits, in every lane
#pragma unroll
  for (int o = 16; o; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

}  // namespace detattn
