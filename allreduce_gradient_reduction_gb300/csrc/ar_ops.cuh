// Device-side pieces that the training-step operators share: elements of
// f32, bf16 and f16 widened to binary32 and rounded back to nearest even, one
// or 16 bytes at a time, and sums over groups of threads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ar_ops.h"

namespace ar {

template <class T> struct Conv;
template <> struct Conv<float> {
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};
template <> struct Conv<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Conv<__half> {
  static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
};

// N consecutive elements, moved by one access of N * sizeof(T) bytes.
template <class T, int N>
struct alignas(N * sizeof(T)) Pack {
  T v[N];
};

template <class T, int N>
__device__ __forceinline__ Pack<T, N> zero_pack() {
  Pack<T, N> p;
#pragma unroll
  for (int i = 0; i < N; ++i) p.v[i] = Conv<T>::down(0.f);
  return p;
}

// Elements [c, c + N) of a row of `cols`, those past its end as zeros.
template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* row, int c, int cols) {
  if (c + N <= cols) return *reinterpret_cast<const Pack<T, N>*>(row + c);
  Pack<T, N> p = zero_pack<T, N>();
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (c + i < cols) p.v[i] = row[c + i];
  return p;
}

template <class T, int N>
__device__ __forceinline__ void store_pack(T* row, int c, int cols, const Pack<T, N>& p) {
  if (c + N <= cols) {
    *reinterpret_cast<Pack<T, N>*>(row + c) = p;
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (c + i < cols) row[c + i] = p.v[i];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
  return v;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Applies a launch's element type to a function object: fn(T()).
template <class F>
cudaError_t with_type(int dtype, F fn) {
  switch (dtype) {
    case F32: return fn(float());
    case BF16: return fn(__nv_bfloat16());
    case F16: return fn(__half());
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ar
