// What the backward kernels of ordinary and differential attention share: the
// powers of two that f16 score gradients are held times, the end of a walk, and
// the wait for the kernel before.
#pragma once

#include "ar_tcgen05.cuh"

namespace ar {

// Score gradients are as large as dout, whose size is the user's (a loss may be
// scaled by any power of two), times a probability.  f16 holds them as they are
// where the block's largest lies in [2^-12, 65504], so that what is too small
// to count is below 2^-13 of it.  Otherwise the block walks again, with them
// times another power of two:
//   - One past 65504 is an infinity in f16 and leaves none of its row's sums
//     finite, which is seen when they are written: 2^-13 and, if need be, 2^-26,
//     which no product of f16 operands outgrows.  What is lost is below 2^-28
//     of the largest.
//   - A thread looks at one of its 32 in each step.  If none of the block's is
//     2^-12, 2^26; should larger ones overflow then, 2^13 and 1.
// Device time of 8191 tokens in 13 sequences, 12 heads of 64: 79.1 us, and 76.8
// without any of this; 82.2 with a look at all 32 for the exact power, 81.3 with
// all walks in one loop (the first is compiled apart, its power a constant).
// Walks that follow cost as much each: 3000 tokens, 12 heads of 64, 67 us with
// one walk, 124 with two.  (A power that is known beforehand would have to bound
// v and dout over a whole sequence, a pass of its own over both; a fixed one
// loses either kind.)
template <class T>
constexpr bool kScaled = __is_same(T, __half);
constexpr float kTooSmall = 0x1p-12f, kUnknown = 0x1p-100f;
constexpr float kRaised = 0x1p26f, kLowered = 0x1p-13f, kLeast = 0x1p-26f;

// The end of the kernel that makes delta.  What else a block reads was there
// before that kernel began, so its loads and first products need not wait; but
// every block waits before it ends, so that whatever comes next in the stream
// finds both kernels done.
__device__ __forceinline__ void wait_for_delta() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Where a first walk has met nothing but zeros: whether a worker's part of its
// row of dout (64 of the tile's bytes) holds anything else.
__device__ __forceinline__ bool any_element(uint32_t at) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + i * 16) : "memory");
    any |= v.x | v.y | v.z | v.w;
  }
  return (any & 0x7FFF7FFFu) != 0;
}

// What a worker has seen, for leave(): infinity where sums are not finite, zero
// if there is nothing but zeros.
template <class T>
__device__ __forceinline__ void put_most(float most, bool finite, float* each) {
  if constexpr (!kScaled<T>) return;
  __syncwarp();
  most = warp_max(finite ? most : INFINITY);
  if ((threadIdx.x & 31) == 0) each[threadIdx.x >> 5] = most;
}

// What a block keeps from one walk to the next.
struct State {
  float by = 1.f;           // what the score gradients are held times
  int walks = 0;            // made
  uint32_t own_parity = 0;  // the loader's
};

// The end of a walk: true, with another power, if the block has to walk again.
template <class T, class F>
__device__ __forceinline__ bool leave(int* gave_up, int warp, uint32_t tmem, const float* each, State& state) {
  tc_fence_before();
  __syncthreads();
  if (*(volatile int*)gave_up) {
    // copies and products in flight end by themselves: give them time
    for (int i = 0; i < 100; ++i) __nanosleep(100000);
    if (threadIdx.x == 0) g_status = AR_ERR_TIMEOUT;
    __syncthreads();
  } else if (kScaled<T>) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < F::kWorkers / 32; ++i) most = fmaxf(most, each[i]);
    const bool lower = most == INFINITY && state.by > kLeast;
    const bool raise = state.walks == 0 && most > 0.f && most < kTooSmall;
    if (lower || raise) {
      state.by = lower ? state.by * kLowered : kRaised;
      ++state.walks;
      fence_async_shared();  // tiles are copied to where results have been
      __syncthreads();
      tc_fence_after();
      return true;
    }
  }
  if (warp == F::kIssuer) tmem_free(tmem, F::kColumns);
  return false;
}

// Elements x and x + 1 of a vector in shared memory, x even, read four at a time.
__device__ __forceinline__ Two two_of(const float* v, int x) {
  const ulonglong2 four = *reinterpret_cast<const ulonglong2*>(v + (x & ~3));
  return Two{x & 2 ? four.y : four.x};
}

}  // namespace ar
