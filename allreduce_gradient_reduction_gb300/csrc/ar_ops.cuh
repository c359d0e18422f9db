// Device-side pieces that the training-step operators share: elements of
// f32, bf16 and f16 widened to binary32 and rounded back to nearest even, one
// or 16 bytes at a time, and sums over groups of threads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "../../include/ar.h"
#include "ar_ops.h"

namespace ar {

// AR_ERR_TIMEOUT once a wait of one of the including file's kernels has run out.
static __device__ int g_status;

// Host: a kernel of the including file has been launched (or captured).
static std::atomic<bool> g_launched{false};
static inline void note_launch() {
  g_launched.store(true, std::memory_order_relaxed);
  count_launch();
}

// Host: reads it into *status if it is set, and clears it, in `stream` alone.
// Nothing is asked of the device before a first launch.
static inline cudaError_t take_status(int* status, cudaStream_t stream) {
  if (!g_launched.load(std::memory_order_relaxed)) return cudaSuccess;
  void* at = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&at, g_status);
  return e == cudaSuccess ? take_word(at, status, stream) : e;
}

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

// Two binary32 values in one register pair, and the operations that take pairs.
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float lo, float hi) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(Two t, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(t.v));
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two neg2(Two a) { return Two{a.v ^ 0x8000000080000000ull}; }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---- pairs of 16-bit elements in one word ------------------------------------------

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The two elements of a word, widened.
template <class T>
__device__ __forceinline__ Two unpack2(uint32_t w);
template <>
__device__ __forceinline__ Two unpack2<__nv_bfloat16>(uint32_t w) {
  return two(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ Two unpack2<__half>(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return two(f.x, f.y);
}
// The larger of each pair; a NaN gives way to a number.
template <class T>
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t max_pairs<__nv_bfloat16>(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t max_pairs<__half>(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 bytes of elements as pairs of binary32 values, and back.
template <class T>
struct Pairs {
  static constexpr int N = 4;  // pairs in 16 bytes
  static __device__ __forceinline__ Two get(const uint4& v, int i) {
    return unpack2<T>(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ void set(uint4& v, int i, Two t) {
    float lo, hi;
    split(t, lo, hi);
    (i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w) = pack2<T>(lo, hi);
  }
};
template <>
struct Pairs<float> {
  static constexpr int N = 2;
  static __device__ __forceinline__ Two get(const uint4& v, int i) {
    return i == 0 ? two(__uint_as_float(v.x), __uint_as_float(v.y)) : two(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ void set(uint4& v, int i, Two t) {
    float lo, hi;
    split(t, lo, hi);
    (i == 0 ? v.x : v.z) = __float_as_uint(lo);
    (i == 0 ? v.y : v.w) = __float_as_uint(hi);
  }
};

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- bulk copies into shared memory, announced on an mbarrier ---------------------

__device__ __forceinline__ uint32_t smem_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void ring_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// The aligned words of `bytes` bytes at `from`.
__device__ __forceinline__ uint32_t covering(const void* from, int bytes) {
  return (((uint32_t)(uintptr_t)from & 15) + bytes + 15) & ~15u;
}
__device__ __forceinline__ void ring_copy(uint32_t to, const void* from, int bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
               "l"((uintptr_t)from & ~(uintptr_t)15), "r"(covering(from, bytes)), "r"(bar)
               : "memory");
}

// Looks for the end of the phase of the given parity, asleep for a while: the
// instruction comes back by itself after 3.8 us, however long a time it is
// given, so a limit has to be counted on the clock and not in looks.
__device__ __forceinline__ bool ring_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(10000000)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // one wait

// Waits for the phase of the given parity to end.  A copy ends by itself, so
// this does too; the limit (two seconds) is for a launch that has gone wrong.
// One wait that runs out ends the block's others, through `gave_up`, and is
// reported in g_status.  The threads go on to the kernel's end all the same,
// so that none is missing at a barrier, but begin no more copies (the last
// ones began two seconds before).
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  if (ring_try(bar, parity)) return true;
  const uint64_t until = global_ns() + kWaitLimitNs;
#pragma unroll 1
  do {
    if (ring_try(bar, parity)) return true;
    if (*gave_up) return false;
  } while (global_ns() < until);
  *gave_up = 1;
  g_status = AR_ERR_TIMEOUT;
  return false;
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
