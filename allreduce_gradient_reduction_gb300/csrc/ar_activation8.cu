// An activation whose input is kept in 8 bits for the backward pass.
//
// 128 elements of a row share a scale: with m the largest of them in size,
//   code_i = the nearest whole number to x_i (127 / m), scale = m / 127,
// one division and one product in binary32 each, so that the codes are the same
// wherever they are made.  Forward writes y = act(x), codes and scales;
// backward takes xk = code scale and writes dx = dy act'(xk) and act(xk), the
// next layer's input, which its weight's gradient needs.
//
// Bound by HBM: with 16-bit elements 2 + 2 + 1 bytes an element forward and
// 1 + 2 + 2 + 2 backward.  16 lanes share a block of 128, eight elements each,
// so that its largest takes four exchanges and every access is 8 or 16 bytes
// to a lane; a thread has several blocks' loads under way at once.  Rows that
// do not lie on 16-byte boundaries move element by element, neighbours to
// neighbouring lanes (4095 x 5003 f16 backward 37 us; 86 with aligned words that
// lanes shift against each other).
//
// Measured: 16384 x 10240 bf16, gelu by tanh, forward and backward together 307 us
// (6.6 TB/s); 16384 x 2048 f32 packed and unpacked 58 us (5.9 TB/s).
#include <cuda_runtime.h>

#include <algorithm>

#include "ar_ops.cuh"

namespace ar {
namespace {

constexpr int kBlock = kActivation8Block;
constexpr int kThreads = 256;
constexpr float kLeast = 0x1p-120f;  // blocks below it are zeros

__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ Two reciprocal(Two t) {
  float lo, hi;
  split(t, lo, hi);
  return two(reciprocal(lo), reciprocal(hi));
}
__device__ __forceinline__ Two exp2_approx(Two t) {
  float lo, hi;
  split(t, lo, hi);
  return two(ar::exp2_approx(lo), ar::exp2_approx(hi));
}
__device__ __forceinline__ Two both(float v) { return two(v, v); }
// The largest in size; NaN if there is one.
__device__ __forceinline__ float most_of(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
__device__ __forceinline__ float most_of(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// gelu(x) = x s with s = 1 / (1 + e^-u), u = sqrt(8 / pi) (x + 0.044715 x^3):
// (1 + tanh(u / 2)) / 2 without its cancellation at negative x.
constexpr float kU1 = 1.5957691216057308f, kU3 = kU1 * 0.044715f, kLog2e = 1.4426950408889634f;

// The normal distribution's integral at -|x|, and e^(-x^2 / 2).  erfc(y)
// e^(y^2) = t Q(t) with t = 1 / (1 + y / 2); Q of degree 8 was fitted by
// weighted least squares for the least relative error, 4.4e-8, over y <= 14.7.
__device__ __forceinline__ Two normal_tail(Two x, Two& bell) {
  const Two size = Two{x.v & 0x7FFFFFFF7FFFFFFFull};
  const Two t = reciprocal(fma2(size, both(0.35355339059327379f), both(1.f)));
  bell = exp2_approx(mul2(mul2(x, x), both(-0.72134752044448169f)));
  Two q = fma2(both(-0.0593869729f), t, both(0.286126333f));
  q = fma2(q, t, both(-0.490410976f));
  q = fma2(q, t, both(0.28173817f));
  q = fma2(q, t, both(-0.0291516083f));
  q = fma2(q, t, both(0.203753693f));
  q = fma2(q, t, both(0.242834857f));
  q = fma2(q, t, both(0.282412128f));
  q = fma2(q, t, both(0.28208433f));
  return mul2(mul2(bell, both(0.5f)), mul2(t, q));
}
// From the integral at -|x| that at x.
__device__ __forceinline__ Two normal_at(Two x, Two tail) {
  float x0, x1, t0, t1, u0, u1;
  split(x, x0, x1);
  split(tail, t0, t1);
  split(fma2(tail, both(-1.f), both(1.f)), u0, u1);
  return two(x0 < 0.f ? t0 : u0, x1 < 0.f ? t1 : u1);
}

// Two elements at a time.
template <int KIND>
__device__ __forceinline__ Two activation(Two x) {
  if constexpr (KIND == AR_ACT_GELU_TANH) {
    const Two u = mul2(x, fma2(both(-kU3 * kLog2e), mul2(x, x), both(-kU1 * kLog2e)));
    return mul2(x, reciprocal(add2(both(1.f), exp2_approx(u))));
  } else if constexpr (KIND == AR_ACT_GELU) {
    Two bell;
    const Two tail = normal_tail(x, bell);
    return mul2(x, normal_at(x, tail));
  } else {
    return x;
  }
}

// The activation and its slope.  `one` is one, or a NaN for a block of those.
// Beyond 10.035 (the exact gelu: 18) the slope is that there, 0 or 1, and so is
// the activation's factor: e^-u is 2^127.1 or so, still a number, and its
// reciprocal is flushed to zero.  Farther out an infinity would be multiplied by
// zero.
template <int KIND>
__device__ __forceinline__ void activation_and_slope(Two x, float one, Two& y, Two& slope) {
  if constexpr (KIND == AR_ACT_IDENTITY) {
    y = mul2(x, both(one));
    slope = both(one);
    return;
  }
  constexpr float kFar = KIND == AR_ACT_GELU ? 18.f : 10.035f;
  float x0, x1;
  split(x, x0, x1);
  x0 = fmaxf(x0, -kFar);
  x1 = fmaxf(x1, -kFar);
  const Two low = two(x0, x1), c = two(fminf(x0, kFar), fminf(x1, kFar));
  if constexpr (KIND == AR_ACT_GELU_TANH) {
    const Two sq = mul2(c, c);
    const Two e = exp2_approx(mul2(c, fma2(both(-kU3 * kLog2e), sq, both(-kU1 * kLog2e))));
    const Two s = reciprocal(add2(both(one), e));
    y = mul2(low, s);
    slope = fma2(mul2(mul2(c, s), mul2(e, s)), fma2(both(3.f * kU3), sq, both(kU1)), s);
  } else {
    Two bell;
    const Two tail = normal_tail(c, bell);
    const Two all = mul2(normal_at(c, tail), both(one));
    y = mul2(low, all);
    slope = fma2(mul2(c, both(0.3989422804014327f)), bell, all);
  }
}

// Which elements of a block a lane has, as they are read and written.  Side by
// side: 16 lanes to a block, eight elements each.  Apart: a warp to a block,
// every 32nd element.  `left` of the block's elements are in the row; the
// others are zeros.
template <class T, bool SIDE_BY_SIDE>
struct Places {
  static constexpr int kLanes = 16, kEach = 8, kTwos = 4;
  static constexpr int kGroups = kThreads / kLanes;  // blocks at a time
  static constexpr int kPer = 16 / (int)sizeof(T);   // elements of a vector
  struct Raw {
    uint4 v[kEach / kPer];
  };
  using Codes = uint2;
  // Vectors of neighbouring lanes lie side by side (f32: two of them in each half
  // of the block).
  static __device__ __forceinline__ int vector(int lane, int h) { return h * kLanes * kPer + lane * kPer; }
  static __device__ __forceinline__ Raw load(const T* from, int left, int lane) {
    Raw r;
#pragma unroll
    for (int h = 0; h < kEach / kPer; ++h) {
      if (left >= kBlock) {
        r.v[h] = *reinterpret_cast<const uint4*>(from + vector(lane, h));
      } else {
        const Pack<T, kPer> p = load_pack<T, kPer>(from, vector(lane, h), left);
        r.v[h] = *reinterpret_cast<const uint4*>(&p);
      }
    }
    return r;
  }
  static __device__ __forceinline__ Two get(const Raw& r, int i) { return Pairs<T>::get(r.v[i / (kPer / 2)], i % (kPer / 2)); }
  static __device__ __forceinline__ void store(T* to, int left, int lane, const Two (&f)[kTwos]) {
#pragma unroll
    for (int h = 0; h < kEach / kPer; ++h) {
      uint4 v;
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) Pairs<T>::set(v, i, f[h * (kPer / 2) + i]);
      if (left >= kBlock) *reinterpret_cast<uint4*>(to + vector(lane, h)) = v;
      else store_pack<T, kPer>(to, vector(lane, h), left, *reinterpret_cast<const Pack<T, kPer>*>(&v));
    }
  }
  static __device__ __forceinline__ Codes load_codes(const int8_t* from, int lane) {
    if constexpr (kPer == kEach) return *reinterpret_cast<const uint2*>(from + vector(lane, 0));
    else return make_uint2(*reinterpret_cast<const uint32_t*>(from + vector(lane, 0)),
                           *reinterpret_cast<const uint32_t*>(from + vector(lane, 1)));
  }
  // 2^23 + 128 + code
  static __device__ __forceinline__ Two lifted(const Codes& c, int i) {
    const uint32_t w = (i < 2 ? c.x : c.y) ^ 0x80808080u, at = 2 * (i & 1);
    return two(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | at)),
               __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | (at + 1))));
  }
  // from whole numbers that 1.5 * 2^23 was added to
  static __device__ __forceinline__ void store_codes(int8_t* to, int lane, const Two (&c)[kTwos]) {
    auto four = [&](int i) {
      float a0, a1, a2, a3;
      split(c[i], a0, a1);
      split(c[i + 1], a2, a3);
      return __byte_perm(__byte_perm(__float_as_uint(a0), __float_as_uint(a1), 0x0040),
                         __byte_perm(__float_as_uint(a2), __float_as_uint(a3), 0x0040), 0x5410);
    };
    if constexpr (kPer == kEach) {
      *reinterpret_cast<uint2*>(to + vector(lane, 0)) = make_uint2(four(0), four(2));
    } else {
      *reinterpret_cast<uint32_t*>(to + vector(lane, 0)) = four(0);
      *reinterpret_cast<uint32_t*>(to + vector(lane, 1)) = four(2);
    }
  }
};
template <class T>
struct Places<T, false> {
  static constexpr int kLanes = 32, kEach = 4, kTwos = 2;
  static constexpr int kGroups = kThreads / kLanes;
  struct Raw {
    T v[kEach];
  };
  struct Codes {
    uint8_t v[kEach];
  };
  static __device__ __forceinline__ Raw load(const T* from, int left, int lane) {
    Raw r;
    from += lane;
    if (left >= kBlock) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) r.v[i] = from[32 * i];
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) r.v[i] = lane + 32 * i < left ? from[32 * i] : Conv<T>::down(0.f);
    }
    return r;
  }
  static __device__ __forceinline__ Two get(const Raw& r, int i) {
    return two(Conv<T>::up(r.v[2 * i]), Conv<T>::up(r.v[2 * i + 1]));
  }
  static __device__ __forceinline__ void store(T* to, int left, int lane, const Two (&f)[kTwos]) {
    to += lane;
    T v[kEach];
#pragma unroll
    for (int i = 0; i < kTwos; ++i) {
      float lo, hi;
      split(f[i], lo, hi);
      v[2 * i] = Conv<T>::down(lo);
      v[2 * i + 1] = Conv<T>::down(hi);
    }
    if (left >= kBlock) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) to[32 * i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (lane + 32 * i < left) to[32 * i] = v[i];
    }
  }
  static __device__ __forceinline__ Codes load_codes(const int8_t* from, int lane) {
    Codes c;
#pragma unroll
    for (int i = 0; i < kEach; ++i) c.v[i] = (uint8_t)from[lane + 32 * i];
    return c;
  }
  static __device__ __forceinline__ Two lifted(const Codes& c, int i) {
    return two(__uint_as_float((c.v[2 * i] ^ 0x80u) | 0x4B000000u), __uint_as_float((c.v[2 * i + 1] ^ 0x80u) | 0x4B000000u));
  }
  static __device__ __forceinline__ void store_codes(int8_t* to, int lane, const Two (&c)[kTwos]) {
#pragma unroll
    for (int i = 0; i < kTwos; ++i) {
      float lo, hi;
      split(c[i], lo, hi);
      to[lane + 64 * i] = (int8_t)__float_as_uint(lo);
      to[lane + 64 * i + 32] = (int8_t)__float_as_uint(hi);
    }
  }
};

// Where block n of the matrix lies.
struct Place {
  uint32_t row;
  int col;
};
__device__ __forceinline__ Place place_of(const Activation8Args& a, uint32_t n) {
  const uint32_t row = (uint32_t)(((uint64_t)n * a.magic) >> a.shift);
  return Place{row, (int)(n - row * (uint32_t)a.blocks) * kBlock};
}

template <class T, int KIND, bool SIDE_BY_SIDE, int EACH>
__global__ void __launch_bounds__(kThreads) activation8_kernel(const __grid_constant__ Activation8Args a) {
  using P = Places<T, SIDE_BY_SIDE>;
  const int lane = threadIdx.x % P::kLanes, group = threadIdx.x / P::kLanes;
  const uint32_t first = (blockIdx.x * EACH) * P::kGroups + group;
  typename P::Raw raw[EACH];
  Place at[EACH];
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const uint32_t n = first + u * P::kGroups;
    at[u] = place_of(a, n);
    // no block n: nothing of the row is left
    raw[u] = P::load(static_cast<const T*>(a.x) + (int64_t)at[u].row * a.x_stride + at[u].col,
                     n < a.total ? a.cols - at[u].col : 0, lane);
  }
  // Every block's largest, then 127 / m and m / 127 of block u by the group's
  // lane u: a quotient rounded right takes as many instructions as five elements.
  float mine = 0.f;
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < P::kTwos; ++i) {
      float lo, hi;
      split(P::get(raw[u], i), lo, hi);
      most = most_of(lo, hi, most);
    }
#pragma unroll
    for (int m = P::kLanes / 2; m; m >>= 1) most = most_of(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));
    if (lane == u) mine = most;
  }
  const bool some = mine >= kLeast && mine < INFINITY;
  const float my_by = some ? __fdiv_rn(127.f, mine) : 0.f;
  if (lane < EACH && first + lane * P::kGroups < a.total)
    a.scales_out[first + lane * P::kGroups] = some ? __fdiv_rn(mine, 127.f) : mine < kLeast ? 0.f : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const uint32_t n = first + u * P::kGroups;
    const float by = __shfl_sync(0xFFFFFFFFu, my_by, u, P::kLanes);
    if (n >= a.total) continue;
    Two f[P::kTwos];
#pragma unroll
    for (int i = 0; i < P::kTwos; ++i) f[i] = P::get(raw[u], i);
    // adding 1.5 * 2^23 leaves the nearest whole number in the low bits (one value
    // at a time: of a pair's product and sum the compiler makes one rounding)
    Two code[P::kTwos];
#pragma unroll
    for (int i = 0; i < P::kTwos; ++i) {
      float lo, hi;
      split(f[i], lo, hi);
      lo = __fadd_rn(__fmul_rn(lo, by), 12582912.f);
      hi = __fadd_rn(__fmul_rn(hi, by), 12582912.f);
      code[i] = by > 0.f ? two(lo, hi) : both(12582912.f);
    }
    P::store_codes(a.codes_out + (int64_t)n * kBlock, lane, code);
    if (a.y) {
#pragma unroll
      for (int i = 0; i < P::kTwos; ++i) f[i] = activation<KIND>(f[i]);
      P::store(static_cast<T*>(a.y) + (int64_t)at[u].row * a.y_stride + at[u].col, a.cols - at[u].col, lane, f);
    }
  }
}

template <class T, int KIND, bool SIDE_BY_SIDE, int EACH>
__global__ void __launch_bounds__(kThreads) activation8_backward_kernel(const __grid_constant__ Activation8Args a) {
  using P = Places<T, SIDE_BY_SIDE>;
  const int lane = threadIdx.x % P::kLanes, group = threadIdx.x / P::kLanes;
  const uint32_t first = (blockIdx.x * EACH) * P::kGroups + group;
  typename P::Raw raw[EACH];
  typename P::Codes codes[EACH];
  float scale[EACH];
  Place at[EACH];
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const uint32_t n = first + u * P::kGroups;
    if (n >= a.total) break;
    at[u] = place_of(a, n);
    codes[u] = P::load_codes(a.codes + (int64_t)n * kBlock, lane);
    scale[u] = a.scales[n];
    if (a.dx) raw[u] = P::load(static_cast<const T*>(a.x) + (int64_t)at[u].row * a.x_stride + at[u].col, a.cols - at[u].col, lane);
  }
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    if (first + u * P::kGroups >= a.total) break;
    const float one = scale[u] == scale[u] ? 1.f : scale[u];
    Two y[P::kTwos], d[P::kTwos];
#pragma unroll
    for (int i = 0; i < P::kTwos; ++i) {
      const Two x = mul2(add2(P::lifted(codes[u], i), both(-8388736.f)), both(scale[u]));
      Two slope;
      activation_and_slope<KIND>(x, one, y[i], slope);
      d[i] = slope;
    }
    const int left = a.cols - at[u].col;
    if (a.dx) {
#pragma unroll
      for (int i = 0; i < P::kTwos; ++i) d[i] = mul2(d[i], P::get(raw[u], i));
      P::store(static_cast<T*>(a.dx) + (int64_t)at[u].row * a.dx_stride + at[u].col, left, lane, d);
    }
    if (a.y) P::store(static_cast<T*>(a.y) + (int64_t)at[u].row * a.y_stride + at[u].col, left, lane, y);
  }
}

bool on_16(const void* p, int64_t stride, int64_t rows, int size) {
  return !p || ((uintptr_t)p % 16 == 0 && (rows == 1 || stride * size % 16 == 0));
}

// Blocks side by side where every row lies on 16 bytes.  A thread takes four of
// them once there are enough to fill the device with that, else one.
template <class T, int KIND, bool BACKWARD>
cudaError_t run(const Activation8Args& a, int64_t rows, cudaStream_t s) {
  const bool side = on_16(a.x, a.x_stride, rows, sizeof(T)) && on_16(a.y, a.y_stride, rows, sizeof(T)) &&
                    on_16(a.dx, a.dx_stride, rows, sizeof(T));
  auto go = [&](auto each, auto side_by_side) {
    constexpr int kEach = decltype(each)::value;
    constexpr bool kSide = decltype(side_by_side)::value;
    constexpr uint32_t kPer = Places<T, kSide>::kGroups * kEach;
    const unsigned grid = (unsigned)((a.total + kPer - 1) / kPer);
    if constexpr (BACKWARD) activation8_backward_kernel<T, KIND, kSide, kEach><<<grid, kThreads, 0, s>>>(a);
    else activation8_kernel<T, KIND, kSide, kEach><<<grid, kThreads, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
  };
  const bool many = a.total >= 152u * 8 * 16 * 4;
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  if (side) return many ? go(Four(), std::true_type()) : go(One(), std::true_type());
  return many ? go(Four(), std::false_type()) : go(One(), std::false_type());
}

template <bool BACKWARD>
cudaError_t launch(int dtype, int kind, int64_t rows, Activation8Args a, cudaStream_t s) {
  // n / blocks = n magic >> shift for every n below 2^31: magic is 2^shift / blocks rounded up, too large by
  // less than blocks <= 2^(shift - 31) in 2^shift
  a.shift = 31;
  while ((1ll << (a.shift - 31)) < a.blocks) ++a.shift;
  a.magic = (uint32_t)(((1ull << a.shift) + a.blocks - 1) / a.blocks);
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    switch (kind) {
      case AR_ACT_IDENTITY: return run<T, AR_ACT_IDENTITY, BACKWARD>(a, rows, s);
      case AR_ACT_GELU_TANH: return run<T, AR_ACT_GELU_TANH, BACKWARD>(a, rows, s);
      default: return run<T, AR_ACT_GELU, BACKWARD>(a, rows, s);
    }
  });
}

}  // namespace

cudaError_t launch_activation8(int dtype, int kind, int64_t rows, const Activation8Args& a, cudaStream_t s) {
  return launch<false>(dtype, kind, rows, a, s);
}
cudaError_t launch_activation8_backward(int dtype, int kind, int64_t rows, const Activation8Args& a, cudaStream_t s) {
  return launch<true>(dtype, kind, rows, a, s);
}

}  // namespace ar
