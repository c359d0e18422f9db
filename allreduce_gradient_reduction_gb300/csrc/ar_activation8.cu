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
// neighbouring lanes.
#include <cuda_runtime.h>

#include <algorithm>

#include "ar_ops.cuh"

namespace ar {
namespace {

constexpr int kBlock = kActivation8Block;
constexpr int kThreads = 256;
constexpr uint32_t kLeastBits = 0x03800000u;  // 2^-120: blocks below it are zeros
constexpr uint32_t kInfinityBits = 0x7F800000u;

__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// gelu(x) = x s with s = 1 / (1 + e^-u), u = sqrt(8 / pi) (x + 0.044715 x^3):
// (1 + tanh(u / 2)) / 2 without its cancellation at negative x.
constexpr float kU1 = 1.5957691216057308f, kU3 = kU1 * 0.044715f, kLog2e = 1.4426950408889634f;

// The normal distribution's integral at -|x|, and e^(-x^2 / 2).  erfc(y)
// e^(y^2) = t Q(t) with t = 1 / (1 + y / 2); Q of degree 8 was fitted by
// weighted least squares for the least relative error, 4.4e-8, over y <= 14.7.
__device__ __forceinline__ float normal_tail(float x, float& bell) {
  const float t = reciprocal(fmaf(fabsf(x), 0.35355339059327379f, 1.f));
  bell = exp2_approx(x * x * -0.72134752044448169f);
  float q = -0.0593869729f;
  q = fmaf(q, t, 0.286126333f);
  q = fmaf(q, t, -0.490410976f);
  q = fmaf(q, t, 0.28173817f);
  q = fmaf(q, t, -0.0291516083f);
  q = fmaf(q, t, 0.203753693f);
  q = fmaf(q, t, 0.242834857f);
  q = fmaf(q, t, 0.282412128f);
  q = fmaf(q, t, 0.28208433f);
  return 0.5f * bell * t * q;
}

template <int KIND>
__device__ __forceinline__ float activation(float x) {
  if constexpr (KIND == AR_ACT_GELU_TANH) {
    const float u = x * fmaf(kU3 * kLog2e, x * x, kU1 * kLog2e);
    return x * reciprocal(1.f + exp2_approx(-u));
  } else if constexpr (KIND == AR_ACT_GELU) {
    float bell;
    const float tail = normal_tail(x, bell);
    return x * (x < 0.f ? tail : 1.f - tail);
  } else {
    return x;
  }
}

// The activation and its slope.  Beyond 10 the slope is that at 10, within
// 2^-120 of 0 or 1, and so is the activation below -10: what follows would
// multiply an infinity by zero.
template <int KIND>
__device__ __forceinline__ void activation_and_slope(float x, float& y, float& slope) {
  if constexpr (KIND == AR_ACT_GELU_TANH) {
    const float c = fabsf(x) > 10.f ? copysignf(10.f, x) : x;
    const float sq = c * c;
    const float e = exp2_approx(-c * fmaf(kU3 * kLog2e, sq, kU1 * kLog2e));
    const float s = reciprocal(1.f + e);
    y = (x < 0.f ? c : x) * s;
    slope = fmaf(c * s * (e * s), fmaf(3.f * kU3, sq, kU1), s);
  } else if constexpr (KIND == AR_ACT_GELU) {
    const float c = fabsf(x) > 18.f ? copysignf(18.f, x) : x;  // e^-162 = 0
    float bell;
    const float tail = normal_tail(c, bell), all = c < 0.f ? tail : 1.f - tail;
    y = x * all;
    slope = fmaf(c * 0.3989422804014327f, bell, all);
  } else {
    y = x;
    slope = 1.f;
  }
}

// Which elements of a block a lane has.  Side by side: 16 lanes to a block,
// eight elements each.  Apart: a warp to a block, every 32nd element.
template <bool SIDE_BY_SIDE>
struct Places {
  static constexpr int kLanes = SIDE_BY_SIDE ? 16 : 32;
  static constexpr int kEach = kBlock / kLanes;
  static constexpr int kGroups = kThreads / kLanes;  // blocks at a time
  static __device__ __forceinline__ int at(int lane, int i) { return SIDE_BY_SIDE ? lane * kEach + i : lane + 32 * i; }
};

// A lane's elements of the block that begins at `row`[c0], `left` of whose
// elements there are; zeros past them.
template <class T, bool SIDE_BY_SIDE>
__device__ __forceinline__ void load_elements(const T* from, int left, int lane, float (&f)[Places<SIDE_BY_SIDE>::kEach]) {
  using P = Places<SIDE_BY_SIDE>;
  if constexpr (SIDE_BY_SIDE) {
    constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
    for (int h = 0; h < P::kEach; h += kPer) {
      const Pack<T, kPer> p = load_pack<T, kPer>(from, P::at(lane, h), left);
#pragma unroll
      for (int i = 0; i < kPer; ++i) f[h + i] = Conv<T>::up(p.v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < P::kEach; ++i) f[i] = P::at(lane, i) < left ? Conv<T>::up(from[P::at(lane, i)]) : 0.f;
  }
}
template <class T, bool SIDE_BY_SIDE>
__device__ __forceinline__ void store_elements(T* to, int left, int lane, const float (&f)[Places<SIDE_BY_SIDE>::kEach]) {
  using P = Places<SIDE_BY_SIDE>;
  if constexpr (SIDE_BY_SIDE) {
    constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
    for (int h = 0; h < P::kEach; h += kPer) {
      Pack<T, kPer> p;
#pragma unroll
      for (int i = 0; i < kPer; ++i) p.v[i] = Conv<T>::down(f[h + i]);
      store_pack<T, kPer>(to, P::at(lane, h), left, p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < P::kEach; ++i)
      if (P::at(lane, i) < left) to[P::at(lane, i)] = Conv<T>::down(f[i]);
  }
}

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
  using P = Places<SIDE_BY_SIDE>;
  const int lane = threadIdx.x % P::kLanes, group = threadIdx.x / P::kLanes;
  const uint32_t first = (blockIdx.x * EACH) * P::kGroups + group;
  const T* x = static_cast<const T*>(a.x);
  float f[EACH][P::kEach];
  Place at[EACH];
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const uint32_t n = first + u * P::kGroups;
    at[u] = place_of(a, n);
    // no block n: nothing of the row is left
    load_elements<T, SIDE_BY_SIDE>(x + (int64_t)at[u].row * a.x_stride + at[u].col, n < a.total ? a.cols - at[u].col : 0,
                                   lane, f[u]);
  }
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const uint32_t n = first + u * P::kGroups;
    // sizes are compared as bits: a NaN is above all
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < P::kEach; ++i) most = max(most, __float_as_uint(f[u][i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int m = P::kLanes / 2; m; m >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));
    if (n >= a.total) continue;
    const bool some = most >= kLeastBits && most < kInfinityBits;
    const float m = __uint_as_float(most);
    const float by = some ? __fdiv_rn(127.f, m) : 0.f;
    if (lane == 0) a.scales_out[n] = some ? __fdiv_rn(m, 127.f) : most >= kInfinityBits ? __uint_as_float(0x7FC00000u) : 0.f;
    // adding 1.5 * 2^23 leaves the nearest whole number in the low bits
    uint32_t code[P::kEach];
#pragma unroll
    for (int i = 0; i < P::kEach; ++i)
      code[i] = some ? __float_as_uint(__fadd_rn(__fmul_rn(f[u][i], by), 12582912.f)) : 0;
    int8_t* to = a.codes_out + (int64_t)n * kBlock;
    if constexpr (SIDE_BY_SIDE) {
      auto four = [&](int i) {
        return __byte_perm(__byte_perm(code[i], code[i + 1], 0x0040), __byte_perm(code[i + 2], code[i + 3], 0x0040), 0x5410);
      };
      *reinterpret_cast<uint2*>(to + lane * 8) = make_uint2(four(0), four(4));
    } else {
#pragma unroll
      for (int i = 0; i < P::kEach; ++i) to[P::at(lane, i)] = (int8_t)code[i];
    }
    if (a.y) {
#pragma unroll
      for (int i = 0; i < P::kEach; ++i) f[u][i] = activation<KIND>(f[u][i]);
      store_elements<T, SIDE_BY_SIDE>(static_cast<T*>(a.y) + (int64_t)at[u].row * a.y_stride + at[u].col,
                                      a.cols - at[u].col, lane, f[u]);
    }
  }
}

template <class T, int KIND, bool SIDE_BY_SIDE, int EACH>
__global__ void __launch_bounds__(kThreads) activation8_backward_kernel(const __grid_constant__ Activation8Args a) {
  using P = Places<SIDE_BY_SIDE>;
  const int lane = threadIdx.x % P::kLanes, group = threadIdx.x / P::kLanes;
  const uint32_t first = (blockIdx.x * EACH) * P::kGroups + group;
  const T* dy = static_cast<const T*>(a.x);
  float d[EACH][P::kEach], scale[EACH];
  uint32_t codes[EACH][SIDE_BY_SIDE ? 2 : P::kEach];
  Place at[EACH];
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const uint32_t n = first + u * P::kGroups;
    if (n >= a.total) break;
    at[u] = place_of(a, n);
    const int8_t* from = a.codes + (int64_t)n * kBlock;
    if constexpr (SIDE_BY_SIDE) {
      const uint2 c = *reinterpret_cast<const uint2*>(from + lane * 8);
      codes[u][0] = c.x;
      codes[u][1] = c.y;
    } else {
#pragma unroll
      for (int i = 0; i < P::kEach; ++i) codes[u][i] = (uint32_t)(int32_t)from[P::at(lane, i)];
    }
    scale[u] = a.scales[n];
    if (a.dx)
      load_elements<T, SIDE_BY_SIDE>(dy + (int64_t)at[u].row * a.x_stride + at[u].col, a.cols - at[u].col, lane, d[u]);
  }
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const uint32_t n = first + u * P::kGroups;
    if (n >= a.total) break;
    float y[P::kEach];
#pragma unroll
    for (int i = 0; i < P::kEach; ++i) {
      int code;
      if constexpr (SIDE_BY_SIDE) code = (int)(codes[u][i / 4] << (24 - 8 * (i % 4))) >> 24;
      else code = (int)codes[u][i];
      float slope;
      activation_and_slope<KIND>(scale[u] * (float)code, y[i], slope);
      d[u][i] *= slope;
    }
    const int left = a.cols - at[u].col;
    if (a.dx)
      store_elements<T, SIDE_BY_SIDE>(static_cast<T*>(a.dx) + (int64_t)at[u].row * a.dx_stride + at[u].col, left, lane, d[u]);
    if (a.y)
      store_elements<T, SIDE_BY_SIDE>(static_cast<T*>(a.y) + (int64_t)at[u].row * a.y_stride + at[u].col, left, lane, y);
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
    constexpr uint32_t kPer = Places<kSide>::kGroups * kEach;
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
