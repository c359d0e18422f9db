// Layer norm over the last axis, forward and backward.
//
//   mean = sum(x) / C, rstd = (sum((x - mean)^2) / C + eps)^-1/2
//   y  = (x - mean) rstd w + b
//   with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g)/C - xh sum(g xh)/C)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both directions are bound by HBM: a row is read once, held in registers, and
// everything about it is computed from there in binary32.  The variance is
// taken about the row's own mean (a second pass over the registers), not as a
// difference of two large sums.
//
// A row belongs to a group of whole warps; each warp owns a run of 32 NV
// vectors of it, its lanes every 32nd of them, so accesses are contiguous and
// a thread's columns are the same in every row.  That lets the backward kernel
// keep its columns' share of dw and db in registers while its group walks
// over rows; the groups' sums are joined in a fixed order, in the block and
// then in a second kernel, so the result does not depend on timing.
//
// Measured (device time from HBM, share of the measured copy bandwidth): forward
// 16384 rows of bf16 with f32 parameters, 512 columns 10.4 us, 48%; 768 16.1 us,
// 47%; 1024 19.2 us, 53%; 2048 29.7 us, 68%; 4096 55.6 us, 72%; 5120 60.0 us,
// 84% (narrower rows wait for their two reductions, two or three rows to a
// multiprocessor at a time); 8192 x 768 f32 12.8 us, 59% (8.1 where the rows are
// in L2).  Backward 32768 x 4096 bf16 with f32 parameters 142 us, 85% (with its
// second kernel); 8192 x 768 f32 20.0 us, 57% (15.4 from L2); 8192 x 16384 bf16
// 285 us, 42% (64 registers a thread, which spill).  Rows of odd width are read
// and written element by element: forward 16384 x 5121 bf16 91 us, 56%, no unit
// above 39%: few warps, each between two barriers; backward 8192 x 16383 f16 329
// us, 37%.
#include "ar_ops.cuh"

#include <algorithm>
#include <type_traits>

#include "ar_device.cuh"

namespace ar {
namespace {

constexpr int kGroups = 16;  // most groups in one block (named barriers 1..15 and __syncthreads' own)

// Sum of v over the block's group of threads.  `slot` alternates between two
// halves of the group's scratch, so that one barrier a call is enough: a
// thread that is still reading a half has not passed the next call's barrier.
__device__ __forceinline__ float group_sum(float v, float (*scratch)[32], int slot) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  float* s = scratch[slot];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s[w] = v;
  if (blockDim.y == 1) __syncthreads();
  else named_barrier(1 + threadIdx.y, blockDim.x);
  return warp_sum(lane < warps ? s[lane] : 0.f);
}

// Rows too wide for a ring (see below): up to 32 elements in each of up to
// 1024 threads, one row to a block.
template <class T, class P, int VW, int NV>
__global__ void __launch_bounds__(1024) layer_norm_kernel(const LayerNormArgs a) {
  __shared__ float scratch[2][32];
  const int64_t row = blockIdx.x;
  const int cols = (int)a.cols;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
  const P* weight = static_cast<const P*>(a.weight);
  const P* bias = static_cast<const P*>(a.bias);
  const int g = blockDim.x, t = threadIdx.x;
  const float inv = 1.0f / (float)cols;

  Pack<T, VW> xr[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) xr[k] = load_pack<T, VW>(x, (k * g + t) * VW, cols);
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VW; ++i) sum += Conv<T>::up(xr[k].v[i]);
  const float mean = group_sum(sum, scratch, 0) * inv;
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * g + t) * VW;
#pragma unroll
    for (int i = 0; i < VW; ++i) {
      const float d = Conv<T>::up(xr[k].v[i]) - mean;
      if (c + i < cols) sq = fmaf(d, d, sq);
    }
  }
  const float rstd = rsqrtf(group_sum(sq, scratch, 1) * inv + a.eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * g + t) * VW;
    if (c >= cols) break;
    const Pack<P, VW> w = load_pack<P, VW>(weight, c, cols);
    const Pack<P, VW> b = bias ? load_pack<P, VW>(bias, c, cols) : zero_pack<P, VW>();
    Pack<T, VW> o;
#pragma unroll
    for (int i = 0; i < VW; ++i)
      o.v[i] = Conv<T>::down(fmaf((Conv<T>::up(xr[k].v[i]) - mean) * rstd, Conv<P>::up(w.v[i]), Conv<P>::up(b.v[i])));
    store_pack<T, VW>(y, c, cols, o);
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// Rows of any width: three passes, the second and third of which find the row
// in the caches.
template <class T, class P>
__global__ void __launch_bounds__(1024) layer_norm_wide_kernel(const LayerNormArgs a) {
  __shared__ float scratch[2][32];
  const int64_t row = blockIdx.x, cols = a.cols;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
  const P* weight = static_cast<const P*>(a.weight);
  const P* bias = static_cast<const P*>(a.bias);
  float sum = 0.f, sq = 0.f;
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) sum += Conv<T>::up(x[c]);
  const float mean = group_sum(sum, scratch, 0) / (float)cols;
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) {
    const float d = Conv<T>::up(x[c]) - mean;
    sq = fmaf(d, d, sq);
  }
  const float rstd = rsqrtf(group_sum(sq, scratch, 1) / (float)cols + a.eps);
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x)
    y[c] = Conv<T>::down(fmaf((Conv<T>::up(x[c]) - mean) * rstd, Conv<P>::up(weight[c]),
                              bias ? Conv<P>::up(bias[c]) : 0.f));
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// A block's share of dw and db: its groups' sums added in order (through
// `joined`, two floats for each of a group's columns) and written as row
// blockIdx.x of the partial sums.  column(k): the first of the VW columns that
// the thread's k-th sums stand for.
template <int VW, int NV, class C>
__device__ __forceinline__ void join_params(const float (&dw)[NV][VW], const float (&db)[NV][VW], float* joined,
                                            float* partial, int cols, C column) {
  const int width = blockDim.x * NV * VW;
  float* out = partial + (int64_t)blockIdx.x * 2 * cols;
  __syncthreads();
  for (int y = 0; y + 1 < (int)blockDim.y; ++y) {
    if ((int)threadIdx.y == y) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          const int c = column(k) + i;
          joined[c] = dw[k][i] + (y ? joined[c] : 0.f);
          joined[width + c] = db[k][i] + (y ? joined[width + c] : 0.f);
        }
    }
    __syncthreads();
  }
  if (threadIdx.y == blockDim.y - 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const int c = column(k) + i;
        if (c < cols) {
          out[c] = dw[k][i] + (blockDim.y > 1 ? joined[c] : 0.f);
          out[cols + c] = db[k][i] + (blockDim.y > 1 ? joined[width + c] : 0.f);
        }
      }
  }
}

// f32 rows too wide for a ring: a block walks over the rows with a stride of
// all blocks, up to 16 columns in each of up to 1024 threads.
template <class T, class P, int VW, int NV>
__global__ void __launch_bounds__(1024) layer_norm_backward_kernel(const LayerNormBackwardArgs a) {
  __shared__ float scratch[2][2][32];
  const int cols = (int)a.cols, g = blockDim.x, t = threadIdx.x;
  const P* weight = static_cast<const P*>(a.weight);
  const float inv = 1.0f / (float)cols;

  float dw[NV][VW], db[NV][VW];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VW; ++i) dw[k][i] = db[k][i] = 0.f;

  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* d = static_cast<const T*>(a.dy) + row * a.dy_stride;
    Pack<T, VW> xr[NV], dr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      xr[k] = load_pack<T, VW>(x, (k * g + t) * VW, cols);
      dr[k] = load_pack<T, VW>(d, (k * g + t) * VW, cols);
    }
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const Pack<P, VW> w = load_pack<P, VW>(weight, (k * g + t) * VW, cols);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float dy = Conv<T>::up(dr[k].v[i]);
        const float xh = (Conv<T>::up(xr[k].v[i]) - mean) * rstd;
        const float gw = dy * Conv<P>::up(w.v[i]);
        dw[k][i] = fmaf(dy, xh, dw[k][i]);
        db[k][i] += dy;
        s1 += gw;
        s2 = fmaf(gw, xh, s2);
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    // by turns, so that one barrier a row is enough
    if ((t & 31) == 0) scratch[turn][0][t >> 5] = s1, scratch[turn][1][t >> 5] = s2;
    __syncthreads();
    s1 = warp_sum((t & 31) < g >> 5 ? scratch[turn][0][t & 31] : 0.f) * inv;
    s2 = warp_sum((t & 31) < g >> 5 ? scratch[turn][1][t & 31] : 0.f) * inv;
    T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * g + t) * VW;
      if (c >= cols) break;
      const Pack<P, VW> w = load_pack<P, VW>(weight, c, cols);
      Pack<T, VW> o;
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float xh = (Conv<T>::up(xr[k].v[i]) - mean) * rstd;
        const float gw = Conv<T>::up(dr[k].v[i]) * Conv<P>::up(w.v[i]);
        o.v[i] = Conv<T>::down(rstd * (gw - s1 - xh * s2));
      }
      store_pack<T, VW>(dx, c, cols, o);
    }
  }
  join_params<VW, NV>(dw, db, nullptr, a.partial, cols, [&](int k) { return (k * g + t) * VW; });
}

// ---- rows through shared memory -----------------------------------------------------
//
// Each group keeps a ring of rows in shared memory, filled by bulk copies that
// its first thread issues ahead, so the bytes in flight do not depend on
// registers or occupancy (16384 x 5120 bf16 forward: 116 us with loads into
// registers, 61 us so).  A copy takes
// the aligned 16-byte words that hold a row.

__device__ __forceinline__ void group_barrier() {
  if (blockDim.x == 32) __syncwarp();
  else named_barrier(1 + threadIdx.y, blockDim.x);
}

// Pairs of a thread's parameters, from the caches: keeping them in registers
// would cost more in threads than it saves in loads.
template <class P, int N>
__device__ __forceinline__ void param_pairs(const P* p, Two (&out)[N]) {
  if constexpr (sizeof(P) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 2 * i);
      out[i] = Pairs<float>::get(v, 0);
      out[i + 1] = Pairs<float>::get(v, 1);
    }
  } else {
    uint4 v;
    if constexpr (N == 4) {
      v = *reinterpret_cast<const uint4*>(p);
    } else {
      const uint2 h = *reinterpret_cast<const uint2*>(p);
      v = make_uint4(h.x, h.y, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = Pairs<P>::get(v, i);
  }
}

constexpr int kRing = 4;  // most rows of a group in flight

__device__ __forceinline__ void open_ring(uint64_t* full, int* gave_up) {
  if (threadIdx.x == 0) {
    *gave_up = 0;
    for (int i = 0; i < kRing; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_at(full + i)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// Sums of two values over the group, through one of two halves of its scratch
// by turns: one barrier a call.
template <int WARPS>
__device__ __forceinline__ float2 group_sum2(float2 v, float2 (*scratch)[WARPS], int turn) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  const int warps = blockDim.x >> 5;
  if (warps == 1) {
    __syncwarp();
    return v;
  }
  float2* s = scratch[turn];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s[w] = v;
  group_barrier();
  v = lane < warps ? s[lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// Registers of the forward kernel, which holds a thread's columns widened.
__host__ __device__ constexpr int forward_registers(int columns) { return columns <= 16 ? 64 : columns <= 24 ? 80 : 96; }
// Registers of the backward kernel: two sums for each of a thread's columns,
// and xh and dy w of the current row.
__host__ __device__ constexpr int backward_registers(int columns) { return columns <= 8 ? 72 : 120; }

// slot: bytes of one row's place in shared memory; stages: rows in flight.
// Every row of every operand and the parameters begin on a vector boundary
// and rows are whole vectors.
template <class T, class P, int NV, bool KEEP>
__global__ void __maxnreg__(KEEP ? 88 : forward_registers(NV * (16 / sizeof(T))))
    layer_norm_ring_kernel(const LayerNormArgs a, int slot, int stages) {
  constexpr int VW = 16 / sizeof(T), N = Pairs<T>::N;
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ float scratch[kGroups][2][32];
  __shared__ __align__(8) uint64_t filled[kGroups][kRing];
  __shared__ int gave_up;
  const int cols = (int)a.cols, g = blockDim.x, t = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const T* x = static_cast<const T*>(a.x);
  // a warp has 32 NV vectors in a row, its lanes every 32nd of them
  const int vecs = cols / VW, v0 = (t >> 5) * 32 * NV + (t & 31);
  const bool full = ((t >> 5) + 1) * 32 * NV <= vecs;
  const P* weight = static_cast<const P*>(a.weight) + v0 * VW;
  const P* bias = a.bias ? static_cast<const P*>(a.bias) + v0 * VW : nullptr;
  uint8_t* mine = rows + (int64_t)threadIdx.y * stages * slot;
  uint64_t* bars = filled[threadIdx.y];
  const float inv = 1.0f / (float)cols;
  auto issue = [&](int64_t row, int stage) {
    const T* from = x + row * a.x_stride;
    const uint32_t bar = smem_at(bars + stage);
    ring_expect(bar, covering(from, cols * (int)sizeof(T)));
    ring_copy(smem_at(mine + stage * slot), from, cols * (int)sizeof(T), bar);
  };
  open_ring(bars, &gave_up);
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t == 0)
    for (int i = 0; i < stages && row + i * step < a.rows; ++i) issue(row + i * step, i);

  Two kept_w[KEEP ? NV : 1][N], kept_b[KEEP ? NV : 1][N];
  if constexpr (KEEP) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < N; ++i) kept_w[k][i] = kept_b[k][i] = two(0.f, 0.f);
      if (v0 + k * 32 < vecs) {
        param_pairs<P, N>(weight + k * 32 * VW, kept_w[k]);
        if (bias) param_pairs<P, N>(bias + k * 32 * VW, kept_b[k]);
      }
    }
  }
  int stage = 0, parity = 0;
  for (; row < a.rows; row += step) {
    const bool came = ring_wait(smem_at(bars + stage), parity, &gave_up);
    const uint8_t* from = mine + stage * slot + v0 * 16;
    Two e[NV][N];  // the elements, then their distance from the mean
    Two acc[2] = {two(0.f, 0.f), two(0.f, 0.f)};
    auto take = [&](int k, const uint4& raw) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        e[k][i] = Pairs<T>::get(raw, i);
        acc[i & 1] = add2(acc[i & 1], e[k][i]);
      }
    };
    if (full) {
#pragma unroll
      for (int k = 0; k < NV; ++k) take(k, *reinterpret_cast<const uint4*>(from + k * 512));
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        take(k, v0 + k * 32 < vecs ? *reinterpret_cast<const uint4*>(from + k * 512) : make_uint4(0, 0, 0, 0));
    }
    float lo, hi;
    split(add2(acc[0], acc[1]), lo, hi);
    const float mean = group_sum(lo + hi, scratch[threadIdx.y], 0) * inv;
    if (g == 32) __syncwarp();
    if (t == 0 && came && row + stages * step < a.rows) issue(row + stages * step, stage);  // the group has read the slot
    const Two minus = two(-mean, -mean);
    acc[0] = acc[1] = two(0.f, 0.f);
    auto square = [&](int k) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        e[k][i] = add2(e[k][i], minus);
        acc[i & 1] = fma2(e[k][i], e[k][i], acc[i & 1]);
      }
    };
    if (full) {
#pragma unroll
      for (int k = 0; k < NV; ++k) square(k);
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (v0 + k * 32 < vecs) square(k);
    }
    split(add2(acc[0], acc[1]), lo, hi);
    const float rstd = rsqrtf(group_sum(lo + hi, scratch[threadIdx.y], 1) * inv + a.eps);
    const Two scale = two(rstd, rstd);
    T* y = static_cast<T*>(a.y) + row * a.y_stride + v0 * VW;
    auto put = [&](int k) {
      Two w[N], b[N];
      uint4 out;
      if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < N; ++i) Pairs<T>::set(out, i, fma2(mul2(e[k][i], scale), kept_w[k][i], kept_b[k][i]));
        *reinterpret_cast<uint4*>(y + k * 32 * VW) = out;
        return;
      }
      param_pairs<P, N>(weight + k * 32 * VW, w);
      if (bias) param_pairs<P, N>(bias + k * 32 * VW, b);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const Two xh = mul2(e[k][i], scale);
        Pairs<T>::set(out, i, bias ? fma2(xh, w[i], b[i]) : mul2(xh, w[i]));
      }
      *reinterpret_cast<uint4*>(y + k * 32 * VW) = out;
    };
    if (full) {
#pragma unroll
      for (int k = 0; k < NV; ++k) put(k);
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (v0 + k * 32 < vecs) put(k);
    }
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (++stage == stages) stage = 0, parity ^= 1;
  }
}

// WIDE: a group of more than 512 threads.  They have 64 registers each, so xh
// and dy w are made again from shared memory after the sums, and a row's place
// is filled again only after that.
template <class T, class P, int NV, bool WIDE>
__global__ void __maxnreg__(WIDE ? 64 : backward_registers(NV * (16 / sizeof(T))))
    layer_norm_backward_ring_kernel(const LayerNormBackwardArgs a, int slot, int stages) {
  constexpr int VW = 16 / sizeof(T), N = Pairs<T>::N;
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ float2 scratch[WIDE ? 1 : kGroups][2][WIDE ? 32 : 16];
  __shared__ __align__(8) uint64_t filled[kGroups][kRing];
  __shared__ int gave_up;
  const int cols = (int)a.cols, t = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const int vecs = cols / VW, v0 = (t >> 5) * 32 * NV + (t & 31);
  const bool full = ((t >> 5) + 1) * 32 * NV <= vecs;
  const P* weight = static_cast<const P*>(a.weight) + v0 * VW;
  uint8_t* mine = rows + (int64_t)threadIdx.y * 2 * stages * slot;
  uint64_t* bars = filled[threadIdx.y];
  const float inv = 1.0f / (float)cols;
  auto issue = [&](int64_t row, int stage) {
    const int bytes = cols * (int)sizeof(T);
    const T *fx = x + row * a.x_stride, *fd = dy + row * a.dy_stride;
    const uint32_t bar = smem_at(bars + stage), to = smem_at(mine + stage * 2 * slot);
    ring_expect(bar, covering(fx, bytes) + covering(fd, bytes));
    ring_copy(to, fx, bytes, bar);
    ring_copy(to + slot, fd, bytes, bar);
  };
  open_ring(bars, &gave_up);
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t == 0)
    for (int i = 0; i < stages && row + i * step < a.rows; ++i) issue(row + i * step, i);

  Two dw[NV][N], db[NV][N];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[k][i] = db[k][i] = two(0.f, 0.f);
  float mean = 0.f, rstd = 0.f;
  if (row < a.rows) mean = a.mean[row], rstd = a.rstd[row];
  int stage = 0, parity = 0;
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    float mean_n = 0.f, rstd_n = 0.f;
    if (row + step < a.rows) mean_n = a.mean[row + step], rstd_n = a.rstd[row + step];
    const bool came = ring_wait(smem_at(bars + stage), parity, &gave_up);
    const Two minus = two(-mean, -mean), scale = two(rstd, rstd);
    const uint8_t* from = mine + stage * 2 * slot + v0 * 16;
    Two xh[WIDE ? 1 : NV][N], gw[WIDE ? 1 : NV][N];
    Two s1 = two(0.f, 0.f), s2 = two(0.f, 0.f);
    auto take = [&](int k, bool again) {
      const int at = WIDE ? 0 : k;
      const uint4 xr = *reinterpret_cast<const uint4*>(from + k * 512);
      const uint4 dr = *reinterpret_cast<const uint4*>(from + slot + k * 512);
      Two w[N];
      param_pairs<P, N>(weight + k * 32 * VW, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const Two d = Pairs<T>::get(dr, i);
        xh[at][i] = mul2(add2(Pairs<T>::get(xr, i), minus), scale);
        gw[at][i] = mul2(d, w[i]);
        if (again) continue;
        dw[k][i] = fma2(d, xh[at][i], dw[k][i]);
        db[k][i] = add2(db[k][i], d);
        s1 = add2(s1, gw[at][i]);
        s2 = fma2(gw[at][i], xh[at][i], s2);
      }
    };
    if (full) {
#pragma unroll
      for (int k = 0; k < NV; ++k) take(k, false);
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (v0 + k * 32 < vecs) take(k, false);
    }
    float a1, b1, a2, b2;
    split(s1, a1, b1);
    split(s2, a2, b2);
    const float2 s = group_sum2(make_float2(a1 + b1, a2 + b2), scratch[threadIdx.y], turn);
    if (!WIDE && t == 0 && came && row + stages * step < a.rows) issue(row + stages * step, stage);  // the group has read the slot
    // dx = rstd gw - rstd s1 / C - xh rstd s2 / C
    const float m1 = -rstd * (s.x * inv), m2 = -rstd * (s.y * inv);
    const Two m1s = two(m1, m1), m2s = two(m2, m2);
    T* dx = static_cast<T*>(a.dx) + row * a.dx_stride + v0 * VW;
    auto put = [&](int k) {
      const int at = WIDE ? 0 : k;
      if (WIDE) take(k, true);
      uint4 out;
#pragma unroll
      for (int i = 0; i < N; ++i) Pairs<T>::set(out, i, fma2(xh[at][i], m2s, fma2(gw[at][i], scale, m1s)));
      *reinterpret_cast<uint4*>(dx + k * 32 * VW) = out;
    };
    if (full) {
#pragma unroll
      for (int k = 0; k < NV; ++k) put(k);
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (v0 + k * 32 < vecs) put(k);
    }
    if (WIDE) {
      group_barrier();
      if (t == 0 && came && row + stages * step < a.rows) issue(row + stages * step, stage);
    }
    mean = mean_n;
    rstd = rstd_n;
    if (++stage == stages) stage = 0, parity ^= 1;
  }
  float dw1[NV][VW], db1[NV][VW];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      split(dw[k][i], dw1[k][2 * i], dw1[k][2 * i + 1]);
      split(db[k][i], db1[k][2 * i], db1[k][2 * i + 1]);
    }
  join_params<VW, NV>(dw1, db1, reinterpret_cast<float*>(rows), a.partial, cols,
                      [&](int k) { return (v0 + k * 32) * VW; });
}

// Rows that are not whole vectors, or begin anywhere: a warp has 32 NE
// elements in a row, its lanes every 32nd of them, so its accesses are
// contiguous whatever the addresses; a thread's parameters stay in its
// registers.  (Vectors put right by shifts, on their way in and, through
// shared memory, out again, took 28 instructions an element and 125 us for
// 16384 x 5121 bf16 forward.)  Elements 2 i and 2 i + 1 of a thread go through
// the arithmetic as a pair.
template <class P, int N>
__device__ __forceinline__ void strided_params(const P* p, int c0, int cols, Two (&out)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = c0 + i * 64;
    out[i] = two(p && c < cols ? Conv<P>::up(p[c]) : 0.f, p && c + 32 < cols ? Conv<P>::up(p[c + 32]) : 0.f);
  }
}

// Pair i of the elements from `row` on; left: how many there are (FULL: enough).
template <bool FULL, class T>
__device__ __forceinline__ Two strided_pair(const T* row, int i, int left) {
  if constexpr (FULL) return two(Conv<T>::up(row[i * 64]), Conv<T>::up(row[i * 64 + 32]));
  else
    return two(i * 64 < left ? Conv<T>::up(row[i * 64]) : 0.f, i * 64 + 32 < left ? Conv<T>::up(row[i * 64 + 32]) : 0.f);
}
template <bool FULL, class T>
__device__ __forceinline__ void strided_store(T* row, int i, int left, Two v) {
  float lo, hi;
  split(v, lo, hi);
  if constexpr (sizeof(T) == 2) {
    const uint32_t both = pack2<T>(lo, hi);
    uint16_t* to = reinterpret_cast<uint16_t*>(row);
    if (FULL || i * 64 < left) to[i * 64] = (uint16_t)both;
    if (FULL || i * 64 + 32 < left) to[i * 64 + 32] = (uint16_t)(both >> 16);
  } else {
    if (FULL || i * 64 < left) row[i * 64] = lo;
    if (FULL || i * 64 + 32 < left) row[i * 64 + 32] = hi;
  }
}

__host__ __device__ constexpr int strided_registers(int columns) { return columns <= 8 ? 56 : columns <= 16 ? 80 : 128; }

template <class T, class P, int NE>
__global__ void __maxnreg__(strided_registers(NE))
    layer_norm_strided_kernel(const LayerNormArgs a, int slot, int stages) {
  constexpr int N = NE / 2;
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ float scratch[kGroups][2][32];
  __shared__ __align__(8) uint64_t filled[kGroups][kRing];
  __shared__ int gave_up;
  const int cols = (int)a.cols, g = blockDim.x, t = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const T* x = static_cast<const T*>(a.x);
  uint8_t* mine = rows + (int64_t)threadIdx.y * stages * slot;
  uint64_t* bars = filled[threadIdx.y];
  const float inv = 1.0f / (float)cols;
  auto issue = [&](int64_t row, int stage) {
    const T* from = x + row * a.x_stride;
    const uint32_t bar = smem_at(bars + stage);
    ring_expect(bar, covering(from, cols * (int)sizeof(T)));
    ring_copy(smem_at(mine + stage * slot), from, cols * (int)sizeof(T), bar);
  };
  open_ring(bars, &gave_up);
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t == 0)
    for (int i = 0; i < stages && row + i * step < a.rows; ++i) issue(row + i * step, i);
  const int c0 = (t >> 5) * 32 * NE + (t & 31), left = cols - c0;
  const bool full = ((t >> 5) + 1) * 32 * NE <= cols;
  Two w[N], b[N];
  strided_params<P, N>(static_cast<const P*>(a.weight), c0, cols, w);
  strided_params<P, N>(static_cast<const P*>(a.bias), c0, cols, b);

  int stage = 0, parity = 0;
  for (; row < a.rows; row += step) {
    const bool came = ring_wait(smem_at(bars + stage), parity, &gave_up);
    const T* from = reinterpret_cast<const T*>(mine + stage * slot + ((uintptr_t)(x + row * a.x_stride) & 15)) + c0;
    Two e[N], acc[2] = {two(0.f, 0.f), two(0.f, 0.f)};
    if (full) {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = strided_pair<true>(from, i, left);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = strided_pair<false>(from, i, left);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i & 1] = add2(acc[i & 1], e[i]);
    float lo, hi;
    split(add2(acc[0], acc[1]), lo, hi);
    const float mean = group_sum(lo + hi, scratch[threadIdx.y], 0) * inv;
    if (g == 32) __syncwarp();
    if (t == 0 && came && row + stages * step < a.rows) issue(row + stages * step, stage);  // the group has read the slot
    const Two minus = two(-mean, -mean);
    acc[0] = acc[1] = two(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      e[i] = add2(e[i], minus);
      if (!full) {
        split(e[i], lo, hi);
        e[i] = two(i * 64 < left ? lo : 0.f, i * 64 + 32 < left ? hi : 0.f);
      }
      acc[i & 1] = fma2(e[i], e[i], acc[i & 1]);
    }
    split(add2(acc[0], acc[1]), lo, hi);
    const float rstd = rsqrtf(group_sum(lo + hi, scratch[threadIdx.y], 1) * inv + a.eps);
    const Two scale = two(rstd, rstd);
    T* y = static_cast<T*>(a.y) + row * a.y_stride + c0;
    if (full) {
#pragma unroll
      for (int i = 0; i < N; ++i) strided_store<true>(y, i, left, fma2(mul2(e[i], scale), w[i], b[i]));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) strided_store<false>(y, i, left, fma2(mul2(e[i], scale), w[i], b[i]));
    }
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (++stage == stages) stage = 0, parity ^= 1;
  }
}

template <class T, class P, int NE, bool WIDE>
__global__ void __maxnreg__(WIDE ? 64 : backward_registers(NE))
    layer_norm_backward_strided_kernel(const LayerNormBackwardArgs a, int slot, int stages) {
  constexpr int N = NE / 2;
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ float2 scratch[WIDE ? 1 : kGroups][2][WIDE ? 32 : 16];
  __shared__ __align__(8) uint64_t filled[kGroups][kRing];
  __shared__ int gave_up;
  const int cols = (int)a.cols, t = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  uint8_t* mine = rows + (int64_t)threadIdx.y * 2 * stages * slot;
  uint64_t* bars = filled[threadIdx.y];
  const float inv = 1.0f / (float)cols;
  auto issue = [&](int64_t row, int stage) {
    const int bytes = cols * (int)sizeof(T);
    const T *fx = x + row * a.x_stride, *fd = dy + row * a.dy_stride;
    const uint32_t bar = smem_at(bars + stage), to = smem_at(mine + stage * 2 * slot);
    ring_expect(bar, covering(fx, bytes) + covering(fd, bytes));
    ring_copy(to, fx, bytes, bar);
    ring_copy(to + slot, fd, bytes, bar);
  };
  open_ring(bars, &gave_up);
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t == 0)
    for (int i = 0; i < stages && row + i * step < a.rows; ++i) issue(row + i * step, i);
  const int c0 = (t >> 5) * 32 * NE + (t & 31), left = cols - c0;
  const bool full = ((t >> 5) + 1) * 32 * NE <= cols;
  const P* weight = static_cast<const P*>(a.weight);
  Two w[WIDE ? 1 : N], dw[N], db[N];
  if constexpr (!WIDE) strided_params<P, N>(weight, c0, cols, w);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = db[i] = two(0.f, 0.f);
  float mean = 0.f, rstd = 0.f;
  if (row < a.rows) mean = a.mean[row], rstd = a.rstd[row];
  int stage = 0, parity = 0;
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    float mean_n = 0.f, rstd_n = 0.f;
    if (row + step < a.rows) mean_n = a.mean[row + step], rstd_n = a.rstd[row + step];
    const bool came = ring_wait(smem_at(bars + stage), parity, &gave_up);
    const Two minus = two(-mean, -mean), scale = two(rstd, rstd);
    const uint8_t* from = mine + stage * 2 * slot;
    const T* xs = reinterpret_cast<const T*>(from + ((uintptr_t)(x + row * a.x_stride) & 15)) + c0;
    const T* ds = reinterpret_cast<const T*>(from + slot + ((uintptr_t)(dy + row * a.dy_stride) & 15)) + c0;
    Two xh[WIDE ? 1 : N], gw[WIDE ? 1 : N], s1 = two(0.f, 0.f), s2 = two(0.f, 0.f);
    auto take = [&](auto full_row, int i, bool again) {
      constexpr bool FULL = decltype(full_row)::value;
      const int at = WIDE ? 0 : i;
      // dy is 0 outside the row, so what stands for x there does not count
      const Two d = strided_pair<FULL>(ds, i, left);
      if constexpr (WIDE) w[0] = strided_pair<FULL>(weight + c0, i, left);
      xh[at] = mul2(add2(strided_pair<FULL>(xs, i, left), minus), scale);
      gw[at] = mul2(d, w[at]);
      if (again) return;
      dw[i] = fma2(d, xh[at], dw[i]);
      db[i] = add2(db[i], d);
      s1 = add2(s1, gw[at]);
      s2 = fma2(gw[at], xh[at], s2);
    };
    if (full) {
#pragma unroll
      for (int i = 0; i < N; ++i) take(std::true_type(), i, false);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) take(std::false_type(), i, false);
    }
    float a1, b1, a2, b2;
    split(s1, a1, b1);
    split(s2, a2, b2);
    const float2 s = group_sum2(make_float2(a1 + b1, a2 + b2), scratch[threadIdx.y], turn);
    if (!WIDE && t == 0 && came && row + stages * step < a.rows) issue(row + stages * step, stage);  // the group has read the slot
    const float m1 = -rstd * (s.x * inv), m2 = -rstd * (s.y * inv);
    const Two m1s = two(m1, m1), m2s = two(m2, m2);
    T* dx = static_cast<T*>(a.dx) + row * a.dx_stride + c0;
    auto put = [&](auto full_row, int i) {
      const int at = WIDE ? 0 : i;
      if (WIDE) take(full_row, i, true);
      strided_store<decltype(full_row)::value>(dx, i, left, fma2(xh[at], m2s, fma2(gw[at], scale, m1s)));
    };
    if (full) {
#pragma unroll
      for (int i = 0; i < N; ++i) put(std::true_type(), i);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) put(std::false_type(), i);
    }
    if (WIDE) {
      group_barrier();
      if (t == 0 && came && row + stages * step < a.rows) issue(row + stages * step, stage);
    }
    mean = mean_n;
    rstd = rstd_n;
    if (++stage == stages) stage = 0, parity ^= 1;
  }
  float dw1[NE][1], db1[NE][1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    split(dw[i], dw1[2 * i][0], dw1[2 * i + 1][0]);
    split(db[i], db1[2 * i][0], db1[2 * i + 1][0]);
  }
  join_params<1, NE>(dw1, db1, reinterpret_cast<float*>(rows), a.partial, cols, [&](int k) { return c0 + k * 32; });
}

// Rows of any width: dx in three passes over a row by one block.
template <class T, class P>
__global__ void __launch_bounds__(1024) layer_norm_backward_wide_kernel(const LayerNormBackwardArgs a) {
  __shared__ float scratch[2][32];
  const int64_t row = blockIdx.x, cols = a.cols;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
  T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
  const P* weight = static_cast<const P*>(a.weight);
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) {
    const float gw = Conv<T>::up(dy[c]) * Conv<P>::up(weight[c]);
    s1 += gw;
    s2 = fmaf(gw, (Conv<T>::up(x[c]) - mean) * rstd, s2);
  }
  s1 = group_sum(s1, scratch, 0) / (float)cols;
  s2 = group_sum(s2, scratch, 1) / (float)cols;
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) {
    const float gw = Conv<T>::up(dy[c]) * Conv<P>::up(weight[c]);
    const float xh = (Conv<T>::up(x[c]) - mean) * rstd;
    dx[c] = Conv<T>::down(rstd * (gw - s1 - xh * s2));
  }
}

// ... and its parameters' partial sums: block (i, j) takes 256 columns and
// every gridDim.y-th row.  Runs before the kernel above, which may write dx
// over dy or x.
template <class T>
__global__ void __launch_bounds__(256) layer_norm_params_wide_kernel(const LayerNormBackwardArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float dy = Conv<T>::up(static_cast<const T*>(a.dy)[row * a.dy_stride + c]);
    dw = fmaf(dy, (Conv<T>::up(static_cast<const T*>(a.x)[row * a.x_stride + c]) - a.mean[row]) * a.rstd[row], dw);
    db += dy;
  }
  float* out = a.partial + (int64_t)blockIdx.y * 2 * a.cols;
  out[c] = dw;
  out[a.cols + c] = db;
}

// Sums the blocks' partial rows in order: 32 columns and 32 slices of blocks
// to a block, the slices joined in shared memory.
template <class P>
__global__ void __launch_bounds__(1024) layer_norm_params_kernel(const float* partial, int blocks, int64_t cols,
                                                                 P* dweight, P* dbias) {
  __shared__ float part[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < 2 * cols) {
#pragma unroll 4
    for (int b = threadIdx.y; b < blocks; b += 32) s += partial[(int64_t)b * 2 * cols + c];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(part[threadIdx.x][threadIdx.y]);
  const int64_t o = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && o < 2 * cols) {
    if (o < cols) dweight[o] = Conv<P>::down(s);
    else if (dbias) dbias[o - cols] = Conv<P>::down(s);
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool rows_aligned16(const void* p, int64_t stride, int64_t rows, int es) {
  return aligned16(p) && (rows <= 1 || stride * es % 16 == 0);
}

// How a row of `vecs` vectors is dealt out: `nv` vectors to each of `threads`
// (a multiple of 32).
struct Deal {
  int nv, threads;
};

// The one of the compiled counts that pads the row least; on a tie the larger
// (fewer threads, more loads in flight in each).
template <int N>
Deal deal(int64_t vecs, const int (&counts)[N], int max_threads) {
  Deal best{0, 0};
  for (int nv : counts) {
    const int64_t threads = (vecs + (int64_t)32 * nv - 1) / ((int64_t)32 * nv) * 32;
    if (threads > max_threads) continue;
    if (!best.nv || threads * nv <= (int64_t)best.nv * best.threads) best = Deal{nv, (int)threads};
  }
  return best;
}

// A row's place in a ring: the words it may lie in, and one more that a
// shifted read may touch.
template <class T>
int ring_slot(int64_t cols) {
  return (int)((cols * (int64_t)sizeof(T) + 15 + 15) / 16 * 16) + 16;
}

constexpr int kRingMaxShared = 200 * 1024;

// How many blocks of a persistent kernel the device holds.
template <class K>
cudaError_t resident(K* kernel, int threads, int smem, int64_t* blocks) {
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  *blocks = (int64_t)sm_count() * std::max(per_sm, 1);
  return e;
}

// How deep a group's ring is.  A row is in registers while it is worked on and
// its place is being filled again, so one place is enough to keep loads on
// their way; more where the groups that fit a multiprocessor (by registers)
// have less than `bytes` of places.  Not more than that: what shared memory
// does not take is the L1 cache that the parameters are read from (16384 x
// 4096 bf16 with f32 parameters read again for each row, forward: 64 KB 65 us,
// 128 KB 80 us; backward, from HBM, 8192 x 768 f32 and 32768 x 4096 bf16: 64 KB
// 23.7 and 152 us, 96 KB 21.8 and 147, 128 KB 21.9 and 149).
constexpr int kForwardRing = 64 * 1024, kBackwardRing = 96 * 1024;
int ring_stages(int bytes, int row_bytes, int threads, int registers) {
  const int groups = std::max(1, 65536 / registers / threads);
  return std::max(1, std::min(kRing, (bytes / groups + row_bytes / 2) / row_bytes));
}

template <class T, class P>
bool params_aligned(const void* p) {
  return (uintptr_t)p % (16 / sizeof(T) * sizeof(P)) == 0;
}

// Groups in a block: enough of them to fill 256 threads, but not so many that
// few rows leave multiprocessors idle.
int ring_groups(int threads, int64_t rows) {
  const int64_t each = rows / sm_count();
  return (int)std::max<int64_t>(1, std::min<int64_t>({kGroups - 1, 256 / threads, each}));
}

template <class T>
cudaError_t start_ring(void (*kernel)(LayerNormArgs, int, int), std::atomic<unsigned long long>* opened, int threads,
                       int registers, const LayerNormArgs& a, cudaStream_t s) {
  const int slot = ring_slot<T>(a.cols), stages = ring_stages(kForwardRing, slot, threads, registers);
  const int groups = threads >= 128 ? 1 : ring_groups(threads, a.rows);
  const int smem = groups * stages * slot;
  cudaError_t e = open_kernel((const void*)kernel, kRingMaxShared, false, opened);
  if (e != cudaSuccess) return e;
  int64_t blocks = 0;
  if ((e = resident(kernel, threads * groups, smem, &blocks)) != cudaSuccess) return e;
  blocks = std::min<int64_t>(blocks, (a.rows + groups - 1) / groups);
  kernel<<<(unsigned)blocks, dim3(threads, groups), smem, s>>>(a, slot, stages);
  note_launch();
  return cudaGetLastError();
}

template <class T, class P, int NV, bool KEEP = false>
cudaError_t run_ring(const LayerNormArgs& a, int threads, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  return start_ring<T>(layer_norm_ring_kernel<T, P, NV, KEEP>, opened, threads,
                       KEEP ? 88 : forward_registers(NV * (16 / (int)sizeof(T))), a, s);
}
template <class T, class P, int NE>
cudaError_t run_strided(const LayerNormArgs& a, int threads, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  return start_ring<T>(layer_norm_strided_kernel<T, P, NE>, opened, threads, strided_registers(NE), a, s);
}

template <class T, class P>
bool forward_ring(const LayerNormArgs& a, cudaStream_t s, cudaError_t* e) {
  constexpr int VW = 16 / sizeof(T), A = VW == 8 ? 1 : 2;
  if (a.cols > 32768 || ring_slot<T>(a.cols) > kRingMaxShared) return false;
  const bool whole = a.cols % VW == 0 && rows_aligned16(a.x, a.x_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.y, a.y_stride, a.rows, sizeof(T)) && params_aligned<T, P>(a.weight) &&
                     params_aligned<T, P>(a.bias);
  if (!whole) {
    // 32 elements to a thread only where 16 do not reach (8192 x 16383 f16: 128
    // us, and 397 with rows in 1024 threads' registers, without a ring)
    static const int counts[2] = {8, 16}, wide[1] = {32};
    Deal d = deal(a.cols, counts, 512);
    if (!d.nv) d = deal(a.cols, wide, 512);
    if (d.nv == 8) *e = run_strided<T, P, 8>(a, d.threads, s);
    else if (d.nv == 16) *e = run_strided<T, P, 16>(a, d.threads, s);
    else if (d.nv) *e = run_strided<T, P, 32>(a, d.threads, s);
    return d.nv != 0;
  }
  static const int counts[5] = {1, A, 2 * A, 3 * A, 4 * A};
  if constexpr (sizeof(P) == 4 && sizeof(T) == 2) {
    // f32 parameters of 16-bit rows stay in registers, two vectors to a thread,
    // unless that leaves more than an eighth of a narrow row's threads without
    // work (16384 rows, the same ones again and again, narrow ones in L2;
    // parameters kept, and read again for each row: 512 columns 7.8 and 10.1 us,
    // 768 15.9 and 12.7, 1536 22.9 and 25.6, 2048 31.0 and 36.5, 4096 58.1 and
    // 67.2).
    static const int kept[1] = {2 * A};
    const Deal d = deal(a.cols / VW, kept, 512);
    if (d.nv && (a.cols >= 2048 || (int64_t)d.threads * d.nv * VW * 8 <= a.cols * 9)) {
      *e = run_ring<T, P, 2 * A, true>(a, d.threads, s);
      return true;
    }
  }
  const Deal d = deal(a.cols / VW, counts, 512);
  if (d.nv == 1) {
    *e = run_ring<T, P, 1>(a, d.threads, s);
    return true;
  }
  switch (d.nv) {
    case A: *e = run_ring<T, P, A>(a, d.threads, s); return true;
    case 2 * A: *e = run_ring<T, P, 2 * A>(a, d.threads, s); return true;
    case 3 * A: *e = run_ring<T, P, 3 * A>(a, d.threads, s); return true;
    case 4 * A: *e = run_ring<T, P, 4 * A>(a, d.threads, s); return true;
  }
  return false;
}

template <class T, class P, int VW>
cudaError_t forward_wide(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int NV = 32 / VW;
  static const int counts[1] = {NV};
  if (const Deal d = deal((a.cols + VW - 1) / VW, counts, 1024); d.nv)
    layer_norm_kernel<T, P, VW, NV><<<(unsigned)a.rows, d.threads, 0, s>>>(a);
  else
    layer_norm_wide_kernel<T, P><<<(unsigned)a.rows, 1024, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

template <class P>
cudaError_t run_params(const LayerNormBackwardArgs& a, int blocks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((2 * a.cols + 31) / 32));
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, layer_norm_params_kernel<P>, (const float*)a.partial, blocks, a.cols,
                                     static_cast<P*>(a.dweight), static_cast<P*>(a.dbias));
  note_launch();
  return e;
}

// columns: what one thread sums for
template <class T, class P>
cudaError_t start_backward_ring(void (*kernel)(LayerNormBackwardArgs, int, int), std::atomic<unsigned long long>* opened,
                                int threads, int columns, bool wide, const LayerNormBackwardArgs& a, cudaStream_t s) {
  const int slot = ring_slot<T>(a.cols);
  const int stages = wide ? std::min(2, kRingMaxShared / (2 * slot))
                          : ring_stages(kBackwardRing, 2 * slot, threads, backward_registers(columns));
  const int groups = wide ? 1 : ring_groups(threads, a.rows);
  const int smem = std::max(groups * 2 * stages * slot, groups > 1 ? 2 * threads * columns * (int)sizeof(float) : 0);
  cudaError_t e = open_kernel((const void*)kernel, kRingMaxShared, false, opened);
  if (e != cudaSuccess) return e;
  int64_t blocks = 0;
  if ((e = resident(kernel, threads * groups, smem, &blocks)) != cudaSuccess) return e;
  blocks = std::min<int64_t>({blocks, layer_norm_partial_rows(a.rows, a.cols), (a.rows + groups - 1) / groups});
  kernel<<<(unsigned)blocks, dim3(threads, groups), smem, s>>>(a, slot, stages);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return run_params<P>(a, (int)blocks, s);
}

template <class T, class P, int NV, bool WIDE = false>
cudaError_t run_backward_ring(const LayerNormBackwardArgs& a, int threads, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  return start_backward_ring<T, P>(layer_norm_backward_ring_kernel<T, P, NV, WIDE>, opened, threads,
                                   NV * (16 / (int)sizeof(T)), WIDE, a, s);
}
template <class T, class P, int NE, bool WIDE = false>
cudaError_t run_backward_strided(const LayerNormBackwardArgs& a, int threads, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  return start_backward_ring<T, P>(layer_norm_backward_strided_kernel<T, P, NE, WIDE>, opened, threads, NE, WIDE, a, s);
}

template <class T, class P>
bool backward_ring(const LayerNormBackwardArgs& a, cudaStream_t s, cudaError_t* e) {
  constexpr int VW = 16 / sizeof(T), A = VW == 8 ? 1 : 2;
  if (a.cols > kLayerNormKeptCols || 2 * ring_slot<T>(a.cols) > kRingMaxShared) return false;
  const bool whole = a.cols % VW == 0 && rows_aligned16(a.x, a.x_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.dy, a.dy_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.dx, a.dx_stride, a.rows, sizeof(T)) && params_aligned<T, P>(a.weight);
  if (!whole) {
    static const int counts[2] = {8, 16}, wide[1] = {16};
    Deal d = deal(a.cols, counts, 512);
    if (d.nv == 8) *e = run_backward_strided<T, P, 8>(a, d.threads, s);
    else if (d.nv) *e = run_backward_strided<T, P, 16>(a, d.threads, s);
    else if ((d = deal(a.cols, wide, 1024)).nv) *e = run_backward_strided<T, P, 16, true>(a, d.threads, s);
    return d.nv != 0;
  }
  static const int counts[3] = {1, A, 2 * A}, wide[1] = {2 * A};
  Deal d = deal(a.cols / VW, counts, 512);
  if (!d.nv) {
    // More than 8192 columns.  16-bit rows: 8192 x 16384 bf16 278 us, and 353
    // with rows in 1024 threads' registers, without a ring.  An f32 row leaves
    // no room for a second one in shared memory (4096 x 16384: 220 us, and 173
    // without a ring) unless it is read element by element anyway (4096 x
    // 16381: 260 and 293).
    if constexpr (sizeof(T) == 4) return false;
    else if ((d = deal(a.cols / VW, wide, 1024)).nv) *e = run_backward_ring<T, P, 2 * A, true>(a, d.threads, s);
    return d.nv != 0;
  }
  if (d.nv == 1) *e = run_backward_ring<T, P, 1>(a, d.threads, s);
  else if (d.nv == A) *e = run_backward_ring<T, P, A>(a, d.threads, s);
  else if (d.nv) *e = run_backward_ring<T, P, 2 * A>(a, d.threads, s);
  return d.nv != 0;
}

template <class T, class P>
cudaError_t backward_wide(const LayerNormBackwardArgs& a, cudaStream_t s) {
  cudaError_t e;
  if constexpr (sizeof(T) == 4) {
    static const int counts[1] = {4};
    const Deal d = deal((a.cols + 3) / 4, counts, 1024);
    if (d.nv && rows_aligned16(a.x, a.x_stride, a.rows, 4) && rows_aligned16(a.dy, a.dy_stride, a.rows, 4) &&
        rows_aligned16(a.dx, a.dx_stride, a.rows, 4) && params_aligned<T, P>(a.weight)) {
      const int blocks = (int)std::min<int64_t>(sm_count(), layer_norm_partial_rows(a.rows, a.cols));
      layer_norm_backward_kernel<T, P, 4, 4><<<blocks, d.threads, 0, s>>>(a);
      note_launch();
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      return run_params<P>(a, blocks, s);
    }
  }
  const int slices = (int)std::min<int64_t>(kLayerNormMaxSlices, layer_norm_partial_rows(a.rows, a.cols));
  layer_norm_params_wide_kernel<T><<<dim3((unsigned)((a.cols + 255) / 256), slices), 256, 0, s>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  layer_norm_backward_wide_kernel<T, P><<<(unsigned)a.rows, 1024, 0, s>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return run_params<P>(a, slices, s);
}

// fn(T(), P()) for the types of the rows and of the parameters
template <class F>
cudaError_t with_types(int dtype, int pdtype, F fn) {
  return with_type(dtype, [&](auto t) {
    if (pdtype == F32) return fn(t, float());
    return fn(t, t);
  });
}

}  // namespace

cudaError_t launch_layer_norm(int dtype, int pdtype, const LayerNormArgs& a, cudaStream_t s) {
  return with_types(dtype, pdtype, [&](auto t, auto p) {
    using T = decltype(t);
    using P = decltype(p);
    constexpr int VW = 16 / sizeof(T);
    cudaError_t e;
    if (forward_ring<T, P>(a, s, &e)) return e;
    // 16-byte vectors where every row starts on one, single elements otherwise
    const bool vec = rows_aligned16(a.x, a.x_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.y, a.y_stride, a.rows, sizeof(T)) &&
                     (uintptr_t)a.weight % (VW * sizeof(P)) == 0 && (uintptr_t)a.bias % (VW * sizeof(P)) == 0;
    return vec ? forward_wide<T, P, VW>(a, s) : forward_wide<T, P, 1>(a, s);
  });
}

cudaError_t launch_layer_norm_backward(int dtype, int pdtype, const LayerNormBackwardArgs& a, cudaStream_t s) {
  return with_types(dtype, pdtype, [&](auto t, auto p) {
    using T = decltype(t);
    using P = decltype(p);
    cudaError_t e;
    return backward_ring<T, P>(a, s, &e) ? e : backward_wide<T, P>(a, s);
  });
}

cudaError_t layer_norm_take_status(int* status, cudaStream_t s) { return take_status(status, s); }

}  // namespace ar
