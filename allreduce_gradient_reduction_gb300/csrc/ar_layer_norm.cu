// Layer norm over the last axis, forward and backward.
//
//   mean = sum(x) / C, rstd = (sum((x - mean)^2) / C + eps)^-1/2
//   y  = (x - mean) rstd w + b
//   with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g)/C - xh sum(g xh)/C)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both directions are bound by HBM: a row is read once, held in registers as
// it was stored, and everything about it is computed from there in binary32.
// The variance is taken about the row's own mean (a second pass over the
// registers), not as a difference of two large sums.
//
// A row belongs to a group of whole warps, thread t of which owns the vectors
// t, t + G, t + 2G, ... of the row, so a group's accesses are contiguous and a
// thread's columns are the same in every row.  That lets the backward kernel
// keep its columns' share of dw and db in registers while its group walks
// over rows; the groups' sums are joined in a fixed order, in the block and
// then in a second kernel, so the result does not depend on timing.
#include "ar_ops.cuh"

#include <algorithm>

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

template <class T, class P, int VW, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_norm_kernel(const LayerNormArgs a) {
  __shared__ float scratch[kGroups][2][32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;
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
  const float mean = group_sum(sum, scratch[threadIdx.y], 0) * inv;
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
  const float rstd = rsqrtf(group_sum(sq, scratch[threadIdx.y], 1) * inv + a.eps);
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
// blockIdx.x of the partial sums.
template <int VW, int NV>
__device__ __forceinline__ void join_params(const float (&dw)[NV][VW], const float (&db)[NV][VW], float* joined,
                                            float* partial, int cols) {
  const int g = blockDim.x, t = threadIdx.x, width = g * NV * VW;
  float* out = partial + (int64_t)blockIdx.x * 2 * cols;
  __syncthreads();
  for (int y = 0; y + 1 < (int)blockDim.y; ++y) {
    if ((int)threadIdx.y == y) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          const int c = (k * g + t) * VW + i;
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
        const int c = (k * g + t) * VW + i;
        if (c < cols) {
          out[c] = dw[k][i] + (blockDim.y > 1 ? joined[c] : 0.f);
          out[cols + c] = db[k][i] + (blockDim.y > 1 ? joined[width + c] : 0.f);
        }
      }
  }
}

// One block's groups walk over the rows with a stride of all groups; the next
// row's loads are in flight while the current one is reduced.
template <class T, class P, int VW, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_norm_backward_kernel(const LayerNormBackwardArgs a) {
  constexpr bool kAhead = MAXT <= 512;  // 1024 threads have 64 registers each: no room for a second row
  __shared__ float scratch[kGroups][2][32];
  extern __shared__ float joined[];  // [2][groups' columns] when the block has several groups
  const int cols = (int)a.cols;
  const int g = blockDim.x, t = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const P* weight = static_cast<const P*>(a.weight);
  const float inv = 1.0f / (float)cols;

  float dw[NV][VW], db[NV][VW];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VW; ++i) dw[k][i] = db[k][i] = 0.f;

  Pack<T, VW> xr[NV], dr[NV], xn[NV], dn[NV];
  float mean_n = 0.f, rstd_n = 0.f;
  auto fetch = [&](int64_t row, Pack<T, VW>* px, Pack<T, VW>* pd, float& m, float& r) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * g + t) * VW;
      px[k] = load_pack<T, VW>(x, c, cols);
      pd[k] = load_pack<T, VW>(dy, c, cols);
    }
    m = a.mean[row];
    r = a.rstd[row];
  };
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (kAhead && row < a.rows) fetch(row, xn, dn, mean_n, rstd_n);
  for (; row < a.rows; row += step) {
    float mean, rstd;
    if constexpr (kAhead) {
#pragma unroll
      for (int k = 0; k < NV; ++k) xr[k] = xn[k], dr[k] = dn[k];
      mean = mean_n;
      rstd = rstd_n;
      if (row + step < a.rows) fetch(row + step, xn, dn, mean_n, rstd_n);
    } else {
      fetch(row, xr, dr, mean, rstd);
    }
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
    const int warps = g >> 5;
    if (warps > 1) {
      float* s = scratch[threadIdx.y][0];
      float* u = scratch[threadIdx.y][1];
      const int w = t >> 5, lane = t & 31;
      if (blockDim.y == 1) __syncthreads();
      else named_barrier(1 + threadIdx.y, g);
      if (lane == 0) s[w] = s1, u[w] = s2;
      if (blockDim.y == 1) __syncthreads();
      else named_barrier(1 + threadIdx.y, g);
      s1 = warp_sum(lane < warps ? s[lane] : 0.f);
      s2 = warp_sum(lane < warps ? u[lane] : 0.f);
    }
    s1 *= inv;
    s2 *= inv;
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
  join_params<VW, NV>(dw, db, joined, a.partial, cols);
}

// ---- rows through shared memory -----------------------------------------------------
//
// For rows of 1 KB and more: each group keeps a ring of rows in shared memory,
// filled by bulk copies that its first thread issues several rows ahead, so
// the bytes in flight do not depend on registers or occupancy.  A copy takes
// the aligned 16-byte words that hold a row; a row that starts inside a word
// is put right when it is read (two words and a shift), and so is a result
// row that starts inside one, on its way through a buffer of the group's.
// Vectors are therefore counted from the row's first column whatever its
// address, and the parameters' values for a thread's columns are loaded once.

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

// A copy ends by itself, so this wait does; the limit is for a launch that
// has gone wrong, whose results are then wrong too but which ends.
__device__ __forceinline__ void ring_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < (1 << 22); ++i) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return;
  }
}

// 16 bytes at `at`, `shift` bytes past an aligned word (a multiple of ES).
template <int ES>
__device__ __forceinline__ uint4 shifted16(const uint8_t* word, int shift) {
  const uint4 a = *reinterpret_cast<const uint4*>(word);
  if (shift == 0) return a;
  const uint4 b = *reinterpret_cast<const uint4*>(word + 16);
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (ES == 2 && (shift & 2)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Vector v of a row in its slot, places past the row's end as zeros.
template <class T>
__device__ __forceinline__ Pack<T, 16 / sizeof(T)> slot_vector(const uint8_t* slot, int shift, int v, int cols) {
  constexpr int VW = 16 / sizeof(T);
  if (v * VW >= cols) return zero_pack<T, VW>();
  const uint4 raw = shifted16<sizeof(T)>(slot + v * 16, shift);
  Pack<T, VW> p = *reinterpret_cast<const Pack<T, VW>*>(&raw);
  if ((v + 1) * VW > cols) {
#pragma unroll
    for (int i = 0; i < VW; ++i)
      if (v * VW + i >= cols) p.v[i] = Conv<T>::down(0.f);
  }
  return p;
}

__device__ __forceinline__ void group_barrier() {
  if (blockDim.x == 32) __syncwarp();
  else if (blockDim.y == 1) __syncthreads();
  else named_barrier(1 + threadIdx.y, blockDim.x);
}

// A thread's parameters, element by element where they are not aligned.
template <class P, int VW>
__device__ __forceinline__ Pack<P, VW> param_vector(const P* p, int c, int cols) {
  if (p && ((uintptr_t)p & (sizeof(Pack<P, VW>) - 1)) == 0) return load_pack<P, VW>(p, c, cols);
  Pack<P, VW> r = zero_pack<P, VW>();
#pragma unroll
  for (int i = 0; i < VW; ++i)
    if (p && c + i < cols) r.v[i] = p[c + i];
  return r;
}

// Writes the group's row, vector k * blockDim.x + t of which is o[k].
template <class T, int NV>
__device__ __forceinline__ void write_row(T* row, const Pack<T, 16 / sizeof(T)> (&o)[NV], int cols, uint8_t* buffer) {
  constexpr int VW = 16 / sizeof(T), ES = sizeof(T);
  const int g = blockDim.x, t = threadIdx.x;
  const int phase = (int)((uintptr_t)row & 15);
  if (phase == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * g + t) * VW < cols) store_pack<T, VW>(row, (k * g + t) * VW, cols, o[k]);
    return;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if ((k * g + t) * VW < cols) *reinterpret_cast<Pack<T, VW>*>(buffer + (k * g + t) * 16) = o[k];
  group_barrier();
  // aligned word u of the result row holds its bytes [16 u - phase, 16 u - phase + 16)
  const int bytes = cols * ES, words = (bytes + phase + 15) / 16;
  for (int u = t; u < words; u += g) {
    const int b = u * 16 - phase;
    if (b >= 0 && b + 16 <= bytes) {
      *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(row) + b) = shifted16<ES>(buffer + (b & ~15), b & 15);
    } else {
      for (int c = max(b, 0) / ES; c < min(b + 16, bytes) / ES; ++c) row[c] = reinterpret_cast<const T*>(buffer)[c];
    }
  }
}

constexpr int kRing = 4;  // rows of a group in flight

__device__ __forceinline__ void open_ring(uint64_t* full) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_at(full + i)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// slot: bytes of one row's place in shared memory
template <class T, class P, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_norm_ring_kernel(const LayerNormArgs a, int slot) {
  constexpr int VW = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ float scratch[kGroups][2][32];
  __shared__ __align__(8) uint64_t full[kGroups][kRing];
  const int cols = (int)a.cols, g = blockDim.x, t = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const T* x = static_cast<const T*>(a.x);
  uint8_t* mine = rows + (int64_t)threadIdx.y * (kRing + 1) * slot;
  uint64_t* bars = full[threadIdx.y];
  const float inv = 1.0f / (float)cols;
  auto issue = [&](int64_t row, int stage) {
    const T* from = x + row * a.x_stride;
    const uint32_t bar = smem_at(bars + stage);
    ring_expect(bar, covering(from, cols * (int)sizeof(T)));
    ring_copy(smem_at(mine + stage * slot), from, cols * (int)sizeof(T), bar);
  };
  open_ring(bars);
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t == 0)
    for (int i = 0; i < kRing && row + i * step < a.rows; ++i) issue(row + i * step, i);

  Pack<P, VW> w[NV], b[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    w[k] = param_vector<P, VW>(static_cast<const P*>(a.weight), (k * g + t) * VW, cols);
    b[k] = param_vector<P, VW>(static_cast<const P*>(a.bias), (k * g + t) * VW, cols);
  }
  int stage = 0, parity = 0;
  for (; row < a.rows; row += step) {
    ring_wait(smem_at(bars + stage), parity);
    Pack<T, VW> xr[NV];
    const int shift = (int)((uintptr_t)(x + row * a.x_stride) & 15);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      xr[k] = slot_vector<T>(mine + stage * slot, shift, k * g + t, cols);
#pragma unroll
      for (int i = 0; i < VW; ++i) sum += Conv<T>::up(xr[k].v[i]);
    }
    const float mean = group_sum(sum, scratch[threadIdx.y], 0) * inv;
    if (g == 32) __syncwarp();
    if (t == 0 && row + kRing * step < a.rows) issue(row + kRing * step, stage);  // the group has read the slot
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float d = Conv<T>::up(xr[k].v[i]) - mean;
        if ((k * g + t) * VW + i < cols) sq = fmaf(d, d, sq);
      }
    const float rstd = rsqrtf(group_sum(sq, scratch[threadIdx.y], 1) * inv + a.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VW; ++i)
        xr[k].v[i] = Conv<T>::down(fmaf((Conv<T>::up(xr[k].v[i]) - mean) * rstd, Conv<P>::up(w[k].v[i]), Conv<P>::up(b[k].v[i])));
    write_row<T, NV>(static_cast<T*>(a.y) + row * a.y_stride, xr, cols, mine + kRing * slot);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (++stage == kRing) stage = 0, parity ^= 1;
  }
}

template <class T, class P, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_norm_backward_ring_kernel(const LayerNormBackwardArgs a, int slot) {
  constexpr int VW = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t rows[];
  __shared__ float scratch[kGroups][2][2][32];
  __shared__ __align__(8) uint64_t full[kGroups][kRing];
  const int cols = (int)a.cols, g = blockDim.x, t = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  uint8_t* mine = rows + (int64_t)threadIdx.y * (2 * kRing + 1) * slot;
  uint64_t* bars = full[threadIdx.y];
  const float inv = 1.0f / (float)cols;
  auto issue = [&](int64_t row, int stage) {
    const int bytes = cols * (int)sizeof(T);
    const T *fx = x + row * a.x_stride, *fd = dy + row * a.dy_stride;
    const uint32_t bar = smem_at(bars + stage), to = smem_at(mine + stage * 2 * slot);
    ring_expect(bar, covering(fx, bytes) + covering(fd, bytes));
    ring_copy(to, fx, bytes, bar);
    ring_copy(to + slot, fd, bytes, bar);
  };
  open_ring(bars);
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t == 0)
    for (int i = 0; i < kRing && row + i * step < a.rows; ++i) issue(row + i * step, i);

  Pack<P, VW> w[NV];
  float dw[NV][VW], db[NV][VW];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    w[k] = param_vector<P, VW>(static_cast<const P*>(a.weight), (k * g + t) * VW, cols);
#pragma unroll
    for (int i = 0; i < VW; ++i) dw[k][i] = db[k][i] = 0.f;
  }
  float mean = 0.f, rstd = 0.f;
  if (row < a.rows) mean = a.mean[row], rstd = a.rstd[row];
  int stage = 0, parity = 0;
  for (int64_t n = 0; row < a.rows; row += step, ++n) {
    float mean_n = 0.f, rstd_n = 0.f;
    if (row + step < a.rows) mean_n = a.mean[row + step], rstd_n = a.rstd[row + step];
    ring_wait(smem_at(bars + stage), parity);
    Pack<T, VW> xr[NV], dr[NV];
    const int sx = (int)((uintptr_t)(x + row * a.x_stride) & 15), sd = (int)((uintptr_t)(dy + row * a.dy_stride) & 15);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      xr[k] = slot_vector<T>(mine + stage * 2 * slot, sx, k * g + t, cols);
      dr[k] = slot_vector<T>(mine + stage * 2 * slot + slot, sd, k * g + t, cols);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float d = Conv<T>::up(dr[k].v[i]);
        const float xh = (Conv<T>::up(xr[k].v[i]) - mean) * rstd;
        const float gw = d * Conv<P>::up(w[k].v[i]);
        dw[k][i] = fmaf(d, xh, dw[k][i]);
        db[k][i] += d;
        s1 += gw;
        s2 = fmaf(gw, xh, s2);
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (g > 32) {
      // one barrier a row: the scratch of the row before last is free by then
      float (*s)[32] = scratch[threadIdx.y][n & 1];
      const int wp = t >> 5, lane = t & 31;
      if (lane == 0) s[0][wp] = s1, s[1][wp] = s2;
      group_barrier();
      s1 = warp_sum(lane < (g >> 5) ? s[0][lane] : 0.f);
      s2 = warp_sum(lane < (g >> 5) ? s[1][lane] : 0.f);
    } else {
      __syncwarp();
    }
    if (t == 0 && row + kRing * step < a.rows) issue(row + kRing * step, stage);  // the group has read the slot
    s1 *= inv;
    s2 *= inv;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float xh = (Conv<T>::up(xr[k].v[i]) - mean) * rstd;
        const float gw = Conv<T>::up(dr[k].v[i]) * Conv<P>::up(w[k].v[i]);
        xr[k].v[i] = Conv<T>::down(rstd * (gw - s1 - xh * s2));
      }
    write_row<T, NV>(static_cast<T*>(a.dx) + row * a.dx_stride, xr, cols, mine + 2 * kRing * slot);
    mean = mean_n;
    rstd = rstd_n;
    if (++stage == kRing) stage = 0, parity ^= 1;
  }
  join_params<VW, NV>(dw, db, reinterpret_cast<float*>(rows), a.partial, cols);
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

template <class T, class P, int VW, int NV, int MAXT>
cudaError_t run_forward(const LayerNormArgs& a, int threads, cudaStream_t s) {
  const int groups = std::max(1, std::min(kGroups - 1, 128 / threads));
  const int64_t blocks = (a.rows + groups - 1) / groups;
  layer_norm_kernel<T, P, VW, NV, MAXT><<<(unsigned)blocks, dim3(threads, groups), 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

// A row's place in a ring: the words it may lie in, and one more that a
// shifted read may touch.
template <class T>
int ring_slot(int64_t cols) {
  return (int)((cols * (int64_t)sizeof(T) + 15 + 15) / 16 * 16) + 16;
}

constexpr int kRingMinBytes = 1024;       // shorter rows: one warp takes one at a time, without a ring
constexpr int kRingMaxShared = 200 * 1024;

// How many blocks of a persistent kernel the device holds.
template <class K>
cudaError_t resident(K* kernel, int threads, int smem, int64_t* blocks) {
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  *blocks = (int64_t)sm_count() * std::max(per_sm, 1);
  return e;
}

template <class T, class P, int NV, int MAXT>
cudaError_t run_ring(const LayerNormArgs& a, int threads, cudaStream_t s) {
  auto* kernel = layer_norm_ring_kernel<T, P, NV, MAXT>;
  static std::atomic<unsigned long long> opened[256];
  const int slot = ring_slot<T>(a.cols), ring = (kRing + 1) * slot;
  const int groups = std::max(1, std::min({kGroups - 1, 256 / threads, kRingMaxShared / ring}));
  cudaError_t e = open_kernel((const void*)kernel, kRingMaxShared, false, opened);
  if (e != cudaSuccess) return e;
  int64_t blocks = 0;
  if ((e = resident(kernel, threads * groups, groups * ring, &blocks)) != cudaSuccess) return e;
  blocks = std::min<int64_t>(blocks, (a.rows + groups - 1) / groups);
  kernel<<<(unsigned)blocks, dim3(threads, groups), groups * ring, s>>>(a, slot);
  count_launch();
  return cudaGetLastError();
}

template <class T, class P>
bool forward_ring(const LayerNormArgs& a, cudaStream_t s, cudaError_t* e) {
  constexpr int VW = 16 / sizeof(T), A = VW == 8 ? 1 : 2;
  if (a.cols * (int64_t)sizeof(T) < kRingMinBytes || (kRing + 1) * (int64_t)ring_slot<T>(a.cols) > kRingMaxShared) return false;
  static const int counts[2] = {A, 2 * A};
  const Deal d = deal((a.cols + VW - 1) / VW, counts, 512);
  if (d.nv == A) *e = run_ring<T, P, A, 512>(a, d.threads, s);
  else if (d.nv) *e = run_ring<T, P, 2 * A, 512>(a, d.threads, s);
  else return false;
  return true;
}

template <class T, class P, int VW>
cudaError_t forward(const LayerNormArgs& a, cudaStream_t s) {
  const int64_t vecs = (a.cols + VW - 1) / VW;
  // a row of up to 32 elements a thread stays in registers
  constexpr int A = VW == 1 ? 4 : VW == 8 ? 1 : 2, B = 2 * A, C = VW == 1 ? 16 : 3 * A, D = VW == 1 ? 32 : 4 * A;
  static const int counts[4] = {A, B, C, D};
  const Deal d = deal(vecs, counts, 512);
  switch (d.nv) {
    case A: return run_forward<T, P, VW, A, 512>(a, d.threads, s);
    case B: return run_forward<T, P, VW, B, 512>(a, d.threads, s);
    case C: return run_forward<T, P, VW, C, 512>(a, d.threads, s);
    case D: return run_forward<T, P, VW, D, 512>(a, d.threads, s);
  }
  static const int most[1] = {D};
  if (const Deal w = deal(vecs, most, 1024); w.nv) return run_forward<T, P, VW, D, 1024>(a, w.threads, s);
  layer_norm_wide_kernel<T, P><<<(unsigned)a.rows, 1024, 0, s>>>(a);
  count_launch();
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
  count_launch();
  return e;
}

template <class T, class P, int VW, int NV, int MAXT>
cudaError_t run_backward(const LayerNormBackwardArgs& a, int threads, cudaStream_t s) {
  auto* kernel = layer_norm_backward_kernel<T, P, VW, NV, MAXT>;
  const int groups = std::max(1, std::min(kGroups - 1, std::min(MAXT, 512) / threads));
  const int smem = groups > 1 ? 2 * threads * NV * VW * (int)sizeof(float) : 0;
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads * groups, smem);
  if (e != cudaSuccess) return e;
  const int64_t want = std::min<int64_t>((int64_t)sm_count() * std::max(per_sm, 1), kLayerNormMaxBlocks);
  const int blocks = (int)std::min<int64_t>(want, (a.rows + groups - 1) / groups);
  kernel<<<blocks, dim3(threads, groups), smem, s>>>(a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return run_params<P>(a, blocks, s);
}

template <class T, class P, int NV, int MAXT>
cudaError_t run_backward_ring(const LayerNormBackwardArgs& a, int threads, cudaStream_t s) {
  constexpr int VW = 16 / sizeof(T);
  auto* kernel = layer_norm_backward_ring_kernel<T, P, NV, MAXT>;
  static std::atomic<unsigned long long> opened[256];
  const int slot = ring_slot<T>(a.cols), ring = (2 * kRing + 1) * slot;
  const int groups = std::max(1, std::min({kGroups - 1, 256 / threads, kRingMaxShared / ring}));
  const int smem = std::max(groups * ring, groups > 1 ? 2 * threads * NV * VW * (int)sizeof(float) : 0);
  cudaError_t e = open_kernel((const void*)kernel, kRingMaxShared, false, opened);
  if (e != cudaSuccess) return e;
  int64_t blocks = 0;
  if ((e = resident(kernel, threads * groups, smem, &blocks)) != cudaSuccess) return e;
  blocks = std::min<int64_t>({blocks, kLayerNormMaxBlocks, (a.rows + groups - 1) / groups});
  kernel<<<(unsigned)blocks, dim3(threads, groups), smem, s>>>(a, slot);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return run_params<P>(a, (int)blocks, s);
}

template <class T, class P>
bool backward_ring(const LayerNormBackwardArgs& a, cudaStream_t s, cudaError_t* e) {
  constexpr int VW = 16 / sizeof(T), A = VW == 8 ? 1 : 2;
  if (a.cols * (int64_t)sizeof(T) < kRingMinBytes || (2 * kRing + 1) * (int64_t)ring_slot<T>(a.cols) > kRingMaxShared) return false;
  static const int counts[2] = {A, 2 * A};
  const Deal d = deal((a.cols + VW - 1) / VW, counts, 512);
  if (d.nv == A) *e = run_backward_ring<T, P, A, 512>(a, d.threads, s);
  else if (d.nv) *e = run_backward_ring<T, P, 2 * A, 512>(a, d.threads, s);
  else return false;
  return true;
}

template <class T, class P, int VW>
cudaError_t backward(const LayerNormBackwardArgs& a, cudaStream_t s) {
  const int64_t vecs = (a.cols + VW - 1) / VW;
  // up to 16 columns a thread: their two sums, weights and rows fit its registers
  constexpr int A = VW == 8 ? 1 : VW == 4 ? 1 : 4, B = 2 * A, C = 4 * A;
  Deal d;
  if constexpr (VW == 8) {
    static const int counts[2] = {A, B};
    d = deal(vecs, counts, 512);
    if (d.nv == A) return run_backward<T, P, VW, A, 512>(a, d.threads, s);
    if (d.nv == B) return run_backward<T, P, VW, B, 512>(a, d.threads, s);
    d = deal(vecs, counts, 1024);
    if (d.nv) return run_backward<T, P, VW, B, 1024>(a, (int)((vecs + 32 * B - 1) / (32 * B) * 32), s);
  } else {
    static const int counts[3] = {A, B, C};
    d = deal(vecs, counts, 512);
    if (d.nv == A) return run_backward<T, P, VW, A, 512>(a, d.threads, s);
    if (d.nv == B) return run_backward<T, P, VW, B, 512>(a, d.threads, s);
    if (d.nv == C) return run_backward<T, P, VW, C, 512>(a, d.threads, s);
    d = deal(vecs, counts, 1024);
    if (d.nv) return run_backward<T, P, VW, C, 1024>(a, (int)((vecs + 32 * C - 1) / (32 * C) * 32), s);
  }
  const int slices = (int)std::min<int64_t>(a.rows, 64);
  layer_norm_params_wide_kernel<T><<<dim3((unsigned)((a.cols + 255) / 256), slices), 256, 0, s>>>(a);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  layer_norm_backward_wide_kernel<T, P><<<(unsigned)a.rows, 1024, 0, s>>>(a);
  count_launch();
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
    return vec ? forward<T, P, VW>(a, s) : forward<T, P, 1>(a, s);
  });
}

cudaError_t launch_layer_norm_backward(int dtype, int pdtype, const LayerNormBackwardArgs& a, cudaStream_t s) {
  return with_types(dtype, pdtype, [&](auto t, auto p) {
    using T = decltype(t);
    using P = decltype(p);
    constexpr int VW = 16 / sizeof(T);
    cudaError_t e;
    if (backward_ring<T, P>(a, s, &e)) return e;
    const bool vec = rows_aligned16(a.x, a.x_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.dy, a.dy_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.dx, a.dx_stride, a.rows, sizeof(T)) &&
                     (uintptr_t)a.weight % (VW * sizeof(P)) == 0;
    return vec ? backward<T, P, VW>(a, s) : backward<T, P, 1>(a, s);
  });
}

}  // namespace ar
