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

  // the block's groups are added in order
  float* out = a.partial + (int64_t)blockIdx.x * 2 * cols;
  const int width = g * NV * VW;
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
    const bool vec = rows_aligned16(a.x, a.x_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.dy, a.dy_stride, a.rows, sizeof(T)) &&
                     rows_aligned16(a.dx, a.dx_stride, a.rows, sizeof(T)) &&
                     (uintptr_t)a.weight % (VW * sizeof(P)) == 0;
    return vec ? backward<T, P, VW>(a, s) : backward<T, P, 1>(a, s);
  });
}

}  // namespace ar
