// Norm of each head of the queries and keys, and the rotation by the token's
// position, in one pass; and the gradient.
//
//   rstd = (sum x^2 / dim + eps)^-1/2, n = x rstd w,
//   y_a = n_a cos - n_b sin, y_b = n_b cos + n_a sin
// for each pair (a, b) of the first `rotary` elements, whose angle is position
// times the pair's frequency; the others are n.  Backward turns dy back (g),
//   dw = sum over tokens and heads of g x rstd,
//   dx = rstd (g w - x rstd^2 sum(g w x) / dim).
//
// Bound by HBM: each element read and written once (two reads backward).  A
// group of lanes has one head of one token, VEC pairs to a lane, both elements
// of a pair in the same lane, so that the rotation exchanges nothing.  A warp
// takes a token's heads one after another, since all of them turn by the same
// angles, and has the next head under way while one is worked on.
//
// Angles: the frequency is a 64-bit fraction of a turn, so the product with the
// position, modulo one turn, is an integer product that loses nothing (a
// frequency is off by 2^-65 turns at most, at position 2^31 by 2^-34).  The top
// two bits after rounding are the quarter; what is left is at most an eighth of
// a turn, for which Taylor's series to x^9 and x^10 are within 2e-9.
#include <cuda_runtime.h>

#include <algorithm>

#include "ar_ops.cuh"

namespace ar {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = kQkMaxDim / 2;

__device__ __forceinline__ void cos_sin(int32_t position, uint64_t turn, float& c, float& s) {
  const uint64_t angle = (uint64_t)(int64_t)position * turn;
  const uint64_t round = angle + (1ull << 61);
  const uint32_t quarter = (uint32_t)(round >> 62);
  // what is left of the turn, in [-1/8, 1/8) times 2^64
  const int64_t rest = (int64_t)((round & ((1ull << 62) - 1)) - (1ull << 61));
  const float x = __ll2float_rn(rest >> 24) * (float)(6.283185307179586 / (1ull << 40));
  const float sq = x * x;
  float sn = fmaf(sq, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, 1/7!
  sn = fmaf(sn, sq, 8.33333333e-3f);
  sn = fmaf(sn, sq, -1.66666667e-1f);
  sn = fmaf(sn * sq, x, x);
  float cs = fmaf(sq, -2.75573192e-7f, 2.48015873e-5f);  // 1/10!, 1/8!
  cs = fmaf(cs, sq, -1.38888889e-3f);
  cs = fmaf(cs, sq, 4.16666667e-2f);
  cs = fmaf(cs, sq, -0.5f);
  cs = fmaf(cs, sq, 1.f);
  const bool odd = quarter & 1;
  c = odd ? sn : cs;
  s = odd ? cs : sn;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter >= 2) s = -s;
}

// The layout of a head over LANES lanes: CHUNKS times VEC pairs to a lane.
template <class T, int VEC, int LANES, int CHUNKS, bool INTERLEAVED>
struct Head {
  static constexpr int kPairs = VEC * CHUNKS;  // of a lane
  using P = Pack<T, VEC>;
  struct Raw {
    P lo[CHUNKS], hi[CHUNKS];
  };
  // Pair p (a multiple of VEC): where its elements are.  Side by side: pair i
  // is (2i, 2i + 1).  Else the first half of what is rotated pairs with the
  // second, and so does the first half of the rest with its second.
  static __device__ __forceinline__ void places(const QkArgs& a, int p, int& lo, int& hi) {
    if constexpr (INTERLEAVED) {
      lo = 2 * p;
      hi = 2 * p + VEC;
    } else {
      const int half = a.rotary / 2;
      const bool turned = p < half;
      lo = turned ? p : p + half;
      hi = lo + (turned ? half : (a.dim - a.rotary) / 2);
    }
  }
  static __device__ __forceinline__ int pair(int lane, int c) { return (c * LANES + lane) * VEC; }
  static __device__ __forceinline__ Raw load(const QkArgs& a, const T* row, int lane) {
    Raw r;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      r.lo[c] = r.hi[c] = zero_pack<T, VEC>();
      if (pair(lane, c) >= a.dim / 2) continue;
      int lo, hi;
      places(a, pair(lane, c), lo, hi);
      r.lo[c] = *reinterpret_cast<const P*>(row + lo);
      r.hi[c] = *reinterpret_cast<const P*>(row + hi);
    }
    return r;
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&x)[kPairs], float (&y)[kPairs]) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        auto at = [&](int e) { return Conv<T>::up(e < VEC ? r.lo[c].v[e % VEC] : r.hi[c].v[e % VEC]); };
        x[c * VEC + i] = INTERLEAVED ? at(2 * i) : at(i);
        y[c * VEC + i] = INTERLEAVED ? at(2 * i + 1) : at(VEC + i);
      }
  }
  static __device__ __forceinline__ void store(const QkArgs& a, T* row, int lane, const float (&x)[kPairs],
                                               const float (&y)[kPairs]) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (pair(lane, c) >= a.dim / 2) continue;
      P lo, hi;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        auto to = [&](int e, float f) { (e < VEC ? lo.v[e % VEC] : hi.v[e % VEC]) = Conv<T>::down(f); };
        to(INTERLEAVED ? 2 * i : i, x[c * VEC + i]);
        to(INTERLEAVED ? 2 * i + 1 : VEC + i, y[c * VEC + i]);
      }
      int at_lo, at_hi;
      places(a, pair(lane, c), at_lo, at_hi);
      *reinterpret_cast<P*>(row + at_lo) = lo;
      *reinterpret_cast<P*>(row + at_hi) = hi;
    }
  }
};

// What a block keeps in shared memory, by pair: weights of both elements
// (ones without a weight), of queries and keys, and turns.
struct Kept {
  alignas(16) float weight[2][2][kMaxPairs];
  alignas(16) uint64_t turn[kMaxPairs];
};

template <class W, bool INTERLEAVED>
__device__ __forceinline__ void keep(const QkArgs& a, Kept& kept) {
  for (int i = threadIdx.x; i < kMaxPairs; i += kThreads) {
    int lo = 2 * i, hi = 2 * i + 1;
    if (!INTERLEAVED) {
      const int half = a.rotary / 2;
      lo = i < half ? i : i + half;
      hi = lo + (i < half ? half : (a.dim - a.rotary) / 2);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const W* w = static_cast<const W*>(a.weight[t]);
      const bool there = w && i < a.dim / 2;
      kept.weight[t][0][i] = there ? Conv<W>::up(w[lo]) : 1.f;
      kept.weight[t][1][i] = there ? Conv<W>::up(w[hi]) : 1.f;
    }
    kept.turn[i] = i < a.rotary / 2 ? a.turn[i] : 0;
  }
  __syncthreads();
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

// `parts` warps share a token's heads; each takes a round of kGroups heads,
// then the parts * kGroups-th after it.
template <class T, class W, int VEC, int LANES, int CHUNKS, bool INTERLEAVED, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, BACKWARD ? 2 : 3) qk_kernel(const __grid_constant__ QkArgs a, int parts) {
  using H = Head<T, VEC, LANES, CHUNKS, INTERLEAVED>;
  constexpr int kGroups = 32 / LANES, kPairs = H::kPairs;
  __shared__ Kept kept;
  const int lane = threadIdx.x % LANES, group = threadIdx.x % 32 / LANES;
  const int rows = a.heads[0] + a.heads[1], step = parts * kGroups;
  const int64_t warps = (int64_t)gridDim.x * kWarps, all = a.tokens * parts;

  int64_t item = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  int64_t token = item / parts;
  int row = (int)(item - token * parts) * kGroups + group;
  auto fetch = [&](int64_t token, int row, typename H::Raw& x, typename H::Raw& dy) {
    const int t = row >= a.heads[0], head = t ? row - a.heads[0] : row;
    if (token >= a.tokens || row >= rows) return;
    x = H::load(a, static_cast<const T*>(a.x[t].ptr) + token * a.x[t].token_stride + head * a.x[t].head_stride, lane);
    if (BACKWARD)
      dy = H::load(a, static_cast<const T*>(a.dy[t].ptr) + token * a.dy[t].token_stride + head * a.dy[t].head_stride, lane);
  };
  typename H::Raw x_next = {}, dy_next = {};
  fetch(token, row, x_next, dy_next);
  int32_t position = item < all ? a.positions[token] : 0;
  keep<W, INTERLEAVED>(a, kept);

  float sum[2][2][BACKWARD ? kPairs : 1] = {};  // of the weights' gradients: queries and keys, both elements
  float c[kPairs], s[kPairs];
  const float mean = 1.f / (float)a.dim;
  while (item < all) {
    // the token's angles, for all of its heads
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      cos_sin(position, kept.turn[H::pair(lane, i / VEC) + i % VEC], c[i], s[i]);
    const int64_t here = token;
    item += warps;
    token = item / parts;
    const int first = (int)(item - token * parts) * kGroups + group;
    if (item < all) position = a.positions[token];
    // a round of the warp's; every lane makes as many
    for (int base = row - group; base < rows; base += step) {
      const typename H::Raw x_raw = x_next, dy_raw = dy_next;
      const int now = base + group;
      const bool more = base + step < rows;
      fetch(more ? here : token, more ? now + step : first, x_next, dy_next);
      const int t = now >= a.heads[0], head = t ? now - a.heads[0] : now;
      float xa[kPairs], xb[kPairs];
      H::widen(x_raw, xa, xb);
      float wa[kPairs], wb[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int p = H::pair(lane, i / VEC) + i % VEC;
        wa[i] = kept.weight[t][0][p];
        wb[i] = kept.weight[t][1][p];
      }
      float squares = 0.f;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) squares = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], squares));
      if constexpr (!BACKWARD) {
        const float rstd = rsqrtf(fmaf(group_sum<LANES>(squares), mean, a.eps));
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float na = xa[i] * rstd * wa[i], nb = xb[i] * rstd * wb[i];
          xa[i] = na * c[i] - nb * s[i];
          xb[i] = nb * c[i] + na * s[i];
        }
      } else {
        float ga[kPairs], gb[kPairs], along = 0.f;
        H::widen(dy_raw, ga, gb);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float da = ga[i], db = gb[i];
          ga[i] = da * c[i] + db * s[i];
          gb[i] = db * c[i] - da * s[i];
          along = fmaf(ga[i] * wa[i], xa[i], fmaf(gb[i] * wb[i], xb[i], along));
        }
        const float rstd = rsqrtf(fmaf(group_sum<LANES>(squares), mean, a.eps));
        const float back = group_sum<LANES>(along) * mean * rstd * rstd;
        if (now < rows) {
          // (a row past the last holds what was fetched before)
          auto add = [&](float (&of)[2][BACKWARD ? kPairs : 1]) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
              of[0][i] = fmaf(ga[i], xa[i] * rstd, of[0][i]);
              of[1][i] = fmaf(gb[i], xb[i] * rstd, of[1][i]);
            }
          };
          if (t) add(sum[1]);
          else add(sum[0]);
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          xa[i] = rstd * (ga[i] * wa[i] - xa[i] * back);
          xb[i] = rstd * (gb[i] * wb[i] - xb[i] * back);
        }
      }
      if (now < rows)
        H::store(a, static_cast<T*>(const_cast<void*>(a.y[t].ptr)) + here * a.y[t].token_stride + head * a.y[t].head_stride,
                 lane, xa, xb);
    }
    row = first;
  }

  if constexpr (BACKWARD) {
    if (!a.partial) return;
    // the block's sums in a fixed order: over the groups of each warp, then warp after warp
    __shared__ float warp_sums[kWarps][2 * kMaxPairs];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          float v = sum[t][e][i];
#pragma unroll
          for (int m = LANES; m < 32; m <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
          const int p = H::pair(lane, i / VEC) + i % VEC;
          if (group == 0 && p < a.dim / 2) {
            int lo = 2 * p, hi = 2 * p + 1;
            if (!INTERLEAVED) {
              const int half = a.rotary / 2;
              lo = p < half ? p : p + half;
              hi = lo + (p < half ? half : (a.dim - a.rotary) / 2);
            }
            warp_sums[threadIdx.x / 32][e ? hi : lo] = v;
          }
        }
      __syncthreads();
      for (int d = threadIdx.x; d < a.dim; d += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += warp_sums[w][d];
        a.partial[((int64_t)blockIdx.x * 2 + t) * a.dim + d] = v;
      }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
}

// The weights' gradients: sums of the blocks' in their order, eight columns to a
// block, 32 rows of threads.
constexpr int kSumCols = 8, kSumRows = 32;
template <class W>
__global__ void __launch_bounds__(kSumCols* kSumRows) qk_weight_kernel(const float* partial, int blocks, int dim, W* dq, W* dk) {
  __shared__ float part[kSumRows][kSumCols];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int col = blockIdx.x * kSumCols + threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;
  float v = 0.f;
  if (col < 2 * dim)
    for (int b = row; b < blocks; b += kSumRows) v += partial[(int64_t)b * 2 * dim + col];
  part[row][threadIdx.x % kSumCols] = v;
  __syncthreads();
  if (row || col >= 2 * dim) return;
  v = 0.f;
#pragma unroll
  for (int r = 0; r < kSumRows; ++r) v += part[r][threadIdx.x];
  W* to = col < dim ? dq : dk;
  if (to) to[col < dim ? col : col - dim] = Conv<W>::down(v);
}

template <class W>
cudaError_t sum_weights(const QkArgs& a, int blocks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * a.dim + kSumCols - 1) / kSumCols);
  cfg.blockDim = dim3(kSumCols * kSumRows);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, qk_weight_kernel<W>, (const float*)a.partial, blocks, (int)a.dim,
                                           static_cast<W*>(a.dweight[0]), static_cast<W*>(a.dweight[1]));
  note_launch();
  return e;
}

template <class T, class W, int VEC, int LANES, int CHUNKS, bool INTERLEAVED, bool BACKWARD>
cudaError_t run(const QkArgs& a, cudaStream_t s) {
  constexpr int kGroups = 32 / LANES;
  const int rows = a.heads[0] + a.heads[1], rounds = (rows + kGroups - 1) / kGroups;
  // warps that share a token: one where the tokens fill the device, as many as there are rounds for a few
  constexpr int64_t kFull = 152 * 32;
  const int parts = (int)std::min<int64_t>(rounds, std::max<int64_t>(1, kFull / a.tokens));
  const int64_t most = BACKWARD ? kQkMaxBlocks : 152 * 8;
  const int blocks = (int)std::min<int64_t>(most, (a.tokens * parts + kWarps - 1) / kWarps);
  qk_kernel<T, W, VEC, LANES, CHUNKS, INTERLEAVED, BACKWARD><<<blocks, kThreads, 0, s>>>(a, parts);
  note_launch();
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess || !BACKWARD || !a.partial ? e : sum_weights<W>(a, blocks, s);
}

// Lanes to a head: as few powers of two as hold its pairs.
template <class T, class W, int VEC, bool INTERLEAVED, bool BACKWARD>
cudaError_t by_lanes(const QkArgs& a, cudaStream_t s) {
  const int lanes = (a.dim / 2 + VEC - 1) / VEC;
  if constexpr (VEC == 1) {
    return run<T, W, 1, 32, kMaxPairs / 32, INTERLEAVED, BACKWARD>(a, s);
  } else {
    if (lanes <= 4) return run<T, W, VEC, 4, 1, INTERLEAVED, BACKWARD>(a, s);
    if (lanes <= 8) return run<T, W, VEC, 8, 1, INTERLEAVED, BACKWARD>(a, s);
    if (VEC == 8 || lanes <= 16) return run<T, W, VEC, 16, 1, INTERLEAVED, BACKWARD>(a, s);
    if constexpr (VEC == 4) return run<T, W, VEC, 32, 1, INTERLEAVED, BACKWARD>(a, s);
    return cudaErrorInvalidValue;
  }
}

// Whether every pair's place, in all operands, allows accesses of `vec` elements.
bool fits(const QkArgs& a, bool interleaved, bool backward, int vec, int size) {
  if (a.dim / 2 % vec) return false;
  if (!interleaved && (a.rotary / 2 % vec || (a.dim - a.rotary) / 2 % vec)) return false;
  for (int t = 0; t < 2; ++t) {
    if (!a.heads[t]) continue;
    for (const QkTensor* x : {&a.x[t], &a.y[t], &a.dy[t]}) {
      if (x == &a.dy[t] && !backward) continue;
      if ((uintptr_t)x->ptr % (vec * size)) return false;
      if ((a.tokens > 1 && x->token_stride % vec) || (a.heads[t] > 1 && x->head_stride % vec)) return false;
    }
  }
  return true;
}

template <class T, class W, bool INTERLEAVED, bool BACKWARD>
cudaError_t by_vector(const QkArgs& a, cudaStream_t s) {
  constexpr int kWide = 16 / (int)sizeof(T);
  if (fits(a, INTERLEAVED, BACKWARD, kWide, sizeof(T))) return by_lanes<T, W, kWide, INTERLEAVED, BACKWARD>(a, s);
  if constexpr (kWide == 8)
    if (fits(a, INTERLEAVED, BACKWARD, 4, sizeof(T))) return by_lanes<T, W, 4, INTERLEAVED, BACKWARD>(a, s);
  return by_lanes<T, W, 1, INTERLEAVED, BACKWARD>(a, s);
}

template <class T, class W>
cudaError_t by_kind(bool backward, bool interleaved, const QkArgs& a, cudaStream_t s) {
  if (backward) return interleaved ? by_vector<T, W, true, true>(a, s) : by_vector<T, W, false, true>(a, s);
  return interleaved ? by_vector<T, W, true, false>(a, s) : by_vector<T, W, false, false>(a, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, int wdtype, bool backward, bool interleaved, const QkArgs& a, cudaStream_t s) {
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    return wdtype == F32 ? by_kind<T, float>(backward, interleaved, a, s) : by_kind<T, T>(backward, interleaved, a, s);
  });
}

}  // namespace ar
