// Distillation from a teacher's top logits, forward and backward.
//
//   p = softmax over a row's listed teacher logits t / tau
//   q = softmax over the vocabulary of the student's logits z / tau
//   loss = tau^2 sum_k p_k (log p_k - log q[i_k])
//   dz   = scale tau (q - sum_k p_k onehot(i_k))
//
// Bound by HBM: the vocabulary row is long (50257 words: 100 KB in bf16) and
// each of its elements needs one exponential a pass.  One block (or, with few
// rows, several) streams a row once with a running maximum and sum; when the
// gradient is wanted too, it goes over the row a second time while the row is
// still in L2 (at four blocks of 512 threads on each of 152 multiprocessors
// 61 MB of rows are in flight, under half of L2), so HBM sees one read and one
// write.  The few listed words are corrected afterwards, each computed once in
// binary32 and rounded once.
#include "ar_ops.cuh"

#include <algorithm>

namespace ar {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxParts = 8;  // portable cluster size
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A softmax's running maximum (of the unscaled logits) and the sum of
// 2^(c (z - m)), c = log2(e) / tau.
struct Stat {
  float m, s;
};

__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return Stat{m, a.s + b.s};  // nothing but -inf (or NaN) so far
  return Stat{m, a.s * exp2_fast((a.m - m) * c) + b.s * exp2_fast((b.m - m) * c)};
}

__device__ __forceinline__ Stat warp_join(Stat a, float c) {
#pragma unroll
  for (int i = 16; i; i >>= 1)
    a = join(a, Stat{__shfl_xor_sync(0xFFFFFFFFu, a.m, i), __shfl_xor_sync(0xFFFFFFFFu, a.s, i)}, c);
  return a;
}

// Takes U vectors in.  With the maximum known first, an element costs one
// fused multiply-add and one exponential; a maximum so large (a type's lowest
// value, as masks have) that c m overflows takes differences instead.
template <class T, int N, int U>
__device__ __forceinline__ void accumulate(Stat& st, const Pack<T, N> (&p)[U], float c) {
  float m = st.m;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, Conv<T>::up(p[u].v[i]));
  const float base = m * c;
  if (fabsf(base) < INFINITY) {
    st.s *= exp2_fast(fmaf(st.m, c, -base));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) st.s += exp2_fast(fmaf(Conv<T>::up(p[u].v[i]), c, -base));
  } else {
    const float from = m == -INFINITY ? 0.f : m;  // nothing but -inf (or NaN) so far
    st.s *= exp2_fast((st.m - from) * c);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) st.s += exp2_fast((Conv<T>::up(p[u].v[i]) - from) * c);
  }
  st.m = m;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ float cluster_read(const float* own, int rank) {
  const unsigned at = static_cast<unsigned>(__cvta_generic_to_shared(own));
  unsigned remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

__device__ __forceinline__ float block_sum(float v, float* scratch) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < kThreads / 32 ? scratch[threadIdx.x & 31] : 0.f);
}

__device__ __forceinline__ float block_max(float v, float* scratch) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_max((threadIdx.x & 31) < kThreads / 32 ? scratch[threadIdx.x & 31] : -INFINITY);
}

// A row's elements as the aligned 16-byte vectors they lie in: with `shift`
// the elements between the vector boundary before the row and its first
// element, vector v holds elements [v N - shift, v N - shift + N).
template <class T, int N>
struct RowVectors {
  const T* row;
  int vocab, shift;
  __device__ RowVectors(const T* r, int n) : row(r), vocab(n), shift((int)(((uintptr_t)r & 15) / sizeof(T))) {}
  __device__ int count() const { return (vocab + shift + N - 1) / N; }
  __device__ int first(int v) const { return v * N - shift; }
  __device__ bool whole(int v) const { return first(v) >= 0 && first(v) + N <= vocab; }
  __device__ Pack<T, N> load(int v) const { return *reinterpret_cast<const Pack<T, N>*>(row + first(v)); }
  // any vector: places outside the row as -inf
  __device__ Pack<T, N> some(int v) const {
    if (whole(v)) return load(v);
    Pack<T, N> p;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = first(v) + i;
      p.v[i] = e >= 0 && e < vocab ? row[e] : Conv<T>::down(-INFINITY);
    }
    return p;
  }
};

// Block b of a row's `parts` blocks takes the b-th share of its vectors.  In
// the forward direction they are one cluster and join their sums there.
template <class T, class V, bool BACKWARD>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a, int parts) {
  constexpr int N = 16 / sizeof(T);
  constexpr int U = 4;  // vectors in flight in each thread
  __shared__ float prob[kDistillMaxTop], logit[kDistillMaxTop];
  __shared__ int word[kDistillMaxTop];
  __shared__ float scratch[32], scratch2[32];
  __shared__ float shared_stat[2];

  const int64_t row = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const int t = threadIdx.x, vocab = (int)a.vocab, top = a.top;
  const float tau = a.temperature, c2 = kLog2e / tau;
  const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
  const RowVectors<T, N> rv(z, vocab);
  const int v0 = (int)((int64_t)rv.count() * part / parts), v1 = (int)((int64_t)rv.count() * (part + 1) / parts);
  const int lo = max(rv.first(v0), 0), hi = min(rv.first(v1), vocab);  // this block's words

  // the teacher's distribution over the list; entries outside the vocabulary are no entries
  const V* value = static_cast<const V*>(a.value) + row * top;
  float tmax = -INFINITY;
  for (int k = t; k < top; k += kThreads) {
    const int w = a.index[row * top + k];
    const bool there = w >= 0 && w < vocab;
    const float x = there ? Conv<V>::up(value[k]) / tau : -INFINITY;
    word[k] = there ? w : -1;
    prob[k] = x;
    logit[k] = there && (!BACKWARD || (w >= lo && w < hi)) ? Conv<T>::up(z[w]) : 0.f;
    tmax = fmaxf(tmax, x);
  }
  tmax = block_max(tmax, scratch);
  if (tmax == -INFINITY) tmax = 0.f;
  float tsum = 0.f;
  for (int k = t; k < top; k += kThreads) tsum += expf(prob[k] - tmax);
  tsum = block_sum(tsum, scratch);
  const bool some = tsum > 0.f;
  const float log_tsum = logf(tsum);

  float lse;
  if constexpr (BACKWARD) {
    lse = a.lse[row];
  } else {
    Stat st{-INFINITY, 0.f};
    for (int v = v0 + t; v < v1; v += U * kThreads) {
      if (v + (U - 1) * kThreads < v1 && rv.whole(v) && rv.whole(v + (U - 1) * kThreads)) {
        Pack<T, N> p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) p[u] = rv.load(v + u * kThreads);
        accumulate<T, N, U>(st, p, c2);
      } else {
        for (int u = 0; u < U && v + u * kThreads < v1; ++u) {
          const Pack<T, N> p[1] = {rv.some(v + u * kThreads)};
          accumulate<T, N, 1>(st, p, c2);
        }
      }
    }
    st = warp_join(st, c2);
    __syncthreads();  // the last reads of the scratch are done
    if ((t & 31) == 0) scratch[t >> 5] = st.m, scratch2[t >> 5] = st.s;
    __syncthreads();
    st = Stat{-INFINITY, 0.f};
    if ((t & 31) < kThreads / 32) st = Stat{scratch[t & 31], scratch2[t & 31]};
    st = warp_join(st, c2);
    if (parts > 1) {
      if (t == 0) shared_stat[0] = st.m, shared_stat[1] = st.s;
      cluster_barrier();
      st = Stat{cluster_read(&shared_stat[0], 0), cluster_read(&shared_stat[1], 0)};
      for (int r = 1; r < parts; ++r) st = join(st, Stat{cluster_read(&shared_stat[0], r), cluster_read(&shared_stat[1], r)}, c2);
      cluster_barrier();  // a block's shared memory outlives the others' reads of it
    }
    lse = st.m / tau + logf(st.s);
    if (part == 0) {
      float l = 0.f;
      for (int k = t; k < top; k += kThreads) {
        const float lp = prob[k] - tmax - log_tsum, p = expf(prob[k] - tmax) / tsum;
        if (some && p > 0.f) l += p * (lp - (logit[k] / tau - lse));
      }
      l = block_sum(l, scratch);
      if (t == 0) {
        a.loss[row] = l * tau * tau;
        a.lse[row] = lse;
      }
    }
    if (!a.dlogits) return;
  }

  const float scale = a.scale ? a.scale[row] : 1.f;
  const float coef = scale * tau;
  const bool live = some && scale != 0.f;
  const float base = lse * kLog2e, inv_tau = 1.f / tau;
  // q scaled: a 16-bit result hides the rounding of a base-2 exponent, an f32
  // one would show it (about 7e-7 at a probability of 2^-17)
  auto q_of = [&](float x) {
    if constexpr (sizeof(T) == 4) return expf(fmaf(x, inv_tau, -lse));
    else return fabsf(base) < INFINITY ? exp2_fast(fmaf(x, c2, -base)) : exp2_fast(fmaf(x, inv_tau, -lse) * kLog2e);
  };
  auto gradient = [&](float x) { return coef * q_of(x); };
  T* dz = static_cast<T*>(a.dlogits) + row * a.dlogits_stride;
  const bool same = (((uintptr_t)dz ^ (uintptr_t)z) & 15) == 0;
  // with dlogits in the place of the logits, every listed logit has been read by now
  __syncthreads();
  for (int v = v0 + t; v < v1; v += U * kThreads) {
    if (same && v + (U - 1) * kThreads < v1 && rv.whole(v) && rv.whole(v + (U - 1) * kThreads)) {
      Pack<T, N> p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) p[u] = rv.load(v + u * kThreads);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          p[u].v[i] = Conv<T>::down(live ? gradient(Conv<T>::up(p[u].v[i])) : 0.f);
        *reinterpret_cast<Pack<T, N>*>(dz + rv.first(v + u * kThreads)) = p[u];
      }
    } else {
      for (int u = 0; u < U && v + u * kThreads < v1; ++u) {
        const int e = rv.first(v + u * kThreads);
        Pack<T, N> p = rv.some(v + u * kThreads);
#pragma unroll
        for (int i = 0; i < N; ++i) p.v[i] = Conv<T>::down(live ? gradient(Conv<T>::up(p.v[i])) : 0.f);
        if (same && rv.whole(v + u * kThreads)) {
          *reinterpret_cast<Pack<T, N>*>(dz + e) = p;
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (e + i >= 0 && e + i < vocab) dz[e + i] = p.v[i];
        }
      }
    }
  }
  if (!live) return;
  __syncthreads();
  // the listed words of this block's share: a word listed more than once is
  // corrected by its first entry, with the sum of all of them in list order
  for (int k = t; k < top; k += kThreads) {
    const int w = word[k];
    if (w < lo || w >= hi) continue;
    float p = 0.f;
    bool first = true;
    for (int j = 0; j < top; ++j)
      if (word[j] == w) {
        if (j < k) first = false;
        p += expf(prob[j] - tmax) / tsum;
      }
    if (first) dz[w] = Conv<T>::down(coef * (q_of(logit[k]) - p));
  }
}

template <class T, class V, bool BACKWARD>
cudaError_t run(const DistillArgs& a, cudaStream_t s) {
  // Few rows: several blocks to a row, until there are about two blocks for
  // each multiprocessor.
  int parts = 1;
  while (parts < kMaxParts && a.rows * parts * 2 <= 2 * sm_count() && a.vocab / (parts * 2) >= 4 * kThreads) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = parts;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = !BACKWARD && parts > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, distill_kernel<T, V, BACKWARD>, a, parts);
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_distill(int dtype, int vdtype, bool backward, const DistillArgs& a, cudaStream_t s) {
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    if (vdtype == F32) return backward ? run<T, float, true>(a, s) : run<T, float, false>(a, s);
    return backward ? run<T, T, true>(a, s) : run<T, T, false>(a, s);
  });
}

}  // namespace ar
