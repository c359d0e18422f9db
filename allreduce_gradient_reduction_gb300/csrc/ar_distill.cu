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
// in shared memory or still in L2 (four blocks on each of 152 multiprocessors
// have 61 MB of such rows in flight, under half of L2), so HBM sees one read
// and one write.  The few listed words are corrected afterwards, each computed
// once in binary32 and rounded once.
//
// Measured (device time, share of the measured copy bandwidth): loss of 2048 x
// 50257 f32 66 us, 94%, of 8192 x 30000 f16 109 us, 68%; loss and gradient of
// 8192 x 50257 bf16 343 us, 72% (two exponentials, a maximum and three
// conversions an element: the pipe that has the last two is 44% busy, the
// multiprocessor waits for itself more than for memory), of 4096 x 50257 f32 333
// us, 74%; gradient alone of 1023 x 128003 f16 108 us, 73%, f32 196 us, 80%.
// Lists beyond 88 entries leave room for one block a multiprocessor where rows
// are kept: 8192 x 50257 bf16 with 128 entries 519 us.
#include "ar_ops.cuh"

#include <algorithm>

namespace ar {
namespace {

constexpr int kThreads = 256;
constexpr int kStream = kThreads - 32;  // threads that stream the row, while one warp makes the list
constexpr int kBlocks = 4;    // on a multiprocessor
constexpr int kMaxParts = 8;  // portable cluster size
constexpr float kLog2e = 1.4426950408889634f;

// A softmax's running maximum (of the unscaled logits) and the sum of
// 2^(c (z - m)), c = log2(e) / tau.
struct Stat {
  float m, s;
};

__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return Stat{m, a.s + b.s};  // nothing but -inf (or NaN) so far
  return Stat{m, a.s * exp2_approx((a.m - m) * c) + b.s * exp2_approx((b.m - m) * c)};
}

__device__ __forceinline__ Stat warp_join(Stat a, float c) {
#pragma unroll
  for (int i = 16; i; i >>= 1)
    a = join(a, Stat{__shfl_xor_sync(0xFFFFFFFFu, a.m, i), __shfl_xor_sync(0xFFFFFFFFu, a.s, i)}, c);
  a.s = __shfl_sync(0xFFFFFFFFu, a.s, 0);  // the lanes' sums differ in their last bits
  return a;
}

// The largest element of U vectors.
template <class T, int U>
__device__ __forceinline__ float largest(const uint4 (&p)[U]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u)
      m = fmaxf(m, max3(fmaxf(__uint_as_float(p[u].x), __uint_as_float(p[u].y)), __uint_as_float(p[u].z), __uint_as_float(p[u].w)));
    return m;
  } else {
    uint32_t m[2] = {p[0].x, p[0].y};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[0] = max_pairs<T>(m[0], max_pairs<T>(p[u].x, p[u].z));
      m[1] = max_pairs<T>(m[1], max_pairs<T>(p[u].y, p[u].w));
    }
    float lo, hi;
    split(unpack2<T>(max_pairs<T>(m[0], m[1])), lo, hi);
    return fmaxf(lo, hi);
  }
}

// Takes U vectors in.  With the maximum known first, an element costs one
// fused multiply-add and one exponential; a maximum so large (a type's lowest
// value, as masks have) that c m overflows takes differences instead.
template <class T, int U>
__device__ __forceinline__ void accumulate(Stat& st, const uint4 (&p)[U], float c) {
  const float m = fmaxf(st.m, largest<T, U>(p));
  const float base = m * c;
  Two part[2] = {two(0.f, 0.f), two(0.f, 0.f)};
  if (fabsf(base) < INFINITY) {
    st.s *= exp2_approx(fmaf(st.m, c, -base));
    const Two c2 = two(c, c), base2 = two(-base, -base);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < Pairs<T>::N; ++i) {
        float lo, hi;
        split(fma2(Pairs<T>::get(p[u], i), c2, base2), lo, hi);
        part[i & 1] = add2(part[i & 1], two(exp2_approx(lo), exp2_approx(hi)));
      }
  } else {
    const float from = m == -INFINITY ? 0.f : m;  // nothing but -inf (or NaN) so far
    st.s *= exp2_approx((st.m - from) * c);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < Pairs<T>::N; ++i) {
        float lo, hi;
        split(Pairs<T>::get(p[u], i), lo, hi);
        part[i & 1] = add2(part[i & 1], two(exp2_approx((lo - from) * c), exp2_approx((hi - from) * c)));
      }
  }
  float lo, hi;
  split(add2(part[0], part[1]), lo, hi);
  st.s += lo + hi;
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

// A row's elements as the aligned 16-byte vectors they lie in: with `shift`
// the elements between the vector boundary before the row and its first
// element, vector v holds elements [v N - shift, v N - shift + N).
template <class T>
struct RowVectors {
  static constexpr int N = 16 / sizeof(T);
  const T* row;
  int vocab, shift;
  __device__ RowVectors(const T* r, int n) : row(r), vocab(n), shift((int)(((uintptr_t)r & 15) / sizeof(T))) {}
  __device__ int count() const { return (vocab + shift + N - 1) / N; }
  __device__ int first(int v) const { return v * N - shift; }
  __device__ bool whole(int v) const { return first(v) >= 0 && first(v) + N <= vocab; }
  __device__ uint4 load(int v) const { return *reinterpret_cast<const uint4*>(row + first(v)); }
  // any vector: places outside the row as -inf
  __device__ uint4 some(int v) const {
    if (whole(v)) return load(v);
    Pack<T, N> p;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = first(v) + i;
      p.v[i] = e >= 0 && e < vocab ? row[e] : Conv<T>::down(-INFINITY);
    }
    return *reinterpret_cast<const uint4*>(&p);
  }
};

// What one warp makes of a row's list while the others stream the row.  Arrays
// of `top` in shared memory:
//   word   the word, or -1 for an entry outside the vocabulary
//   logit  the student's logit of the word
//   prob   the teacher's probability
//   sum    the word's probability with all of its entries, for the first of
//          them; -1 for the others (NaN is one that counts)
struct List {
  int* word;
  float *logit, *prob, *sum;
  __device__ List(void* at, int top)
      : word(static_cast<int*>(at)),
        logit(reinterpret_cast<float*>(word + top)),
        prob(logit + top),
        sum(prob + top) {}
};
constexpr int kListBytes = 16;  // for each entry

// sum p (log p - z / tau): the loss is tau^2 times this plus lse.
struct Divergence {
  float value;
  bool some;  // the row has a distribution
};

template <class T, class V>
__device__ __forceinline__ Divergence make_list(const DistillArgs& a, int64_t row, const T* z, int vocab, float inv_tau,
                                                bool gradient, const List& list) {
  const int lane = threadIdx.x & 31, top = a.top;
  const int32_t* index = a.index + row * top;
  const V* value = static_cast<const V*>(a.value) + row * top;
  float tmax = -INFINITY;
  for (int k = lane; k < top; k += 32) {
    const int w = index[k];
    const bool is = w >= 0 && w < vocab;
    const float x = is ? Conv<V>::up(value[k]) * inv_tau : -INFINITY;
    list.word[k] = is ? w : -1;
    list.logit[k] = is ? Conv<T>::up(z[w]) : 0.f;
    list.sum[k] = x;
    tmax = fmaxf(tmax, x);
  }
  tmax = warp_max(tmax);
  if (tmax == -INFINITY) tmax = 0.f;
  float total = 0.f;
  for (int k = lane; k < top; k += 32) total += list.prob[k] = expf(list.sum[k] - tmax);
  total = warp_sum(total);
  const float log_total = logf(total);
  float value_sum = 0.f;
  const bool some = total != 0.f;  // NaN (of a teacher's NaN or +inf) is some, and goes on to the results
  for (int k = lane; k < top; k += 32) {
    const float p = list.prob[k] / total;
    if (some && p != 0.f && list.word[k] >= 0) value_sum += p * ((list.sum[k] - tmax - log_total) - list.logit[k] * inv_tau);
    list.prob[k] = p;
  }
  value_sum = warp_sum(value_sum);
  __syncwarp();
  if (gradient) {
    for (int k = lane; k < top; k += 32) {
      const int w = list.word[k];
      float p = 0.f;
      bool first = w >= 0;
#pragma unroll 8
      for (int j = 0; j < top; ++j)
        if (list.word[j] == w) {
          first = first && j >= k;
          p += list.prob[j];
        }
      list.sum[k] = first ? p : -1.f;
    }
  }
  return Divergence{value_sum, some};
}

// scale tau q for elements of one row.  A 16-bit result hides the rounding of
// a base-2 exponent, an f32 one would show it (about 7e-7 at a probability of
// 2^-17).
template <class T>
struct Gradient {
  float coef, lse, c, inv_tau, base;
  bool plain;
  __device__ Gradient(float coef_, float lse_, float c_, float inv_tau_)
      : coef(coef_), lse(lse_), c(c_), inv_tau(inv_tau_), base(lse_ * kLog2e) {
    plain = fabsf(base) < INFINITY;
  }
  __device__ float one(float x) const {
    if constexpr (sizeof(T) == 4) return coef * expf(fmaf(x, inv_tau, -lse));
    else return coef * (plain ? exp2_approx(fmaf(x, c, -base)) : exp2_approx(fmaf(x, inv_tau, -lse) * kLog2e));
  }
  __device__ uint4 vector(uint4 p) const {
    const Two c2 = two(c, c), base2 = two(-base, -base), coef2 = two(coef, coef);
#pragma unroll
    for (int i = 0; i < Pairs<T>::N; ++i) {
      float lo, hi;
      if (sizeof(T) == 4 || !plain) {
        split(Pairs<T>::get(p, i), lo, hi);
        Pairs<T>::set(p, i, two(one(lo), one(hi)));
      } else {
        split(fma2(Pairs<T>::get(p, i), c2, base2), lo, hi);
        Pairs<T>::set(p, i, mul2(coef2, two(exp2_approx(lo), exp2_approx(hi))));
      }
    }
    return p;
  }
};

// The listed words in [lo, hi), each once.
template <class T>
__device__ __forceinline__ void correct_listed(const List& list, int top, int lo, int hi, int t, int threads,
                                               const Gradient<T>& gradient, T* dz) {
  for (int k = t; k < top; k += threads) {
    const int w = list.word[k];
    if (w >= lo && w < hi && !(list.sum[k] < 0.f))
      dz[w] = Conv<T>::down(gradient.one(list.logit[k]) - gradient.coef * list.sum[k]);
  }
}

// Block b of a row's `parts` blocks takes the b-th share of its vectors.  In
// the forward direction they are one cluster and join their sums there.  The
// block's last warp makes the list.
template <class T, class V, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, kBlocks) distill_kernel(const DistillArgs a, int parts) {
  constexpr int U = 4;  // vectors in flight in each thread
  extern __shared__ __align__(16) uint8_t lists[];
  __shared__ float scratch[32], scratch2[32];
  __shared__ float shared_stat[2];
  __shared__ Divergence divergence;

  const int64_t row = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const int t = threadIdx.x, lane = t & 31, vocab = (int)a.vocab, top = a.top;
  const float tau = a.temperature, c = kLog2e / tau, inv_tau = 1.f / tau;
  const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
  const RowVectors<T> rv(z, vocab);
  const int v0 = (int)((int64_t)rv.count() * part / parts), v1 = (int)((int64_t)rv.count() * (part + 1) / parts);
  const List list(lists, top);
  const bool streams = t < kStream;

  if (!streams) {
    // the student's logits of the listed words are read before anything is
    // written (dlogits may be in the place of the logits)
    const Divergence d = make_list<T, V>(a, row, z, vocab, inv_tau, a.dlogits != nullptr, list);
    if (lane == 0) divergence = d;
  }
  float lse;
  if constexpr (BACKWARD) {
    lse = a.lse[row];
    __syncthreads();
  } else {
    Stat st{-INFINITY, 0.f};
    for (int v = v0 + t; v < v1 && streams; v += U * kStream) {
      if (v + (U - 1) * kStream < v1 && rv.whole(v) && rv.whole(v + (U - 1) * kStream)) {
        uint4 p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) p[u] = rv.load(v + u * kStream);
        accumulate<T, U>(st, p, c);
      } else {
        for (int u = 0; u < U && v + u * kStream < v1; ++u) {
          const uint4 p[1] = {rv.some(v + u * kStream)};
          accumulate<T, 1>(st, p, c);
        }
      }
    }
    st = warp_join(st, c);
    if (lane == 0) scratch[t >> 5] = st.m, scratch2[t >> 5] = st.s;
    __syncthreads();
    st = Stat{-INFINITY, 0.f};
    if (lane < kThreads / 32) st = Stat{scratch[lane], scratch2[lane]};
    st = warp_join(st, c);
    if (parts > 1) {
      if (t == 0) shared_stat[0] = st.m, shared_stat[1] = st.s;
      cluster_barrier();
      st = Stat{cluster_read(&shared_stat[0], 0), cluster_read(&shared_stat[1], 0)};
      for (int r = 1; r < parts; ++r) st = join(st, Stat{cluster_read(&shared_stat[0], r), cluster_read(&shared_stat[1], r)}, c);
      cluster_barrier();  // a block's shared memory outlives the others' reads of it
    }
    lse = st.m / tau + logf(st.s);
    if (part == 0 && t == 0) {
      a.loss[row] = divergence.some ? (divergence.value + lse) * tau * tau : 0.f;
      a.lse[row] = lse;
    }
    if (!a.dlogits) return;
  }

  const float scale = a.scale ? a.scale[row] : 1.f;
  const bool live = divergence.some && scale != 0.f;
  const Gradient<T> gradient(scale * tau, lse, c, inv_tau);
  T* dz = static_cast<T*>(a.dlogits) + row * a.dlogits_stride;
  const bool same = (((uintptr_t)dz ^ (uintptr_t)z) & 15) == 0;
  auto vector = [&](const uint4& p) { return live ? gradient.vector(p) : make_uint4(0, 0, 0, 0); };
  for (int v = v0 + t; v < v1; v += U * kThreads) {
    if (same && v + (U - 1) * kThreads < v1 && rv.whole(v) && rv.whole(v + (U - 1) * kThreads)) {
      uint4 p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) p[u] = rv.load(v + u * kThreads);
#pragma unroll
      for (int u = 0; u < U; ++u) *reinterpret_cast<uint4*>(dz + rv.first(v + u * kThreads)) = vector(p[u]);
    } else {
      for (int u = 0; u < U && v + u * kThreads < v1; ++u) {
        const int e = rv.first(v + u * kThreads);
        const uint4 p = vector(rv.some(v + u * kThreads));
        if (same && rv.whole(v + u * kThreads)) {
          *reinterpret_cast<uint4*>(dz + e) = p;
        } else {
          const Pack<T, 16 / sizeof(T)> q = *reinterpret_cast<const Pack<T, 16 / sizeof(T)>*>(&p);
#pragma unroll
          for (int i = 0; i < RowVectors<T>::N; ++i)
            if (e + i >= 0 && e + i < vocab) dz[e + i] = q.v[i];
        }
      }
    }
  }
  if (!live) return;
  __syncthreads();
  correct_listed<T>(list, top, max(rv.first(v0), 0), min(rv.first(v1), vocab), t, kThreads, gradient, dz);
}

// ---- rows through shared memory ----------------------------------------------------
//
// With enough rows to keep every multiprocessor busy, a block takes row after
// row: one warp has pieces of the rows to come copied into shared memory as
// their places become free, so loads never pause, and three make the lists of
// the next rows, each of which takes a chain of dependent loads.  Where both
// the loss and the gradient are wanted and a whole row fits, the second pass
// reads it there; a longer row is copied in twice, the second time from L2.
constexpr int kListWarps = 3;
constexpr int kWorkers = 384;                                  // threads that compute
constexpr int kRingThreads = kWorkers + 32 * kListWarps + 32;  // the last warp loads
constexpr int kPieceVectors = 2 * kWorkers;                    // two to a thread
constexpr int kPieceBytes = kPieceVectors * 16;
constexpr int kMostPieces = 19;
constexpr int kStreamPieces = 7;  // places where a row is not kept: 84 KB, two blocks to a multiprocessor
constexpr int kRingMaxShared = 224 * 1024;

// The loop of a wait that is not over at the first look, out of line (8192 x
// 30000 f16, forward: 113.6 us with it in line, 108.2 us so).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  return ring_wait(bar, parity, gave_up);
}
__device__ __forceinline__ bool wait(uint64_t* bar, int parity, volatile int* gave_up) {
  return ring_try(smem_at(bar), parity) || wait_on(smem_at(bar), parity, gave_up);
}

__device__ __forceinline__ void workers_barrier() { named_barrier(1, kWorkers); }
__device__ __forceinline__ void arrive_on(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(bar)) : "memory");
}

// The place that a sequence of pieces has come to.
struct Place {
  int slot = 0, round = 0;
  __device__ void next(int places) {
    if (++slot == places) slot = 0, ++round;
  }
};

// pieces: to a row; places: of shared memory; keep: a row's pieces stay for a
// second pass (places == pieces then).  The gradient alone is dealt out by
// 2^`split` parts of a row, as its pieces do not depend on one another (0 in
// the forward direction).
template <class T, class V, bool BACKWARD>
__global__ void __launch_bounds__(kRingThreads, 2)
    distill_ring_kernel(const DistillArgs a, int pieces, int places, bool keep, int split) {
  constexpr int VN = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t buffer[];  // the places, then the lists
  __shared__ Stat scratch[2][32];
  __shared__ Divergence divergence[kListWarps];
  __shared__ __align__(8) uint64_t filled[kMostPieces], empty[kMostPieces], list_made[kListWarps], list_used[kListWarps];
  __shared__ int gave_up;

  const int t = threadIdx.x, lane = t & 31, vocab = (int)a.vocab, top = a.top;
  const float tau = a.temperature, c = kLog2e / tau, inv_tau = 1.f / tau;
  const T* logits = static_cast<const T*>(a.logits);
  const bool twice = !BACKWARD && a.dlogits;
  const int64_t units = BACKWARD ? a.rows << split : a.rows;
  auto row_of = [&](int64_t unit) { return BACKWARD ? unit >> split : unit; };
  auto part_of = [&](int64_t unit) { return BACKWARD ? (int)unit & ((1 << split) - 1) : 0; };
  // the pieces of a part of a row: from edge(part) to edge(part + 1)
  auto edge = [&](int part) { return BACKWARD ? pieces * part >> split : pieces * part; };
  auto list_of = [&](int i) { return List(buffer + places * kPieceBytes + i * kListBytes * top, top); };
  auto init = [](uint64_t* bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(bar)), "r"(count) : "memory");
  };
  if (t == 0) {
    gave_up = 0;
    for (int i = 0; i < places; ++i) {
      init(&filled[i], 1);
      init(&empty[i], kWorkers / 32);
    }
    for (int i = 0; i < kListWarps; ++i) {
      init(&list_made[i], 1);
      init(&list_used[i], kWorkers / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (t >= kRingThreads - 32) {
    // ---- loads
    if (lane == 0) {
      Place at;
      for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const T* z = logits + row_of(unit) * a.logits_stride;
        const int begin = edge(part_of(unit)), end = edge(part_of(unit) + 1);
        const uint8_t* from = reinterpret_cast<const uint8_t*>((uintptr_t)z & ~(uintptr_t)15);
        const int bytes = (int)covering(z, vocab * (int)sizeof(T));
        for (int pass = 0; pass < (twice && !keep ? 2 : 1); ++pass)
          for (int i = begin; i < end; ++i, at.next(places)) {
            if (at.round > 0 && !wait(&empty[at.slot], (at.round - 1) & 1, &gave_up)) return;
            // rows that begin at other places in their first word may have a piece less
            const int n = min(kPieceBytes, bytes - i * kPieceBytes);
            const uint32_t bar = smem_at(&filled[at.slot]);
            ring_expect(bar, max(n, 0));
            if (n > 0) ring_copy(smem_at(buffer + at.slot * kPieceBytes), from + i * kPieceBytes, n, bar);
          }
      }
    }
    return;
  }
  if (t >= kWorkers) {
    // ---- lists: warp i makes those of the block's rows (or parts) i, i + 3, ...
    const int i = (t - kWorkers) >> 5;
    int round = 0;
    for (int64_t unit = blockIdx.x + (int64_t)i * gridDim.x; unit < units; unit += (int64_t)kListWarps * gridDim.x, ++round) {
      const int64_t row = row_of(unit);
      if (round > 0) wait(&list_used[i], (round - 1) & 1, &gave_up);
      const Divergence d = make_list<T, V>(a, row, logits + row * a.logits_stride, vocab, inv_tau, a.dlogits != nullptr, list_of(i));
      if (lane == 0) divergence[i] = d;
      __syncwarp();
      if (lane == 0) arrive_on(&list_made[i]);
    }
    return;
  }

  Place at, list_at;
  int turn = 0;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x, turn ^= 1, list_at.next(kListWarps)) {
    const int64_t row = row_of(unit);
    const int begin = edge(part_of(unit)), end = edge(part_of(unit) + 1);
    const T* z = logits + row * a.logits_stride;
    const RowVectors<T> rv(z, vocab);
    const int vecs = rv.count();
    // vector v of the row, from piece `piece`; places outside the row as -inf
    auto vector_at = [&](const uint8_t* piece, int v, int in_piece) {
      uint4 raw = *reinterpret_cast<const uint4*>(piece + in_piece * 16);
      if (!rv.whole(v)) {
        Pack<T, VN> p = *reinterpret_cast<const Pack<T, VN>*>(&raw);
#pragma unroll
        for (int i = 0; i < VN; ++i)
          if (rv.first(v) + i < 0 || rv.first(v) + i >= vocab) p.v[i] = Conv<T>::down(-INFINITY);
        raw = *reinterpret_cast<const uint4*>(&p);
      }
      return raw;
    };
    auto release = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) arrive_on(bar);
    };

    float lse;
    if constexpr (BACKWARD) {
      lse = a.lse[row];
    } else {
      Stat st{-INFINITY, 0.f};
      Place p1 = at;
      for (int i = begin; i < end; ++i, p1.next(places)) {
        wait(&filled[p1.slot], p1.round & 1, &gave_up);
        const uint8_t* piece = buffer + p1.slot * kPieceBytes;
        const int v = i * kPieceVectors + t;
        if (v + kWorkers < vecs) {
          const uint4 p[2] = {vector_at(piece, v, t), vector_at(piece, v + kWorkers, t + kWorkers)};
          accumulate<T, 2>(st, p, c);
        } else if (v < vecs) {
          const uint4 p[1] = {vector_at(piece, v, t)};
          accumulate<T, 1>(st, p, c);
        }
        if (!keep) release(&empty[p1.slot]);
      }
      if (!keep) at = p1;
      st = warp_join(st, c);
      if (lane == 0) scratch[turn][t >> 5] = st;
      workers_barrier();
      st = lane < kWorkers / 32 ? scratch[turn][lane] : Stat{-INFINITY, 0.f};
      st = warp_join(st, c);
      lse = st.m / tau + logf(st.s);
    }
    wait(&list_made[list_at.slot], list_at.round & 1, &gave_up);
    const Divergence d = divergence[list_at.slot];
    if (!BACKWARD && t == 0) {
      a.loss[row] = d.some ? (d.value + lse) * tau * tau : 0.f;
      a.lse[row] = lse;
    }
    if (!BACKWARD && !a.dlogits) {
      release(&list_used[list_at.slot]);
      continue;
    }

    const float scale = a.scale ? a.scale[row] : 1.f;
    const bool live = d.some && scale != 0.f;
    const Gradient<T> gradient(scale * tau, lse, c, inv_tau);
    T* dz = static_cast<T*>(a.dlogits) + row * a.dlogits_stride;
    const bool same = (((uintptr_t)dz ^ (uintptr_t)z) & 15) == 0;
    for (int i = begin; i < end; ++i, at.next(places)) {
      if (BACKWARD || !keep) wait(&filled[at.slot], at.round & 1, &gave_up);
      const uint8_t* piece = buffer + at.slot * kPieceBytes;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int v = i * kPieceVectors + u * kWorkers + t;
        if (v >= vecs) break;
        const uint4 p = live ? gradient.vector(vector_at(piece, v, u * kWorkers + t)) : make_uint4(0, 0, 0, 0);
        const int e = rv.first(v);
        if (same && rv.whole(v)) {
          *reinterpret_cast<uint4*>(dz + e) = p;
        } else {
          const Pack<T, VN> q = *reinterpret_cast<const Pack<T, VN>*>(&p);
#pragma unroll
          for (int x = 0; x < VN; ++x)
            if (e + x >= 0 && e + x < vocab) dz[e + x] = q.v[x];
        }
      }
      release(&empty[at.slot]);
    }
    workers_barrier();
    if (live)
      correct_listed<T>(list_of(list_at.slot), top, max(rv.first(begin * kPieceVectors), 0),
                        min(rv.first(end * kPieceVectors), vocab), t, kWorkers, gradient, dz);
    release(&list_used[list_at.slot]);
  }
}

template <class T, class V, bool BACKWARD>
cudaError_t run(const DistillArgs& a, cudaStream_t s) {
  // Through shared memory where there are more rows than the other kernel has
  // in flight at once (50257 words in bf16, loss and gradient: 600 rows 31.2 us
  // this way and 28.1 the other, 2048 rows 92.9 and 94.7; the gradient alone of
  // 1000 rows 41.8 and 47.5; the loss alone of 600 rows 13.9 and 10.3).
  if (a.rows > kBlocks * sm_count()) {
    auto* kernel = distill_ring_kernel<T, V, BACKWARD>;
    static std::atomic<unsigned long long> opened[256];
    const int64_t row_bytes = (a.vocab * (int64_t)sizeof(T) + 15 + 15) / 16 * 16;
    const int lists = kListWarps * kListBytes * a.top;
    const int pieces = (int)((row_bytes + kPieceBytes - 1) / kPieceBytes);
    const bool keep = !BACKWARD && a.dlogits && pieces <= kMostPieces && pieces * kPieceBytes + lists <= kRingMaxShared;
    const int places = keep ? pieces : std::min(pieces, kStreamPieces);
    const int shared = places * kPieceBytes + lists;
    cudaError_t e = open_kernel((const void*)kernel, kRingMaxShared, false, opened);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kRingThreads, (size_t)shared)) != cudaSuccess) return e;
    // What the blocks that finish last leave idle: whole rows to a block where
    // that is under 4%, else halves or quarters with at least four pieces
    // (1023 x 128003 f16, 3.4 rows to a block: 109.5 us by rows, 105 us by
    // quarters; each part makes the row's list again).
    const int64_t most = (int64_t)sm_count() * std::max(per_sm, 1);
    int split = 0;
    auto idle = [&] {
      const int64_t units = a.rows << split, turns = (units + most - 1) / most;
      return (double)(turns * most - units) / (double)(turns * most);
    };
    if (BACKWARD)
      while (split < 2 && pieces >> split >= 8 && idle() > 0.04) ++split;
    const int64_t blocks = std::min<int64_t>(a.rows << split, most);
    kernel<<<(unsigned)blocks, kRingThreads, (size_t)shared, s>>>(a, pieces, places, keep, split);
    note_launch();
    return cudaGetLastError();
  }
  // Few rows: several blocks to a row, until there are about two for each
  // multiprocessor, each with 4096 words or more (loss and gradient, bf16: 6
  // rows of 50257 words in eight parts 8.2 us, in one 12.5; 6 rows of 5003 in
  // four 6.2 us, in one 5.3).
  int parts = 1;
  while (parts < kMaxParts && a.rows * parts * 2 <= 2 * sm_count() && a.vocab / (parts * 2) >= 4096) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)kListBytes * a.top;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = parts;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = !BACKWARD && parts > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, distill_kernel<T, V, BACKWARD>, a, parts);
  note_launch();
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

cudaError_t distill_take_status(int* status, cudaStream_t s) { return take_status(status, s); }

}  // namespace ar
