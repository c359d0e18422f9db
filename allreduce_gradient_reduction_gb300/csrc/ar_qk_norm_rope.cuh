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
// of a pair in the same lane, so that the rotation exchanges nothing; a warp has
// as many heads at a time as it has groups (a round).  All rounds of all tokens,
// of the queries by some blocks and of the keys by others, are dealt out to the
// warps evenly.  A warp keeps the weights, the current token's angles and
// its part of the weights' gradients in registers and works in pairs of binary32
// values.  The next rounds are copied into shared memory meanwhile, each lane's
// own vectors into places of its own, so that nothing but its own copies is
// waited for (kept in registers, one round ahead, they left the gradient of
// 16384 tokens at 158 us: the compiler has no room to load early).
//
// Angles: the frequency is a 64-bit fraction of a turn, so the product with the
// position, modulo one turn, is an integer product that loses nothing (a
// frequency is off by 2^-65 turns at most, at position 2^31 by 2^-34).  The top
// two bits after rounding are the quarter; what is left is at most an eighth of
// a turn, for which Taylor's series to x^9 and x^10 are within 2e-9.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

#include "ar_ops.cuh"

namespace ar {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Blocks on a multiprocessor: a lane's eight pairs of weights, angles and sums take
// 128 registers backward; forward three were slower (61 us where two take 59).
constexpr int kResident = 2;
// Tokens to a warp from which on warps take whole ones, every `warps`-th.
constexpr int kMany = 4;

__device__ __forceinline__ void cos_sin(int32_t position, uint64_t turn, float& c, float& s) {
  const uint64_t angle = (uint64_t)(int64_t)position * turn;
  const uint64_t round = angle + (1ull << 61);
  const uint32_t quarter = (uint32_t)(round >> 62);
  // what is left of the turn, in [-1/8, 1/8), to 34 bits after the point
  const int32_t rest = (int32_t)((uint32_t)(round >> 30) ^ 0x80000000u);
  const float x = (float)rest * (float)(6.283185307179586 / 17179869184.0);
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
  // Where the vectors of pair p (a multiple of VEC) are.  With neighbours paired,
  // one in each half of the head, so that neighbouring lanes' lie side by side;
  // else the first half of what is rotated pairs with the second, and so does the
  // first half of the rest with its second.
  static __device__ __forceinline__ void places(const QkArgs& a, int p, int& lo, int& hi) {
    if constexpr (INTERLEAVED) {
      lo = VEC == 1 ? 2 * p : p;
      hi = VEC == 1 ? 2 * p + 1 : p + a.dim / 2;
    } else {
      const int half = a.rotary / 2;
      const bool turned = p < half;
      lo = turned ? p : p + half;
      hi = lo + (turned ? half : (a.dim - a.rotary) / 2);
    }
  }
  // The lane's i-th pair.
  static __device__ __forceinline__ int pair_of(const QkArgs& a, int lane, int i) {
    const int p = pair(lane, i / VEC);
    if (!INTERLEAVED || VEC == 1) return p + i % VEC;
    return p / 2 + (i < VEC / 2 ? i : a.dim / 4 + i - VEC / 2);
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
  // The same by way of shared memory: two vectors of a lane, `apart` from each
  // other.  Only the lane that copied them reads them.
  static constexpr bool kCopied = VEC > 1;
  static __device__ __forceinline__ void copy(const QkArgs& a, const T* row, int lane, uint32_t to, uint32_t apart) {
    if (pair(lane, 0) >= a.dim / 2) return;
    int lo, hi;
    places(a, pair(lane, 0), lo, hi);
    auto one = [](uint32_t to, const T* from) {
      if constexpr (sizeof(P) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"((int)sizeof(P)) : "memory");
    };
    one(to, row + lo);
    one(to + apart, row + hi);
  }
  static __device__ __forceinline__ Raw copied(const QkArgs& a, int lane, const uint8_t* from, uint32_t apart) {
    Raw r;
    r.lo[0] = r.hi[0] = zero_pack<T, VEC>();
    if (pair(lane, 0) < a.dim / 2) {
      r.lo[0] = *reinterpret_cast<const P*>(from);
      r.hi[0] = *reinterpret_cast<const P*>(from + apart);
    }
    return r;
  }
  // Elements e and e + 1 of a vector, e even: 16-bit ones are one word.
  static __device__ __forceinline__ Two get(const P& p, int e) {
    if constexpr (sizeof(T) == 2) return unpack2<T>(reinterpret_cast<const uint32_t*>(p.v)[e / 2]);
    else return two(p.v[e], p.v[e + 1]);
  }
  static __device__ __forceinline__ void set(P& p, int e, float x, float y) {
    if constexpr (sizeof(T) == 2) reinterpret_cast<uint32_t*>(p.v)[e / 2] = pack2<T>(x, y);
    else p.v[e] = x, p.v[e + 1] = y;
  }
  // The lane's pairs (a, b), two at a time.
  static __device__ __forceinline__ void widen(const Raw& r, Two (&a)[kPairs / 2], Two (&b)[kPairs / 2]) {
#pragma unroll
    for (int i = 0; i < kPairs; i += 2) {
      if constexpr (VEC == 1) {
        a[i / 2] = two(Conv<T>::up(r.lo[i].v[0]), Conv<T>::up(r.lo[i + 1].v[0]));
        b[i / 2] = two(Conv<T>::up(r.hi[i].v[0]), Conv<T>::up(r.hi[i + 1].v[0]));
      } else if constexpr (!INTERLEAVED) {
        a[i / 2] = get(r.lo[i / VEC], i % VEC);
        b[i / 2] = get(r.hi[i / VEC], i % VEC);
      } else {
        const int e = 2 * (i % VEC);
        const P& p = e < VEC ? r.lo[i / VEC] : r.hi[i / VEC];
        float a0, b0, a1, b1;
        split(get(p, e % VEC), a0, b0);
        split(get(p, e % VEC + 2), a1, b1);
        a[i / 2] = two(a0, a1);
        b[i / 2] = two(b0, b1);
      }
    }
  }
  static __device__ __forceinline__ void store(const QkArgs& args, T* row, int lane, const Two (&a)[kPairs / 2],
                                               const Two (&b)[kPairs / 2]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < kPairs; i += 2) {
      float a0, b0, a1, b1;
      split(a[i / 2], a0, a1);
      split(b[i / 2], b0, b1);
      if constexpr (VEC == 1) {
        r.lo[i].v[0] = Conv<T>::down(a0);
        r.lo[i + 1].v[0] = Conv<T>::down(a1);
        r.hi[i].v[0] = Conv<T>::down(b0);
        r.hi[i + 1].v[0] = Conv<T>::down(b1);
      } else if constexpr (!INTERLEAVED) {
        set(r.lo[i / VEC], i % VEC, a0, a1);
        set(r.hi[i / VEC], i % VEC, b0, b1);
      } else {
        const int e = 2 * (i % VEC);
        P& p = e < VEC ? r.lo[i / VEC] : r.hi[i / VEC];
        set(p, e % VEC, a0, b0);
        set(p, e % VEC + 2, a1, b1);
      }
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (pair(lane, c) >= args.dim / 2) continue;
      int lo, hi;
      places(args, pair(lane, c), lo, hi);
      *reinterpret_cast<P*>(row + lo) = r.lo[c];
      *reinterpret_cast<P*>(row + hi) = r.hi[c];
    }
  }
};

// Where the first or second element of pair p lies in a head.
template <bool INTERLEAVED>
__device__ __forceinline__ int element(const QkArgs& a, int p, bool second) {
  if (INTERLEAVED) return 2 * p + second;
  const int half = a.rotary / 2;
  return p < half ? p + (second ? half : 0) : p + half + (second ? (a.dim - a.rotary) / 2 : 0);
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

// A warp's ring of rounds: [round][x lo, x hi, dy lo, dy hi][lane].
constexpr int kAhead = 4;
template <class T, int VEC, bool BACKWARD>
struct Ring {
  static constexpr uint32_t kVector = VEC * sizeof(T), kApart = 32 * kVector, kBytes = (BACKWARD ? 4 : 2) * kApart;
  static constexpr uint32_t kWarpBytes = kAhead * kBytes;
};

// The pairs' turns, no more than a kernel's heads have: with 1 KB of them a
// call of 3 tokens takes the host 14.0 us, with 256 bytes 12.9.
template <int PAIRS>
struct Turns {
  uint64_t of[PAIRS];
};

// The first `q_blocks` blocks take the queries, the others the keys.
template <class T, class W, int VEC, int LANES, int CHUNKS, bool INTERLEAVED, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, kResident)
    qk_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ Turns<VEC * LANES * CHUNKS> turn, int q_blocks) {
  using H = Head<T, VEC, LANES, CHUNKS, INTERLEAVED>;
  constexpr int kGroups = 32 / LANES, kPairs = H::kPairs, kTwos = kPairs / 2,
                kMaxPairs = VEC * LANES * CHUNKS;
  __shared__ uint64_t turns[kMaxPairs];
  const int lane = threadIdx.x % LANES, group = threadIdx.x % 32 / LANES;
  const int t = (int)blockIdx.x >= q_blocks;  // which tensor
  const int heads = a.heads[t], rounds = (heads + kGroups - 1) / kGroups;

  // The warp's rounds: a run of them, or those of every `warps`-th token, so that
  // neighbouring warps read neighbouring rows at a time (16384 tokens, 32:8 heads
  // of 128 bf16: forward 59 us and 62 in runs, backward 89 and 94).
  const int64_t all = a.tokens * rounds, warps = (int64_t)(t ? gridDim.x - q_blocks : q_blocks) * kWarps;
  const int64_t warp = (int64_t)(blockIdx.x - (t ? q_blocks : 0)) * kWarps + threadIdx.x / 32;
  const int64_t each = all / warps, over = all - each * warps;
  int left = (int)(each + (warp < over));  // (rows of two elements or more in memory: fewer than 2^31 to a warp)
  const int64_t begin = warp * each + min(warp, over);
  int64_t token = begin / rounds, hop = 1;
  int head = (int)(begin - token * rounds) * kGroups + group;
  if (a.tokens >= kMany * warps) {
    token = warp;
    hop = warps;
    head = group;
    left = (int)((a.tokens - warp + warps - 1) / warps) * rounds;
  }

  // Rounds on their way: a ring of kAhead in shared memory, or one in registers
  // where a vector is too short for that.  A group without a head in a round
  // leaves what was there, which is not used.
  using Slot = Ring<T, VEC, BACKWARD>;
  extern __shared__ __align__(16) uint8_t ring[];
  uint8_t* const slots = ring + (threadIdx.x / 32) * Slot::kWarpBytes + threadIdx.x % 32 * Slot::kVector;
  typename H::Raw x_next = {}, dy_next = {};
  int head_ahead = head, left_ahead = left, slot_ahead = 0, slot = 0;
  const int last = rounds * kGroups + group;  // one past the group's last
  // From one round to the next, and from a token's last to its next token's first.
  auto place = [&](const QkTensor& of) { return token * of.token_stride + head * of.head_stride; };
  auto across = [&](const QkTensor& of) { return kGroups * of.head_stride; };
  auto down = [&](const QkTensor& of) { return hop * of.token_stride - (int64_t)(rounds - 1) * kGroups * of.head_stride; };
  const T* from = static_cast<const T*>(a.x[t].ptr) + place(a.x[t]);
  const T* dfrom = static_cast<const T*>(a.dy[t].ptr) + (BACKWARD ? place(a.dy[t]) : 0);
  T* to_row = static_cast<T*>(const_cast<void*>(a.y[t].ptr)) + place(a.y[t]);
  const int64_t x_across = across(a.x[t]), x_down = down(a.x[t]), dy_across = across(a.dy[t]), dy_down = down(a.dy[t]),
                y_across = across(a.y[t]), y_down = down(a.y[t]);
  auto fetch = [&]() {
    if (left_ahead > 0 && head_ahead < heads) {
      if constexpr (H::kCopied) {
        const uint32_t to = smem_at(slots) + slot_ahead * Slot::kBytes;
        H::copy(a, from, lane, to, Slot::kApart);
        if (BACKWARD) H::copy(a, dfrom, lane, to + 2 * Slot::kApart, Slot::kApart);
      } else {
        x_next = H::load(a, from, lane);
        if (BACKWARD) dy_next = H::load(a, dfrom, lane);
      }
    }
    if constexpr (H::kCopied) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      slot_ahead = slot_ahead + 1 == kAhead ? 0 : slot_ahead + 1;
    }
    --left_ahead;
    head_ahead += kGroups;
    const bool wrap = head_ahead >= last;
    if (wrap) head_ahead = group;
    from += wrap ? x_down : x_across;
    if (BACKWARD) dfrom += wrap ? dy_down : dy_across;
  };
  for (int i = 0; i < (H::kCopied ? kAhead - 1 : 1); ++i) fetch();
  int32_t position = left ? a.positions[token] : 0;
  for (int i = threadIdx.x; i < kMaxPairs; i += kThreads) turns[i] = i < a.rotary / 2 ? turn.of[i] : 0;
  Two wa[kTwos], wb[kTwos];
  {
    const W* w = static_cast<const W*>(a.weight[t]);
    auto at = [&](int i, bool second) {
      const int p = H::pair_of(a, lane, i);
      return w && H::pair(lane, i / VEC) < a.dim / 2 ? Conv<W>::up(w[element<INTERLEAVED>(a, p, second)]) : 1.f;
    };
#pragma unroll
    for (int i = 0; i < kPairs; i += 2) {
      wa[i / 2] = two(at(i, false), at(i + 1, false));
      wb[i / 2] = two(at(i, true), at(i + 1, true));
    }
  }
  __syncthreads();

  constexpr int kSums = BACKWARD ? kTwos : 1;
  Two sum_a[kSums], sum_b[kSums];  // of the weight's gradient
#pragma unroll
  for (int i = 0; i < kSums; ++i) sum_a[i] = sum_b[i] = two(0.f, 0.f);
  Two cs[kTwos], sn[kTwos];
  const float mean = 1.f / (float)a.dim;
  for (bool turned = true; left; --left) {
    if (turned) {
      // another token: its angles, for all of its heads.  The groups have the same
      // pairs, so each takes a part of them and they exchange what they made.
      constexpr int kEach = (kPairs + kGroups - 1) / kGroups;
      float c[kEach], s[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = min(group * kEach, kPairs - kEach) + j;
        cos_sin(position, turns[min(H::pair_of(a, lane, i), kMaxPairs - 1)], c[j], s[j]);
        if (BACKWARD) s[j] = -s[j];  // backward turns the other way
      }
#pragma unroll
      for (int i = 0; i < kPairs; i += 2) {
        auto of = [&](const float (&v)[kEach], int i) {
          return kGroups == 1 ? v[i % kEach] : __shfl_sync(0xFFFFFFFFu, v[i % kEach], i / kEach * LANES + lane);
        };
        cs[i / 2] = two(of(c, i), of(c, i + 1));
        sn[i / 2] = two(of(s, i), of(s, i + 1));
      }
      if (token + hop < a.tokens) position = a.positions[token + hop];
    }
    Two xa[kTwos], xb[kTwos], ga[kTwos], gb[kTwos];
    if constexpr (H::kCopied) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
      const uint8_t* at = slots + slot * Slot::kBytes;
      slot = slot + 1 == kAhead ? 0 : slot + 1;
      x_next = H::copied(a, lane, at, Slot::kApart);
      if (BACKWARD) dy_next = H::copied(a, lane, at + 2 * Slot::kApart, Slot::kApart);
    }
    H::widen(x_next, xa, xb);
    if (BACKWARD) H::widen(dy_next, ga, gb);
    fetch();
    const int now = head;
    T* const to = to_row;
    head += kGroups;
    turned = head >= last;
    if (turned) {
      token += hop;
      head = group;
    }
    to_row += turned ? y_down : y_across;

    Two acc = two(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kTwos; ++i) acc = fma2(xa[i], xa[i], fma2(xb[i], xb[i], acc));
    float lo, hi;
    split(acc, lo, hi);
    const float squares = lo + hi;
    // (a, b) turned: a cos - b sin, b cos + a sin
    auto turn = [&](Two& p, Two& q, int i) {
      const Two less = neg2(sn[i]);
      const Two u = fma2(q, less, mul2(p, cs[i]));
      q = fma2(p, sn[i], mul2(q, cs[i]));
      p = u;
    };
    if constexpr (!BACKWARD) {
      const float rstd = rsqrtf(fmaf(group_sum<LANES>(squares), mean, a.eps));
      const Two r = two(rstd, rstd);
#pragma unroll
      for (int i = 0; i < kTwos; ++i) {
        xa[i] = mul2(mul2(xa[i], r), wa[i]);
        xb[i] = mul2(mul2(xb[i], r), wb[i]);
        turn(xa[i], xb[i], i);
      }
    } else {
      acc = two(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kTwos; ++i) {
        turn(ga[i], gb[i], i);
        acc = fma2(mul2(ga[i], wa[i]), xa[i], fma2(mul2(gb[i], wb[i]), xb[i], acc));
      }
      split(acc, lo, hi);
      const float rstd = rsqrtf(fmaf(group_sum<LANES>(squares), mean, a.eps));
      const float back = group_sum<LANES>(lo + hi) * mean * rstd * rstd;
      const Two r = two(rstd, rstd), less = two(-back, -back);
      if (now < heads) {
#pragma unroll
        for (int i = 0; i < kTwos; ++i) {
          sum_a[i] = fma2(ga[i], mul2(xa[i], r), sum_a[i]);
          sum_b[i] = fma2(gb[i], mul2(xb[i], r), sum_b[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kTwos; ++i) {
        xa[i] = mul2(r, fma2(xa[i], less, mul2(ga[i], wa[i])));
        xb[i] = mul2(r, fma2(xb[i], less, mul2(gb[i], wb[i])));
      }
    }
    if (now < heads) H::store(a, to, lane, xa, xb);
  }

  if constexpr (BACKWARD) {
    if (!a.partial) return;
    // the block's sums in a fixed order: over the groups of each warp, then warp after warp
    __shared__ float warp_sums[kWarps][kQkMaxDim];
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float lo, hi;
        split(e ? sum_b[i / 2] : sum_a[i / 2], lo, hi);
        float v = i & 1 ? hi : lo;
#pragma unroll
        for (int m = LANES; m < 32; m <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
        const int p = H::pair_of(a, lane, i);
        if (group == 0 && H::pair(lane, i / VEC) < a.dim / 2) warp_sums[threadIdx.x / 32][element<INTERLEAVED>(a, p, e)] = v;
      }
    __syncthreads();
    for (int d = threadIdx.x; d < a.dim; d += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += warp_sums[w][d];
      a.partial[(int64_t)blockIdx.x * a.dim + d] = v;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
}

// The weights' gradients: sums of their blocks' in order, eight columns to a
// block, 32 rows of threads.
constexpr int kSumCols = 8, kSumRows = 32;
template <class W>
__global__ void __launch_bounds__(kSumCols* kSumRows)
    qk_weight_kernel(const float* partial, int q_blocks, int blocks, int dim, W* dq, W* dk) {
  __shared__ float part[kSumRows][kSumCols];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.y, col = blockIdx.x * kSumCols + threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;
  float v = 0.f;
  if (col < dim)
    for (int b = (t ? q_blocks : 0) + row; b < (t ? blocks : q_blocks); b += kSumRows) v += partial[(int64_t)b * dim + col];
  part[row][threadIdx.x % kSumCols] = v;
  __syncthreads();
  W* to = t ? dk : dq;
  if (row || col >= dim || !to) return;
  v = 0.f;
#pragma unroll
  for (int r = 0; r < kSumRows; ++r) v += part[r][threadIdx.x];
  to[col] = Conv<W>::down(v);
}

template <class W>
cudaError_t sum_weights(const QkArgs& a, int q_blocks, int blocks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.dim + kSumCols - 1) / kSumCols, 2);
  cfg.blockDim = dim3(kSumCols * kSumRows);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, qk_weight_kernel<W>, (const float*)a.partial, q_blocks, blocks, (int)a.dim,
                                           static_cast<W*>(a.dweight[0]), static_cast<W*>(a.dweight[1]));
  note_launch();
  return e;
}

template <class T, class W, int VEC, int LANES, int CHUNKS, bool INTERLEAVED, bool BACKWARD>
cudaError_t run(const QkArgs& a, cudaStream_t s) {
  constexpr int kGroups = 32 / LANES;
  // Blocks in proportion to the tensors' rounds, as many as are resident at a
  // time, or a warp to a round.  A token's angles cost about as much as a round.
  // Where warps take whole tokens, as many warps as leave each the same number.
  constexpr int64_t kMost = 152 * kResident;
  static_assert(!BACKWARD || kMost <= kQkMaxBlocks, "the workspace has a row for each block");
  int64_t rounds[2], blocks[2];
  for (int t = 0; t < 2; ++t) rounds[t] = (a.heads[t] + kGroups - 1) / kGroups;
  const int64_t cost[2] = {rounds[0] + 1, rounds[1] ? rounds[1] + 1 : 0};
  for (int t = 0; t < 2; ++t) {
    const int64_t share =
        std::max<int64_t>(1, t ? kMost - blocks[0] : kMost * cost[0] / (cost[0] + cost[1]) - (cost[1] > 0));
    blocks[t] = std::min(rounds[t] ? share : 0, (a.tokens * rounds[t] + kWarps - 1) / kWarps);
    if (a.tokens < kMany * share * kWarps || !rounds[t]) continue;
    // (up to 2% more than the queries' share is the keys' to lack)
    const int64_t room = t ? share : std::min<int64_t>(share + share / 50, kMost - (rounds[1] > 0));
    const int64_t each = (a.tokens + room * kWarps - 1) / (room * kWarps);
    blocks[t] = (a.tokens + each * kWarps - 1) / (each * kWarps);
  }
  const int all = (int)(blocks[0] + blocks[1]);
  auto* kernel = qk_kernel<T, W, VEC, LANES, CHUNKS, INTERLEAVED, BACKWARD>;
  constexpr int smem = Head<T, VEC, LANES, CHUNKS, INTERLEAVED>::kCopied ? kWarps * (int)Ring<T, VEC, BACKWARD>::kWarpBytes : 0;
  static std::atomic<unsigned long long> opened[256];
  cudaError_t e = open_kernel((const void*)kernel, smem, false, opened);
  if (e != cudaSuccess) return e;
  Turns<VEC * LANES * CHUNKS> turn = {};
  std::copy_n(a.turn, a.rotary / 2, turn.of);
  kernel<<<all, kThreads, smem, s>>>(a, turn, (int)blocks[0]);
  note_launch();
  e = cudaGetLastError();
  return e != cudaSuccess || !BACKWARD || !a.partial ? e : sum_weights<W>(a, (int)blocks[0], all, s);
}

// Lanes to a head: as few powers of two as hold its pairs.
template <class T, class W, int VEC, bool INTERLEAVED, bool BACKWARD>
cudaError_t by_lanes(const QkArgs& a, cudaStream_t s) {
  const int lanes = (a.dim / 2 + VEC - 1) / VEC;
  if constexpr (VEC == 1) {
    return run<T, W, 1, 32, kQkMaxDim / 64, INTERLEAVED, BACKWARD>(a, s);
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

template <bool BACKWARD>
cudaError_t launch_qk(int dtype, int wdtype, bool interleaved, const QkArgs& a, cudaStream_t s) {
  auto kind = [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    return interleaved ? by_vector<T, W, true, BACKWARD>(a, s) : by_vector<T, W, false, BACKWARD>(a, s);
  };
  return with_type(dtype, [&](auto t) { return wdtype == F32 ? kind(t, float()) : kind(t, t); });
}

}  // namespace
}  // namespace ar
