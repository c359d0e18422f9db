// Causal attention over packed sequences, backward.
//
//   p_ij = exp(a_ij - lse_i), delta_i = dout_i . out_i,
//   ds_ij = p_ij (dout_i . v_j - delta_i),
//   dv_j = sum_i p_ij dout_i, dk_j = scale sum_i ds_ij q_i, dq_i = scale sum_j ds_ij k_j.
//
// Bound by the tensor cores.  Two kernels, so that every sum is made by one
// block in a fixed order and no atomics are needed: one block for each 128
// keys of a K/V head walks over the queries of all heads of its group and
// sums dk and dv in tensor memory (four products a pair of tiles); one for
// each 128 queries walks over the keys and sums dq (three).  That is seven
// products where five are the least; a single kernel would have to add dq from
// many blocks to memory, in an order that changes.
//
// In both, a thread takes the exponentials of 32 columns of a row.  p and ds
// take the places of the scores and of dout v^T in tensor memory, as 16-bit
// pairs, and are the left operands of the sums' products there (rounded to the
// operands' type, as the tensor cores need: half a unit in the last place of
// each term).  The next tiles' products are issued between the current one's
// sums, so the tensor cores work while exponentials are taken.
//
// Measured (device time, bf16): 8192 tokens, 32 heads of 128 over 8 K/V heads,
// 1.07 ms as one sequence (1.28 PFLOP/s counting five products, 1.80 with the two
// that are made twice: 94% of the rate of a plain matrix product on the same
// device), 489 us as three of equal length, 611 as three of 1215, 1830 and 5147;
// 12 heads of 64, 65 us as 13 sequences of equal length, 77 as 13 of up to 1757
// tokens.  The blocks of dq spend 93% of a step in products, those of dk and dv
// 77%: there a step's exponentials come between two products that need them.
#include "ar_tcgen05.cuh"

#include <algorithm>

namespace ar {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Probabilities are at most one.  f16, whose smallest number is 2^-24 and
// largest 2^16, holds them times 2^15 in the product for dv, so that one of
// 2^-40 is not lost yet (thousands of them may add up to a normal number); the
// power is part of the exponential's argument and is taken out of the sums.
// bf16 has the range of binary32.
template <class T>
constexpr float kShift = __is_same(T, __half) ? 15.f : 0.f;
template <class T>
constexpr float kUnshift = __is_same(T, __half) ? 1.f / 32768.f : 1.f;

// Score gradients are as large as dout, whose size is the user's (a loss may be
// scaled by any power of two), times a probability.  f16 holds them as they are
// where the block's largest lies in [2^-12, 65504], so that what is too small
// to count is below 2^-13 of it.  Otherwise the block walks again, with them
// times another power of two:
//   - One past 65504 is an infinity in f16 and leaves none of its row's sums
//     finite, which is seen when they are written: 2^-13 and, if need be, 2^-26,
//     which no product of f16 operands outgrows.  What is lost is below 2^-28
//     of the largest.
//   - A thread looks at one of its 32 in each step.  If none of the block's is
//     2^-12, 2^26; should larger ones overflow then, 2^13 and 1.
// Device time of 8191 tokens in 13 sequences, 12 heads of 64: 79.1 us, and 76.8
// without any of this; 82.2 with a look at all 32 for the exact power, 81.3 with
// all walks in one loop (the first is compiled apart, its power a constant).
// Walks that follow cost as much each: 3000 tokens, 12 heads of 64, 67 us with
// one walk, 124 with two.  (A power that is known beforehand would have to bound
// v and dout over a whole sequence, a pass of its own over both; a fixed one
// loses either kind.)
template <class T>
constexpr bool kScaled = __is_same(T, __half);
constexpr float kTooSmall = 0x1p-12f, kUnknown = 0x1p-100f;
constexpr float kRaised = 0x1p26f, kLowered = 0x1p-13f, kLeast = 0x1p-26f;

constexpr int kKStages = 3, kVStages = 2;  // tiles of k and v in flight, for dq

// A block keeps 128 keys (or queries) and walks over tiles of kWalk queries
// (keys).  Heads of up to 64 elements (one panel) need half of tensor memory
// with 64 of them, so that two blocks share a multiprocessor and one's
// exponentials, or its start and end, overlap the other's products
// (8192 tokens in 13 sequences, 12 heads of 64: 95.7 us with one block and
// tiles of 128, 71.7 us so, with nothing else changed; 8192 tokens of one, 32
// heads of 64: 967 and 879).
// Four threads, or two, have a row's columns.
template <int PANELS>
struct Form {
  static constexpr int kWalk = PANELS == 1 ? 64 : 128;
  static constexpr int kQuarters = kWalk / 32;
  static constexpr int kWorkers = kTile * kQuarters;                          // threads
  static constexpr int kIssuer = kWorkers / 32, kLoader = kWorkers / 32 + 1;  // warps
  static constexpr int kThreads = kWorkers + 64;
  static constexpr int kBlocks = PANELS == 1 ? 2 : 1;  // on a multiprocessor
  static constexpr int kColumns = PANELS == 1 ? 256 : 512;
  static constexpr uint32_t kKeptBytes = PANELS * kPanelBytes, kWalkBytes = PANELS * kWalk * 128;
  static constexpr int kStages = PANELS == 1 ? 4 : 2;  // tiles of q and dout in flight
  // shared memory of the two kinds of block; the first has 128 floats for each worker warp after its tiles
  static constexpr uint32_t kTilesKV = 2 * kKeptBytes + 2 * kStages * kWalkBytes;
  static constexpr uint32_t kTilesQ = 2 * kKeptBytes + (kKStages + kVStages) * kWalkBytes;
};

// delta[head][token] = dout . out: LANES threads to a row, 16 bytes each.
template <class T, int LANES>
__global__ void __launch_bounds__(256) attention_delta_kernel(const AttnArgs a) {
  // the gradients' kernel may be set up meanwhile; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t row = blockIdx.x * (256 / LANES) + threadIdx.x / LANES, token = row / a.heads, head = row % a.heads;
  const int c = threadIdx.x % LANES * 8;
  float s = 0.f;
  if (token < a.tokens && c < a.dim) {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.out.ptr) + token * a.out.token_stride +
                                                    head * a.out.head_stride + c);
    const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.dout.ptr) + token * a.dout.token_stride +
                                                    head * a.dout.head_stride + c);
    Two acc = two(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = fma2(Pairs<T>::get(x, i), Pairs<T>::get(y, i), acc);
    float lo, hi;
    split(acc, lo, hi);
    s = lo + hi;
  }
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
  if (token < a.tokens && c == 0) a.delta[(int64_t)head * a.tokens + token] = s;
}

// The end of the kernel that makes delta.  What else a block reads was there
// before that kernel began, so its loads and first products need not wait; but
// every block waits before it ends, so that whatever comes next in the stream
// finds both kernels done.
__device__ __forceinline__ void wait_for_delta() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The kept tile, in boxes of kWalk rows.
template <int PANELS>
__device__ __forceinline__ void load_kept(const CUtensorMap* map, uint32_t dst, int head, int token, uint32_t bar) {
  constexpr int kWalk = Form<PANELS>::kWalk;
  for (int p = 0; p < PANELS; ++p)
    for (int r = 0; r < kTile; r += kWalk)
      tma_load(dst + p * kPanelBytes + r * 128, map, p * 64, head, token + r, bar);
}

// Where a first walk has met nothing but zeros: whether a worker's part of its
// row of dout (64 of the tile's bytes) holds anything else.
__device__ __forceinline__ bool any_element(uint32_t at) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + i * 16) : "memory");
    any |= v.x | v.y | v.z | v.w;
  }
  return (any & 0x7FFF7FFFu) != 0;
}

// What a worker has seen, for leave(): infinity where sums are not finite, zero
// if there is nothing but zeros.
template <class T>
__device__ __forceinline__ void put_most(float most, bool finite, float* each) {
  if constexpr (!kScaled<T>) return;
  __syncwarp();
  most = warp_max(finite ? most : INFINITY);
  if ((threadIdx.x & 31) == 0) each[threadIdx.x >> 5] = most;
}

// What a block keeps from one walk to the next.
struct State {
  float by = 1.f;           // what the score gradients are held times
  int walks = 0;            // made
  uint32_t own_parity = 0;  // the loader's
};

// The end of a walk: true, with another power, if the block has to walk again.
template <class T, int PANELS>
__device__ __forceinline__ bool leave(int* gave_up, int warp, uint32_t tmem, const float* each, State& state) {
  using F = Form<PANELS>;
  tc_fence_before();
  __syncthreads();
  if (*(volatile int*)gave_up) {
    // copies and products in flight end by themselves: give them time
    for (int i = 0; i < 100; ++i) __nanosleep(100000);
    if (threadIdx.x == 0) g_status = AR_ERR_TIMEOUT;
    __syncthreads();
  } else if (kScaled<T>) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < F::kWorkers / 32; ++i) most = fmaxf(most, each[i]);
    const bool lower = most == INFINITY && state.by > kLeast;
    const bool raise = state.walks == 0 && most > 0.f && most < kTooSmall;
    if (lower || raise) {
      state.by = lower ? state.by * kLowered : kRaised;
      ++state.walks;
      fence_async_shared();  // tiles are copied to where results have been
      __syncthreads();
      tc_fence_after();
      return true;
    }
  }
  if (warp == F::kIssuer) tmem_free(tmem, F::kColumns);
  return false;
}

// 32 scores of a thread become probabilities 2^(c s - lse) in place, and pairs
// of them in `packed`; `seen` is asked where the tile is `masked` alone.
template <class T, class L, class S>
__device__ __forceinline__ void probabilities(float (&p)[32], uint32_t (&packed)[16], float c, L lse, bool masked,
                                              S seen) {
  const Two c2 = two(c, c);
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    split(fma2(two(p[x], p[x + 1]), c2, lse(x)), p[x], p[x + 1]);
    p[x] = exp2_approx(p[x]);
    p[x + 1] = exp2_approx(p[x + 1]);
  }
  if (masked) {
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (!seen(x)) p[x] = 0.f;
  }
#pragma unroll
  for (int x = 0; x < 32; x += 2) packed[x / 2] = pack2<T>(p[x], p[x + 1]);
}

// Pairs of ds = p (by d - by delta).  What is not seen has p = 0 and no ds,
// whatever d holds there (tokens of another sequence, zeros times an infinity).
// The first of them is left in d, where f16 looks at it.
template <class T, class L>
__device__ __forceinline__ void score_gradients(float (&p)[32], float (&d)[32], uint32_t (&packed)[16], float by,
                                                L minus_delta, bool masked) {
  const Two by2 = two(by, by);
  if (masked) {
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (p[x] == 0.f) d[x] = 0.f;
  }
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    split(mul2(two(p[x], p[x + 1]), fma2(two(d[x], d[x + 1]), by2, minus_delta(x))), d[x], d[x + 1]);
    packed[x / 2] = pack2<T>(d[x], d[x + 1]);
  }
}

// Elements x and x + 1 of a vector in shared memory, x even, read four at a time.
__device__ __forceinline__ Two two_of(const float* v, int x) {
  const ulonglong2 four = *reinterpret_cast<const ulonglong2*>(v + (x & ~3));
  return Two{x & 2 ? four.y : four.x};
}

struct Maps {
  CUtensorMap q, k, v, dout;
};

// ---- dk and dv ---------------------------------------------------------------------

constexpr int kMostStages = 4;

struct SharedKV {
  alignas(8) uint64_t kv_full, q_full[kMostStages], do_full[kMostStages], empty[kMostStages], s_full, dp_full, p_ready,
      ds_ready, done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
  float most[16];  // what each worker warp has seen of the score gradients
};

template <int PANELS>
__device__ __forceinline__ void init_barriers(SharedKV& sh) {
  using F = Form<PANELS>;
  uint64_t* const one[] = {&sh.kv_full, &sh.s_full, &sh.dp_full, &sh.done, &sh.own};
  for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
  for (int i = 0; i < F::kStages; ++i) {
    mbar_init(smem_addr(&sh.q_full[i]), 1);
    mbar_init(smem_addr(&sh.do_full[i]), 1);
    mbar_init(smem_addr(&sh.empty[i]), 1);
  }
  mbar_init(smem_addr(&sh.p_ready), F::kWorkers / 32);
  mbar_init(smem_addr(&sh.ds_ready), F::kWorkers / 32);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// A walk over the queries.  True if the block has to make another one; the
// barriers' phases go on counting.
template <class T, int PANELS, bool FIRST>
__device__ __forceinline__ bool dkv_walk(const Maps& maps, const AttnArgs& a, int kv_head, uint8_t* tiles, SharedKV& sh,
                                         State& state) {
  using F = Form<PANELS>;
  constexpr int kStages = F::kStages, kWalk = F::kWalk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SeqUnit unit = sh.unit;
  unit.index = unit.count - 1 - unit.index;  // the first keys are seen by the most queries

  const uint32_t k_tile = smem_addr(tiles), v_tile = k_tile + F::kKeptBytes, q_tile = v_tile + F::kKeptBytes,
                 do_tile = q_tile + kStages * F::kWalkBytes;
  volatile int* gave_up = &sh.gave_up;
  // each step takes a tile of the sequence's queries from the first that sees
  // the keys, head after head of the group
  const int group = a.heads / a.kv_heads, first = unit.index * (kTile / kWalk);
  const int per = (unit.length + kWalk - 1) / kWalk - first, steps = group * per;
  const int dim16 = (a.dim + 15) / 16;
  const int base = FIRST ? 0 : state.walks * steps, end = base + steps;  // steps made before, and after
  const float by = FIRST ? 1.f : state.by;
  if (FIRST && warp == F::kLoader && lane == 0) {
    const uint32_t bar = smem_addr(&sh.kv_full);
    mbar_expect(bar, 2 * F::kKeptBytes);
    load_kept<PANELS>(&maps.k, k_tile, kv_head, unit.begin + unit.index * kTile, bar);
    load_kept<PANELS>(&maps.v, v_tile, kv_head, unit.begin + unit.index * kTile, bar);
  }
  // Tensor memory: scores, dout v^T, dv, dk.  p and ds take the places of the
  // first two, each quarter's 16 columns of pairs at the front of the 32 that
  // it read.
  const uint32_t tmem = sh.tmem, dp_at = tmem + kWalk, dv_at = tmem + 2 * kWalk, dk_at = dv_at + 64 * PANELS;

  if (warp == F::kLoader) {
    int head = kv_head * group, tile = 0;
    for (int n = base; n < end; ++n) {
      const int stage = n % kStages;
      if (n >= kStages && !mbar_wait(smem_addr(&sh.empty[stage]), (n / kStages - 1) & 1, gave_up)) break;
      const int query = (first + tile) * kWalk;
      if (!load_tile<PANELS, kWalk>(&maps.q, q_tile + stage * F::kWalkBytes, head, unit.begin + query,
                                    unit.length - query, smem_addr(&sh.q_full[stage]), smem_addr(&sh.own),
                                    &state.own_parity, gave_up) ||
          !load_tile<PANELS, kWalk>(&maps.dout, do_tile + stage * F::kWalkBytes, head, unit.begin + query,
                                    unit.length - query, smem_addr(&sh.do_full[stage]), smem_addr(&sh.own),
                                    &state.own_parity, gave_up))
        break;
      if (++tile == per) tile = 0, ++head;
    }
  } else if (warp == F::kIssuer) {
    if (elect_one()) {
      const uint32_t wide = mma_shape<T>(kWalk, false), sums = mma_shape<T>(dim16 * 16, true);
      auto at = [&](uint32_t tile, int n) { return tile + (n % kStages) * F::kWalkBytes; };
      auto scores = [&](int n) {  // K Q^T
        if (!mbar_wait(smem_addr(&sh.q_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(tmem, k_tile, at(q_tile, n), wide, dim16);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // V dout^T
        if (!mbar_wait(smem_addr(&sh.do_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(dp_at, v_tile, at(do_tile, n), wide, dim16);
        mma_commit(smem_addr(&sh.dp_full));
        return true;
      };
      auto sum = [&](uint64_t& ready, uint32_t to, uint32_t left, uint32_t right, int n) {
        if (!mbar_wait(smem_addr(&ready), n & 1, gave_up)) return false;
        tc_fence_after();
        for (int h = 0; h < F::kQuarters; ++h) product_ts<2>(to, left + h * 32, right, h, sums, n > base || h > 0);
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.kv_full), 0, gave_up) && scores(base) && dprob(base);
      for (int n = base; n < end && ok; ++n) {
        const bool more = n + 1 < end;
        ok = sum(sh.p_ready, dv_at, tmem, at(do_tile, n), n) && (!more || scores(n + 1)) &&
             sum(sh.ds_ready, dk_at, dp_at, at(q_tile, n), n);
        if (ok) mma_commit(smem_addr(&sh.empty[n % kStages]));
        if (ok && more) ok = dprob(n + 1);
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: key row, queries [32 quarter, 32 quarter + 32) of each tile
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane;
    const int left = unit.length - unit.index * kTile;  // queries from the first key to the sequence's end
    const uint32_t lane0 = (uint32_t)(warp & 3) << 21, s_at = tmem + lane0 + quarter * 32;
    const float c = a.scale * kLog2e;
    float* stats = reinterpret_cast<float*>(tiles + F::kTilesKV) + warp * 128;  // [turn][lse, delta][32]
    // Each warp fetches its 32 queries' -lse in powers of two and -delta for
    // itself: four warps that shared them would meet at every step.  What the
    // probabilities are held times is in the first and out of the second.
    int next_tile = 0;
    int64_t next_head = (int64_t)kv_head * group * a.tokens + unit.begin;
    const float by_unshift = by * kUnshift<T>, unscale = 1.f / by;
    auto fetch = [&]() {  // of the next step, and on
      const int query = (first + next_tile) * kWalk + quarter * 32 + lane;
      const int64_t at = next_head + query;
      if (++next_tile == per) next_tile = 0, next_head += a.tokens;
      if (query >= unit.length) return make_float2(0.f, 0.f);  // masked
      return make_float2(fmaf(-a.lse[at], kLog2e, kShift<T>), -a.delta[at] * by_unshift);
    };
    auto put = [&](int n, float2 v) {
      stats[(n & 1) * 64 + lane] = v.x;
      stats[(n & 1) * 64 + 32 + lane] = v.y;
      __syncwarp();
    };
    wait_for_delta();
    put(base, fetch());
    int tile = 0;
    bool ok = true, finite = true;
    float most = kUnknown;
    for (int n = base; n < end; ++n) {
      const float2 next = n + 1 < end ? fetch() : make_float2(0.f, 0.f);
      const int from = tile * kWalk;  // the tile's first query, counted from the first key
      const bool masked = from < kTile || from + kWalk > left;
      if (!(ok = mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up))) break;
      tc_fence_after();
      float p[32], d[32];
      uint32_t packed[16];
      tmem_load32(s_at, p);
      tmem_wait_load();
      tmem_loaded(p);
      const float* lse = stats + (n & 1) * 64;
      probabilities<T>(p, packed, c, [&](int x) { return two_of(lse, x); }, masked,
                       [&](int x) { return from + quarter * 32 + x >= row && from + quarter * 32 + x < left; });
      tmem_store16(s_at, packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.p_ready));
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full), n & 1, gave_up))) break;
      tc_fence_after();
      tmem_load32(s_at + kWalk, d);
      tmem_wait_load();
      tmem_loaded(d);
      const float* delta = stats + (n & 1) * 64 + 32;
      score_gradients<T>(p, d, packed, by_unshift, [&](int x) { return two_of(delta, x); }, masked);
      tmem_store16(s_at + kWalk, packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.ds_ready));
      if (kScaled<T>) most = fmaxf(most, fabsf(d[0]));
      put(n + 1, next);
      if (++tile == per) tile = 0;
    }
    if (ok && mbar_wait(smem_addr(&sh.done), FIRST ? 0 : state.walks & 1, gave_up)) {
      tc_fence_after();
      // quarter: dv or dk, and which 64 of its columns
      const bool is_dk = quarter & 1;
      const AttnTensor& to = is_dk ? a.dk : a.dv;
      const int key = unit.index * kTile + (warp & 3) * 32;
      T* out = static_cast<T*>(const_cast<void*>(to.ptr)) + (int64_t)(unit.begin + key) * to.token_stride +
               kv_head * to.head_stride;
      finite = write_rows<T, 64>(lane0 + (is_dk ? dk_at : dv_at), q_tile + warp * 4096, out, to.token_stride,
                                 unit.length - key, (quarter >> 1) * 64, a.dim, is_dk ? a.scale * unscale : kUnshift<T>) ||
               !is_dk;
    }
    put_most<T>(most, finite, sh.most);
  }
  return leave<T, PANELS>(&sh.gave_up, warp, tmem, sh.most, state);
}

template <class T, int PANELS>
__device__ __forceinline__ void dkv_block(const Maps& maps, const AttnArgs& a, int block, uint8_t* tiles, SharedKV& sh) {
  using F = Form<PANELS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv_head = block % a.kv_heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, block / a.kv_heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == F::kIssuer) {
    tmem_alloc(smem_addr(&sh.tmem), F::kColumns);
  } else if (warp == F::kLoader && lane == 0) {
    init_barriers<PANELS>(sh);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.unit.count == 0) {
    if (warp == F::kIssuer) tmem_free(sh.tmem, F::kColumns);
    wait_for_delta();
    return;
  }
  State state;
  if (dkv_walk<T, PANELS, true>(maps, a, kv_head, tiles, sh, state)) {
    if constexpr (kScaled<T>)
      while (dkv_walk<T, PANELS, false>(maps, a, kv_head, tiles, sh, state)) {}
  }
}

// ---- dq ---------------------------------------------------------------------------

struct SharedQ {
  alignas(8) uint64_t q_full, k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], s_full, s_read,
      dp_full[2], ds_ready[2], done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
  float most[16];
};

template <int PANELS>
__device__ __forceinline__ void init_barriers(SharedQ& sh) {
  using F = Form<PANELS>;
  uint64_t* const one[] = {&sh.q_full, &sh.s_full, &sh.dp_full[0], &sh.dp_full[1], &sh.done, &sh.own};
  for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
  for (int i = 0; i < kKStages; ++i) {
    mbar_init(smem_addr(&sh.k_full[i]), 1);
    mbar_init(smem_addr(&sh.k_empty[i]), 1);
  }
  for (int i = 0; i < kVStages; ++i) {
    mbar_init(smem_addr(&sh.v_full[i]), 1);
    mbar_init(smem_addr(&sh.v_empty[i]), 1);
  }
  mbar_init(smem_addr(&sh.s_read), F::kWorkers / 32);
  for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&sh.ds_ready[i]), F::kWorkers / 32);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// A walk over the keys, as dkv_walk.
template <class T, int PANELS, bool FIRST>
__device__ __forceinline__ bool dq_walk(const Maps& maps, const AttnArgs& a, int head, uint8_t* tiles, SharedQ& sh,
                                        State& state) {
  using F = Form<PANELS>;
  constexpr int kWalk = F::kWalk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqUnit unit = sh.unit;

  const uint32_t q_tile = smem_addr(tiles), do_tile = q_tile + F::kKeptBytes, k_tile = do_tile + F::kKeptBytes,
                 v_tile = k_tile + kKStages * F::kWalkBytes;
  volatile int* gave_up = &sh.gave_up;
  const int query = unit.index * kTile;
  const int steps = min(query + kTile, unit.length + kWalk - 1) / kWalk;  // tiles of keys that the queries see
  const int dim16 = (a.dim + 15) / 16;
  const int base = FIRST ? 0 : state.walks * steps, end = base + steps;  // steps made before, and after
  const float by = FIRST ? 1.f : state.by;
  if (FIRST && warp == F::kLoader && lane == 0) {
    const uint32_t bar = smem_addr(&sh.q_full);
    mbar_expect(bar, 2 * F::kKeptBytes);
    load_kept<PANELS>(&maps.q, q_tile, head, unit.begin + query, bar);
    load_kept<PANELS>(&maps.dout, do_tile, head, unit.begin + query, bar);
  }
  // Tensor memory: scores, dout v^T (in two places by turns), dq.  The next
  // tile's scores and dout v^T are under way while this one's ds is made.  So a
  // warp may have finished the next step before another has this one, though
  // not one more (the scores after it wait for every warp's s_read): ds_ready is
  // two barriers by turns, as one would count the first warp in both places.
  const uint32_t tmem = sh.tmem, dq_at = tmem + 3 * kWalk;
  auto dp_at = [&](int n) { return tmem + kWalk * (1 + (n & 1)); };

  if (warp == F::kLoader) {
    const int kv_head = head / (a.heads / a.kv_heads);
    for (int n = base; n < end; ++n) {
      const int ks = n % kKStages, vs = n % kVStages, key = (n - base) * kWalk;
      if (n >= kKStages && !mbar_wait(smem_addr(&sh.k_empty[ks]), (n / kKStages - 1) & 1, gave_up)) break;
      // dq sums over the rows of K: those of another sequence are cleared
      if (!load_tile<PANELS, kWalk>(&maps.k, k_tile + ks * F::kWalkBytes, kv_head, unit.begin + key, unit.length - key,
                                    smem_addr(&sh.k_full[ks]), smem_addr(&sh.own), &state.own_parity, gave_up))
        break;
      if (n >= kVStages && !mbar_wait(smem_addr(&sh.v_empty[vs]), (n / kVStages - 1) & 1, gave_up)) break;
      if (!load_tile<PANELS, kWalk>(&maps.v, v_tile + vs * F::kWalkBytes, kv_head, unit.begin + key, kWalk,
                                    smem_addr(&sh.v_full[vs]), smem_addr(&sh.own), &state.own_parity, gave_up))
        break;
    }
  } else if (warp == F::kIssuer) {
    if (elect_one()) {
      const uint32_t wide = mma_shape<T>(kWalk, false), sums = mma_shape<T>(dim16 * 16, true);
      auto scores = [&](int n) {  // Q K^T
        if (!mbar_wait(smem_addr(&sh.k_full[n % kKStages]), (n / kKStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(tmem, q_tile, k_tile + (n % kKStages) * F::kWalkBytes, wide, dim16);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // dout V^T
        if (!mbar_wait(smem_addr(&sh.v_full[n % kVStages]), (n / kVStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(dp_at(n), do_tile, v_tile + (n % kVStages) * F::kWalkBytes, wide, dim16);
        mma_commit(smem_addr(&sh.dp_full[n & 1]));
        mma_commit(smem_addr(&sh.v_empty[n % kVStages]));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.q_full), 0, gave_up) && scores(base) && dprob(base);
      for (int n = base; n < end && ok; ++n) {
        if (n + 1 < end) {
          if (!(ok = mbar_wait(smem_addr(&sh.s_read), n & 1, gave_up))) break;
          tc_fence_after();
          if (!(ok = scores(n + 1) && dprob(n + 1))) break;
        }
        if (!(ok = mbar_wait(smem_addr(&sh.ds_ready[n & 1]), (n >> 1) & 1, gave_up))) break;
        tc_fence_after();
        for (int h = 0; h < F::kQuarters; ++h)
          product_ts<2>(dq_at, dp_at(n) + h * 32, k_tile + (n % kKStages) * F::kWalkBytes, h, sums, n > base || h > 0);
        mma_commit(smem_addr(&sh.k_empty[n % kKStages]));
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: query row, keys [32 quarter, 32 quarter + 32) of each tile
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane0 = (uint32_t)(warp & 3) << 21;
    const float c = a.scale * kLog2e;
    const bool valid = query + row < unit.length;
    wait_for_delta();
    const int64_t at = (int64_t)head * a.tokens + unit.begin + query + row;
    const float l = valid ? -a.lse[at] * kLog2e : -INFINITY, dl = valid ? -a.delta[at] : 0.f;
    const Two lse = two(l, l), delta = two(dl * by, dl * by);
    bool ok = true, finite = true;
    float most = 0.f;
    for (int n = base; n < end; ++n) {
      const int key = (n - base) * kWalk;  // the tile's first
      const bool masked = key + kWalk > query;
      if (!(ok = mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up))) break;
      tc_fence_after();
      float p[32], d[32];
      uint32_t packed[16];
      tmem_load32(lane0 + tmem + quarter * 32, p);
      tmem_wait_load();
      tmem_loaded(p);
      warp_arrive(smem_addr(&sh.s_read));
      probabilities<T>(p, packed, c, [&](int) { return lse; }, masked,
                       [&](int x) { return key + quarter * 32 + x <= query + row; });
      const uint32_t dp = lane0 + dp_at(n) + quarter * 32;
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full[n & 1]), (n >> 1) & 1, gave_up))) break;
      tc_fence_after();
      tmem_load32(dp, d);
      tmem_wait_load();
      tmem_loaded(d);
      score_gradients<T>(p, d, packed, by, [&](int) { return delta; }, masked);
      tmem_store16(dp, packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.ds_ready[n & 1]));
      if (kScaled<T>) most = fmaxf(most, fabsf(d[0]));
    }
    if (ok && mbar_wait(smem_addr(&sh.done), FIRST ? 0 : state.walks & 1, gave_up)) {
      tc_fence_after();
      const int from = query + (warp & 3) * 32;
      T* out = static_cast<T*>(const_cast<void*>(a.dq.ptr)) + (int64_t)(unit.begin + from) * a.dq.token_stride +
               head * a.dq.head_stride;
      finite = write_rows<T, 32>(lane0 + dq_at, k_tile + warp * 2048, out, a.dq.token_stride, unit.length - from,
                                 quarter * 32, a.dim, a.scale * (1.f / by));
    }
    if (kScaled<T> && FIRST && ok && !__any_sync(0xFFFFFFFFu, most > 0.f)) {
      // a prompt's queries often have no gradient at all, and need no other power
      ok = mbar_wait(smem_addr(&sh.q_full), 0, gave_up);
      if (valid && any_element(do_tile + (quarter >> 1) * kPanelBytes + row * 128 + (quarter & 1) * 64)) most = kUnknown;
    }
    put_most<T>(most, finite, sh.most);
  }
  return leave<T, PANELS>(&sh.gave_up, warp, tmem, sh.most, state);
}

template <class T, int PANELS>
__device__ __forceinline__ void dq_block(const Maps& maps, const AttnArgs& a, int block, uint8_t* tiles, SharedQ& sh) {
  using F = Form<PANELS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = block % a.heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, block / a.heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == F::kIssuer) {
    tmem_alloc(smem_addr(&sh.tmem), F::kColumns);
  } else if (warp == F::kLoader && lane == 0) {
    init_barriers<PANELS>(sh);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.unit.count == 0) {
    if (warp == F::kIssuer) tmem_free(sh.tmem, F::kColumns);
    wait_for_delta();
    return;
  }
  State state;
  if (dq_walk<T, PANELS, true>(maps, a, head, tiles, sh, state)) {
    if constexpr (kScaled<T>)
      while (dq_walk<T, PANELS, false>(maps, a, head, tiles, sh, state)) {}
  }
}

// ---- both ---------------------------------------------------------------------------

union Shared {
  SharedKV kv;
  SharedQ q;
  __device__ Shared() {}
};

// One launch, so that the second kind's blocks fill the first's last wave; the
// first `kv_blocks` blocks make dk and dv.
template <class T, int PANELS>
__global__ void __launch_bounds__(Form<PANELS>::kThreads, Form<PANELS>::kBlocks)
    attention_backward_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, int kv_blocks) {
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ Shared sh;
  const int block = blockIdx.x;
  if (block < kv_blocks) dkv_block<T, PANELS>(maps, a, block, tiles, sh.kv);
  else dq_block<T, PANELS>(maps, a, block - kv_blocks, tiles, sh.q);
}

template <class T, int PANELS>
cudaError_t run(int dtype, const AttnArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  using F = Form<PANELS>;
  constexpr int smem = (int)std::max(F::kTilesKV + F::kWorkers / 32 * 512, F::kTilesQ);
  auto* kernel = attention_backward_kernel<T, PANELS>;
  cudaError_t e = open_kernel((const void*)kernel, smem, false, opened);
  if (e != cudaSuccess) return e;
  Maps maps;
  if (!make_tensor_map(&maps.q, dtype, a.q, a.tokens, a.heads, a.dim, F::kWalk) ||
      !make_tensor_map(&maps.k, dtype, a.k, a.tokens, a.kv_heads, a.dim, F::kWalk) ||
      !make_tensor_map(&maps.v, dtype, a.v, a.tokens, a.kv_heads, a.dim, F::kWalk) ||
      !make_tensor_map(&maps.dout, dtype, a.dout, a.tokens, a.heads, a.dim, F::kWalk))
    return cudaErrorInvalidValue;
  constexpr int kLanes = PANELS * 8, kRows = 256 / kLanes;
  attention_delta_kernel<T, kLanes><<<(unsigned)((a.tokens * a.heads + kRows - 1) / kRows), 256, 0, s>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t most = most_units(a.tokens, a.seqs, kTile);
  const int kv_blocks = (int)(most * a.kv_heads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kv_blocks + most * a.heads));
  cfg.blockDim = dim3(F::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, maps, a, kv_blocks);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_attention_backward(int dtype, const AttnArgs& a, cudaStream_t s) {
  if (dtype == BF16) return a.dim <= 64 ? run<__nv_bfloat16, 1>(dtype, a, s) : run<__nv_bfloat16, 2>(dtype, a, s);
  return a.dim <= 64 ? run<__half, 1>(dtype, a, s) : run<__half, 2>(dtype, a, s);
}

cudaError_t attention_backward_take_status(int* status, cudaStream_t s) { return take_status(status, s); }

}  // namespace ar
