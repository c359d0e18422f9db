// Differential attention over packed sequences, backward.
//
//   p_m = exp(a_m - lse_m), delta_1 = dout . second, delta_0 = dout . out + lambda delta_1,
//   dp = dout v^T, ds_0 = p_0 (dp - delta_0), ds_1 = -lambda p_1 (dp - delta_1),
//   dv = (p_0 - lambda p_1)^T dout, dk_m = scale ds_m^T q_m, dq_m = scale ds_m k_m,
//   dlambda = -sum delta_1.
//
// Both maps share dp, and dv is one product of their difference, so a pair of
// tokens costs 12 dim + 4 value_dim operations.  As in the ordinary attention's
// gradient every sum is made by one block in a fixed order: a block for each
// 128 keys of a group walks over its heads' queries and sums dv and both dk in
// tensor memory, one for each 128 queries of a head walks over the keys and sums
// both dq (scores and dp are made by both kinds).  The last blocks of the launch
// sum lambda's gradients.
//
// Tiles of 64 are walked, so that both maps' scores, dp and all sums fit tensor
// memory.  Four threads have a row's 64 columns (424 us at the size below, two
// 434).  The difference of probabilities has a place of its own, two by turns, so
// the next scores are computed as soon as the current ones have been read; both ds
// take dp's place, as 16-bit pairs.  A warp fetches the queries' statistics for
// dk and dv's workers (who waited for them a third of a step before).
//
// What a product of 128 x 64 reads from shared memory takes half as long again as
// the product; dq's blocks have their kept tiles, the left operands of scores and
// dp, in tensor memory instead.
//
// Measured: 8192 tokens in 3 sequences, 16 heads of 2 x 64 over 4, bf16, 425 us a
// call.  A step of dk and dv takes 1940 cycles, of which the tensor cores are busy
// for 1500 (scores and dp wait for shared memory), one of dq 1290; starting and
// ending a block takes 9000, a third of the time where sequences are short.
//
// lambda may differ from one by any factor, and f16 would lose what it makes
// small: ds_1 is held without it in dq's blocks and relative to the group's
// largest in dk's, and the sums are multiplied by the rest.
#include "ar_attention_backward.cuh"

#include <algorithm>
#include <type_traits>

namespace ar {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

constexpr int kWalk = 64;
constexpr uint32_t kPart = kWalk * 128;       // bytes of a panel of a walked tile
constexpr uint32_t kStageBytes = 2 * kPart;   // of a walked tile
constexpr int kStages = 4;                    // tiles of q and of dout in flight, for dk and dv
constexpr int kKStages = 4, kVStages = 4;     // of k and v, for dq
constexpr int kCols = 16;                     // of a walked tile's columns that a worker has
constexpr int kParts = kWalk / kCols;         // workers to a row
constexpr int kStats = 4 * kWalk + 16;        // floats of a tile of queries: [lse 0, lse 1, delta 0, delta 1][query], lambda

struct Form {
  static constexpr int kWorkers = kTile * kParts;  // threads
  static constexpr int kIssuer = kWorkers / 32, kLoader = kIssuer + 1, kFetcher = kIssuer + 2;  // warps
  static constexpr int kThreads = kWorkers + 96;
  static constexpr int kColumns = 512;
};
// shared memory of both kinds of block
constexpr uint32_t kTilesKV = 4 * kPanelBytes + 2 * kStages * kStageBytes;
constexpr uint32_t kTilesQ = 4 * kPanelBytes + (kKStages + kVStages) * kStageBytes;
constexpr uint32_t kSmem = kTilesKV + kStages * kStats * 4;
static_assert(kTilesQ <= kSmem, "both kinds of block share a launch");

struct Maps {
  CUtensorMap q, k, v, dout;
};

// delta[2 head + m][token]: LANES threads to a row, 16 bytes each.  Tokens
// outside all sequences have zeros, whatever they hold.
template <class T, int LANES>
__global__ void __launch_bounds__(256) diff_delta_kernel(const DiffArgs a) {
  // the gradients' kernel may be set up meanwhile; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t row = blockIdx.x * (256 / LANES) + threadIdx.x / LANES, token = row / a.heads, head = row % a.heads;
  const int c = threadIdx.x % LANES * 8;
  const bool there = token < a.tokens && (int)token >= a.cu_seqlens[0] && (int)token < a.cu_seqlens[a.seqs];
  float first = 0.f, second = 0.f;
  if (there && c < a.value_dim) {
    auto piece = [&](const AttnTensor& t) {
      return *reinterpret_cast<const uint4*>(static_cast<const T*>(t.ptr) + token * t.token_stride + head * t.head_stride + c);
    };
    const uint4 x = piece(a.out), y = piece(a.second), z = piece(a.dout);
    Two acc0 = two(0.f, 0.f), acc1 = acc0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc0 = fma2(Pairs<T>::get(x, i), Pairs<T>::get(z, i), acc0);
      acc1 = fma2(Pairs<T>::get(y, i), Pairs<T>::get(z, i), acc1);
    }
    float lo, hi;
    split(acc0, lo, hi);
    first = lo + hi;
    split(acc1, lo, hi);
    second = lo + hi;
  }
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) {
    first += __shfl_xor_sync(0xFFFFFFFFu, first, m);
    second += __shfl_xor_sync(0xFFFFFFFFu, second, m);
  }
  if (token < a.tokens && c == 0) {
    float* to = a.delta + (int64_t)2 * head * a.tokens + token;
    to[0] = there ? fmaf(a.lambda[head], second, first) : 0.f;
    to[a.tokens] = second;
  }
}

// ---- lambda ----------------------------------------------------------------------

// One block to a head, its threads' sums joined in a fixed order.
__device__ __forceinline__ void dlambda_block(const DiffArgs& a, int head, float* part) {
  wait_for_delta();
  const float* delta = a.delta + (int64_t)(2 * head + 1) * a.tokens;
  float sum = 0.f;
  for (int64_t t = threadIdx.x; t < a.tokens; t += Form::kThreads) sum += delta[t];
  sum = warp_sum(sum);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  sum = 0.f;
  for (int i = 0; i < Form::kThreads / 32; ++i) sum += part[i];
  a.dlambda[head] = -sum;
}

// ---- loads ------------------------------------------------------------------------

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// The kept tile of both maps (PANELS 2, a panel each), or of v or dout.
template <int PANELS, bool BOTH_MAPS>
__device__ __forceinline__ void load_kept(const CUtensorMap* map, uint32_t dst, int head, int token, uint32_t bar) {
  mbar_expect(bar, PANELS * kPanelBytes);
  for (int p = 0; p < PANELS; ++p)
    for (int r = 0; r < kTile; r += kWalk)
      tma_load(dst + p * kPanelBytes + r * 128, map, BOTH_MAPS ? 0 : p * 64, BOTH_MAPS ? 2 * head + p : head, token + r, bar);
}

// A walked tile, as load_tile; the panels of v and dout lie kPanelBytes apart, as
// the products over 128 columns expect them, two stages between each other.
template <int PANELS, bool BOTH_MAPS>
__device__ __forceinline__ bool load_walked(const CUtensorMap* map, uint32_t dst, int head, int token, int rows,
                                            uint32_t full, uint32_t own, uint32_t* own_parity, volatile int* gave_up) {
  constexpr uint32_t kApart = BOTH_MAPS ? kPart : kPanelBytes;
  const int lane = threadIdx.x & 31;
  const bool cut = rows < kWalk;
  if (lane == 0) {
    const uint32_t bar = cut ? own : full;
    mbar_expect(bar, PANELS * kPart);
    for (int p = 0; p < PANELS; ++p)
      tma_load(dst + p * kApart, map, BOTH_MAPS ? 0 : p * 64, BOTH_MAPS ? 2 * head + p : head, token, bar);
  }
  if (!cut) return true;
  if (!mbar_wait(own, *own_parity, gave_up)) return false;
  *own_parity ^= 1;
  for (int p = 0; p < PANELS; ++p)
    for (uint32_t b = rows * 128 + lane * 16; b < kPart; b += 512)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + p * kApart + b), "r"(0) : "memory");
  fence_async_shared();
  __syncwarp();
  if (lane == 0) mbar_arrive(full);
  return true;
}
// Where the n-th tile of both maps, and of v or dout, lies.
__device__ __forceinline__ uint32_t maps_at(uint32_t tiles, int stage) { return tiles + stage * kStageBytes; }
__device__ __forceinline__ uint32_t panels_at(uint32_t tiles, int stage) {
  return tiles + (stage >> 1) * 2 * kStageBytes + (stage & 1) * kPart;
}

// Half a row of a panel in shared memory becomes 16 columns of pairs in the
// thread's lane of tensor memory, the form of a left operand there.
__device__ __forceinline__ void keep_half(uint32_t panel, int row, int half, uint32_t to) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[4 * i]), "=r"(r[4 * i + 1]), "=r"(r[4 * i + 2]), "=r"(r[4 * i + 3])
                 : "r"(panel + row * 128 + (((4 * half + i) ^ (row & 7)) << 4))
                 : "memory");
  tmem_store16(to, r);
}
// D = A B^T over `steps` times 16 columns: A's pairs in tensor memory, B K-major.
template <int MAX>
__device__ __forceinline__ void product_tk(uint32_t d, uint32_t a, uint32_t b_tile, uint32_t shape, int steps) {
  const uint64_t b = panel_desc(b_tile, false);
#pragma unroll
  for (int k = 0; k < MAX; ++k)
    if (k < steps) mma_ts(d, a + k * 8, b + k_major_step(k), shape, k > 0);
}

// ---- a worker's arithmetic ----------------------------------------------------------

// A worker's scores become probabilities 2^(c s - lse) in place.  `seen` is asked in
// masked tiles alone, whose steps are compiled apart (as one, every step took the
// comparisons).
template <bool MASKED, class L, class S>
__device__ __forceinline__ void probabilities(float (&p)[kCols], float c, L lse, S seen) {
  const Two c2 = two(c, c);
#pragma unroll
  for (int x = 0; x < kCols; x += 2) {
    split(fma2(two(p[x], p[x + 1]), c2, lse(x)), p[x], p[x + 1]);
    p[x] = exp2_approx(p[x]);
    p[x + 1] = exp2_approx(p[x + 1]);
  }
  if constexpr (MASKED) {
#pragma unroll
    for (int x = 0; x < kCols; ++x)
      if (!seen(x)) p[x] = 0.f;
  }
}

static_assert(kCols == 16, "what a worker loads at a time, and stores as pairs");
__device__ __forceinline__ void store_pairs(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Pairs of ds = p (by d + minus_delta).  What is not seen has p = 0 and no ds,
// whatever d holds there.  The first is returned, where f16 looks at it.
template <class T, bool MASKED, class L>
__device__ __forceinline__ float score_gradients(const float (&p)[kCols], const float (&d)[kCols], uint32_t (&packed)[kCols / 2],
                                                 float by, L minus_delta) {
  const Two by2 = two(by, by);
  float first = 0.f;
#pragma unroll
  for (int x = 0; x < kCols; x += 2) {
    float lo, hi;
    split(mul2(two(p[x], p[x + 1]), fma2(two(d[x], d[x + 1]), by2, minus_delta(x))), lo, hi);
    if constexpr (MASKED) {
      if (p[x] == 0.f) lo = 0.f;
      if (p[x + 1] == 0.f) hi = 0.f;
    }
    if (x == 0) first = lo;
    packed[x / 2] = pack2<T>(lo, hi);
  }
  return first;
}

// ---- dk and dv ---------------------------------------------------------------------

struct SharedKV {
  alignas(8) uint64_t k_full, v_full, q_full[kStages], do_full[kStages], stats_full[kStages], empty[kStages], s_full, s_read,
      dp_full, p_ready[2], ds_ready[2], done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
  float most[Form::kWorkers / 32];  // what each worker warp has seen of the score gradients
  float largest;                    // lambda of the group in size, or 2^-100, whose reciprocal is a number
};

__device__ __forceinline__ void init_barriers(SharedKV& sh) {
  uint64_t* const one[] = {&sh.k_full, &sh.v_full, &sh.s_full, &sh.dp_full, &sh.done, &sh.own};
  for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
  for (int i = 0; i < kStages; ++i) {
    mbar_init(smem_addr(&sh.q_full[i]), 1);
    mbar_init(smem_addr(&sh.do_full[i]), 1);
    mbar_init(smem_addr(&sh.stats_full[i]), 1);
    mbar_init(smem_addr(&sh.empty[i]), 1);
  }
  uint64_t* const warps[] = {&sh.s_read, &sh.p_ready[0], &sh.p_ready[1], &sh.ds_ready[0], &sh.ds_ready[1]};
  for (uint64_t* b : warps) mbar_init(smem_addr(b), Form::kWorkers / 32);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// A walk over the queries.  True if the block has to make another one; the
// barriers' phases go on counting.
template <class T, int VPANELS, bool FIRST>
__device__ __forceinline__ bool dkv_walk(const Maps& maps, const DiffArgs& a, int kv_head, uint8_t* tiles, SharedKV& sh,
                                         State& state) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SeqUnit unit = sh.unit;
  unit.index = unit.count - 1 - unit.index;  // the first keys are seen by the most queries

  const uint32_t k_tile = smem_addr(tiles), v_tile = k_tile + 2 * kPanelBytes, q_tile = v_tile + 2 * kPanelBytes,
                 do_tile = q_tile + kStages * kStageBytes;
  volatile int* gave_up = &sh.gave_up;
  // each step takes a tile of the sequence's queries from the first that sees
  // the keys, head after head of the group
  const int group = a.heads / a.kv_heads, first = unit.index * (kTile / kWalk);
  const int per = (unit.length + kWalk - 1) / kWalk - first, steps = group * per;
  const int dim16 = (a.dim + 15) / 16, value16 = (a.value_dim + 15) / 16;
  const int base = FIRST ? 0 : state.walks * steps, end = base + steps;  // steps made before, and after
  const float by = FIRST ? 1.f : state.by;
  if (FIRST && warp == Form::kFetcher && lane == 0) {
    // (by a warp other than the walked tiles': a copy takes 80 cycles to issue)
    load_kept<2, true>(&maps.k, k_tile, kv_head, unit.begin + unit.index * kTile, smem_addr(&sh.k_full));
    load_kept<VPANELS, false>(&maps.v, v_tile, kv_head, unit.begin + unit.index * kTile, smem_addr(&sh.v_full));
  }
  // Tensor memory: both maps' scores, their difference (two places by turns),
  // dout v^T, dv, both dk.  Both ds take dout v^T's place, half of each part's
  // columns each.  A warp may have made its difference or ds of the next
  // step before another has this one's, though not one more (the scores after it
  // wait for every warp's look at these): p_ready and ds_ready are two barriers
  // by turns.
  const uint32_t tmem = sh.tmem, dp_at = tmem + 192, dv_at = tmem + 256, dk_at = tmem + 384;
  auto diff_at = [&](int n) { return tmem + 128 + (n & 1) * 32; };

  // f16 holds probabilities times a power of two that leaves their difference,
  // at most 1 + |lambda| in size, below 2^15.
  const float largest = sh.largest;
  float shift = 0.f;
  if (kScaled<T>) shift = 14.f - (float)max(0, min(100, (__float_as_int(0.5f * (1.f + largest)) >> 23) - 126));
  const float unshift = exp2f(-shift), by_unshift = by * unshift, unscale = 1.f / by,
              per_largest = -1.f / largest;
  float* const stats = reinterpret_cast<float*>(tiles + kTilesKV);

  if (warp == Form::kFetcher) {
    // The queries' numbers, as the workers take them: a warp of its own has the
    // time to wait for them.
    int tile = 0, head = kv_head * group;
    wait_for_delta();
    for (int n = base; n < end; ++n) {
      const int stage = n % kStages;
      if (n >= kStages && !mbar_wait(smem_addr(&sh.empty[stage]), (n / kStages - 1) & 1, gave_up)) break;
      float* const to = stats + stage * kStats;
      const float lambda = a.lambda[head];
      float v[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (past the sequence's end, where all is masked: its last query's)
        const int query = min((first + tile) * kWalk + i * 32 + lane, unit.length - 1);
        const int64_t at = (int64_t)2 * head * a.tokens + unit.begin + query;
        v[i][0] = a.lse[at];
        v[i][1] = a.lse[at + a.tokens];
        v[i][2] = a.delta[at];
        v[i][3] = a.delta[at + a.tokens];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        to[i * 32 + lane] = fmaf(-v[i][0], kLog2e, shift);
        to[kWalk + i * 32 + lane] = fmaf(-v[i][1], kLog2e, shift);
        to[2 * kWalk + i * 32 + lane] = -v[i][2] * by_unshift;
        to[3 * kWalk + i * 32 + lane] = -v[i][3] * by_unshift * (lambda * per_largest);
      }
      if (lane == 0) to[4 * kWalk] = lambda;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.stats_full[stage]));
      if (++tile == per) tile = 0, ++head;
    }
  } else if (warp == Form::kLoader) {
    int head = kv_head * group, tile = 0;
    for (int n = base; n < end; ++n) {
      const int stage = n % kStages;
      if (n >= kStages && !mbar_wait(smem_addr(&sh.empty[stage]), (n / kStages - 1) & 1, gave_up)) break;
      const int query = (first + tile) * kWalk;
      if (!load_walked<2, true>(&maps.q, maps_at(q_tile, stage), head, unit.begin + query, unit.length - query,
                                smem_addr(&sh.q_full[stage]), smem_addr(&sh.own), &state.own_parity, gave_up) ||
          !load_walked<VPANELS, false>(&maps.dout, panels_at(do_tile, stage), head, unit.begin + query,
                                       unit.length - query, smem_addr(&sh.do_full[stage]), smem_addr(&sh.own),
                                       &state.own_parity, gave_up))
        break;
      if (++tile == per) tile = 0, ++head;
    }
  } else if (warp == Form::kIssuer) {
    if (elect_one()) {
      const uint32_t wide = mma_shape<T>(kWalk, false), keys = mma_shape<T>(dim16 * 16, true),
                     values = mma_shape<T>(value16 * 16, true);
      auto scores = [&](int n) {  // K_m Q_m^T
        if (!mbar_wait(smem_addr(&sh.q_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        for (int m = 0; m < 2; ++m)
          product_ss<4>(tmem + m * 64, k_tile + m * kPanelBytes, maps_at(q_tile, n % kStages) + m * kPart, wide, dim16);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // V dout^T
        if (!mbar_wait(smem_addr(&sh.do_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        product_ss<4 * VPANELS>(dp_at, v_tile, panels_at(do_tile, n % kStages), wide, value16);
        mma_commit(smem_addr(&sh.dp_full));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.k_full), 0, gave_up) && scores(base) &&
                mbar_wait(smem_addr(&sh.v_full), 0, gave_up) && dprob(base);
      for (int n = base; n < end && ok; ++n) {
        const bool more = n + 1 < end;
        // every warp's look at the scores is waited for in the last step too, so that phases keep in step
        if (!(ok = mbar_wait(smem_addr(&sh.s_read), n & 1, gave_up))) break;
        tc_fence_after();
        if (more && !(ok = scores(n + 1))) break;
        if (!(ok = mbar_wait(smem_addr(&sh.p_ready[n & 1]), (n >> 1) & 1, gave_up))) break;
        tc_fence_after();
        product_ts<4>(dv_at, diff_at(n), panels_at(do_tile, n % kStages), 0, values, n > base);
        if (!(ok = mbar_wait(smem_addr(&sh.ds_ready[n & 1]), (n >> 1) & 1, gave_up))) break;
        tc_fence_after();
        for (int m = 0; m < 2; ++m)
          for (int h = 0; h < kParts; ++h)
            product_ts<kCols / 16>(dk_at + m * 64, dp_at + h * kCols + m * kCols / 2, maps_at(q_tile, n % kStages) + m * kPart, h, keys,
                          n > base || h > 0);
        mma_commit(smem_addr(&sh.empty[n % kStages]));
        if (more) ok = dprob(n + 1);
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: key row, a part of the queries of each tile
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;
    const int left = unit.length - unit.index * kTile;  // queries from the first key to the sequence's end
    const uint32_t lane0 = (uint32_t)(warp & 3) << 21, s_at = tmem + lane0 + part * kCols;
    const float c = a.scale * kLog2e;
    int tile = 0;
    bool ok = true, finite = true;
    float most = kUnknown;
    for (int n = base; n < end; ++n) {
      const int from = tile * kWalk;  // the tile's first query, counted from the first key
      const bool masked = from < kTile || from + kWalk > left;
      auto step = [&](auto mask) {
        constexpr bool kMasked = decltype(mask)::value;
        auto seen = [&](int x) { return from + part * kCols + x >= row && from + part * kCols + x < left; };
        const float* at = stats + n % kStages * kStats + part * kCols;
        float p0[kCols], p1[kCols], d[kCols];
        uint32_t packed[kCols / 2];
        if (!mbar_wait(smem_addr(&sh.stats_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        const float lambda = stats[n % kStages * kStats + 4 * kWalk];
        if (!mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up)) return false;
        tc_fence_after();
        tmem_load16(s_at, p0);
        tmem_load16(s_at + 64, p1);
        tmem_wait_load();
        tmem_loaded(p0);
        tmem_loaded(p1);
        warp_arrive(smem_addr(&sh.s_read));
        probabilities<kMasked>(p0, c, [&](int x) { return two_of(at, x); }, seen);
        probabilities<kMasked>(p1, c, [&](int x) { return two_of(at + kWalk, x); }, seen);
        const Two less = two(-lambda, -lambda);
#pragma unroll
        for (int x = 0; x < kCols; x += 2) {
          float lo, hi;
          split(fma2(two(p1[x], p1[x + 1]), less, two(p0[x], p0[x + 1])), lo, hi);
          packed[x / 2] = pack2<T>(lo, hi);
        }
        // (dv's product of the step before last, which read this place, came before these scores)
        store_pairs(lane0 + diff_at(n) + part * (kCols / 2), packed);
        tmem_wait_store();
        warp_arrive(smem_addr(&sh.p_ready[n & 1]));
        const uint32_t dp = lane0 + dp_at + part * kCols;
        if (!mbar_wait(smem_addr(&sh.dp_full), n & 1, gave_up)) return false;
        tc_fence_after();
        tmem_load16(dp, d);
        tmem_wait_load();
        tmem_loaded(d);
        const float e0 = score_gradients<T, kMasked>(p0, d, packed, by_unshift, [&](int x) { return two_of(at + 2 * kWalk, x); });
        store_pairs(dp, packed);
        const float e1 = score_gradients<T, kMasked>(p1, d, packed, by_unshift * (lambda * per_largest),
                                                     [&](int x) { return two_of(at + 3 * kWalk, x); });
        store_pairs(dp + kCols / 2, packed);
        tmem_wait_store();
        warp_arrive(smem_addr(&sh.ds_ready[n & 1]));
        if (kScaled<T>) most = fmaxf(most, fmaxf(fabsf(e0), fabsf(e1)));
        return true;
      };
      if (!(ok = masked ? step(std::true_type()) : step(std::false_type()))) break;
      if (++tile == per) tile = 0;
    }
    if (ok && mbar_wait(smem_addr(&sh.done), FIRST ? 0 : state.walks & 1, gave_up)) {
      tc_fence_after();
      const int key = unit.index * kTile + (warp & 3) * 32;
      const uint32_t stage = q_tile + warp * 4096;
      auto place = [&](const AttnTensor& to, int head) {
        return static_cast<T*>(const_cast<void*>(to.ptr)) + (int64_t)(unit.begin + key) * to.token_stride +
               head * to.head_stride;
      };
      // both dk and the panels of dv
      for (int i = part; i < 2 + VPANELS; i += kParts) {
        if (i < 2)
          finite &= write_rows<T, 64>(lane0 + dk_at + i * 64, stage, place(a.dk, 2 * kv_head + i), a.dk.token_stride,
                                      unit.length - key, 0, a.dim, a.scale * unscale * (i ? largest : 1.f));
        else
          write_rows<T, 64>(lane0 + dv_at, stage, place(a.dv, kv_head), a.dv.token_stride, unit.length - key,
                            (i - 2) * 64, a.value_dim, unshift);
      }
    }
    put_most<T>(most, finite, sh.most);
  }
  return leave<T, Form>(&sh.gave_up, warp, tmem, sh.most, state);
}

template <class T, int VPANELS>
__device__ __forceinline__ void dkv_block(const Maps& maps, const DiffArgs& a, int block, uint8_t* tiles, SharedKV& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv_head = block % a.kv_heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, block / a.kv_heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == Form::kIssuer) {
    tmem_alloc(smem_addr(&sh.tmem), Form::kColumns);
  } else if (warp == Form::kLoader && lane == 0) {
    init_barriers(sh);
    prefetch_map(&maps.k);
    prefetch_map(&maps.q);
  } else if (warp == Form::kFetcher) {
    const int group = a.heads / a.kv_heads;
    float largest = 0x1p-100f;
    for (int h = lane; h < group; h += 32) largest = fmaxf(largest, fabsf(a.lambda[kv_head * group + h]));
    largest = warp_max(largest);
    if (lane == 0) sh.largest = largest;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.unit.count == 0) {
    if (warp == Form::kIssuer) tmem_free(sh.tmem, Form::kColumns);
    wait_for_delta();
    return;
  }
  State state;
  if (dkv_walk<T, VPANELS, true>(maps, a, kv_head, tiles, sh, state)) {
    if constexpr (kScaled<T>)
      while (dkv_walk<T, VPANELS, false>(maps, a, kv_head, tiles, sh, state)) {}
  }
}

// ---- dq ---------------------------------------------------------------------------

struct SharedQ {
  alignas(8) uint64_t q_full, do_full, kept, k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], s_full,
      s_read, dp_full[2], ds_ready[2], done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
  float most[Form::kWorkers / 32];
};

__device__ __forceinline__ void init_barriers(SharedQ& sh) {
  uint64_t* const one[] = {&sh.q_full, &sh.do_full, &sh.s_full, &sh.dp_full[0], &sh.dp_full[1], &sh.done, &sh.own};
  for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
  for (int i = 0; i < kKStages; ++i) {
    mbar_init(smem_addr(&sh.k_full[i]), 1);
    mbar_init(smem_addr(&sh.k_empty[i]), 1);
  }
  for (int i = 0; i < kVStages; ++i) {
    mbar_init(smem_addr(&sh.v_full[i]), 1);
    mbar_init(smem_addr(&sh.v_empty[i]), 1);
  }
  mbar_init(smem_addr(&sh.kept), Form::kWorkers / 32);
  mbar_init(smem_addr(&sh.s_read), Form::kWorkers / 32);
  for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&sh.ds_ready[i]), Form::kWorkers / 32);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// A walk over the keys, as dkv_walk.
template <class T, int VPANELS, bool FIRST>
__device__ __forceinline__ bool dq_walk(const Maps& maps, const DiffArgs& a, int head, uint8_t* tiles, SharedQ& sh,
                                        State& state) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqUnit unit = sh.unit;

  const uint32_t q_tile = smem_addr(tiles), do_tile = q_tile + 2 * kPanelBytes, k_tile = do_tile + 2 * kPanelBytes,
                 v_tile = k_tile + kKStages * kStageBytes;
  volatile int* gave_up = &sh.gave_up;
  const int query = unit.index * kTile;
  const int steps = min(query + kTile, unit.length + kWalk - 1) / kWalk;  // tiles of keys that the queries see
  const int dim16 = (a.dim + 15) / 16, value16 = (a.value_dim + 15) / 16;
  const int base = FIRST ? 0 : state.walks * steps, end = base + steps;  // steps made before, and after
  const float by = FIRST ? 1.f : state.by;
  if (FIRST && warp == Form::kFetcher && lane == 0) {
    load_kept<2, true>(&maps.q, q_tile, head, unit.begin + query, smem_addr(&sh.q_full));
    load_kept<VPANELS, false>(&maps.dout, do_tile, head, unit.begin + query, smem_addr(&sh.do_full));
  }
  // Tensor memory: both maps' scores, dout v^T (in two places by turns), both
  // dq, then the kept tiles q_0, q_1 and dout as pairs.  The next tile's scores and dout v^T are under way while this one's ds
  // are made.  So a warp may have finished the next step before another has this
  // one, though not one more: ds_ready is two barriers by turns.
  const uint32_t tmem = sh.tmem, dq_at = tmem + 256, q_at = tmem + 384, do_at = tmem + 448;
  auto dp_at = [&](int n) { return tmem + 128 + 64 * (n & 1); };

  if (warp == Form::kLoader) {
    const int kv_head = head / (a.heads / a.kv_heads);
    for (int n = base; n < end; ++n) {
      const int ks = n % kKStages, vs = n % kVStages, key = (n - base) * kWalk;
      if (n >= kKStages && !mbar_wait(smem_addr(&sh.k_empty[ks]), (n / kKStages - 1) & 1, gave_up)) break;
      // dq sums over the rows of K: those of another sequence are cleared
      if (!load_walked<2, true>(&maps.k, maps_at(k_tile, ks), kv_head, unit.begin + key, unit.length - key,
                                smem_addr(&sh.k_full[ks]), smem_addr(&sh.own), &state.own_parity, gave_up))
        break;
      if (n >= kVStages && !mbar_wait(smem_addr(&sh.v_empty[vs]), (n / kVStages - 1) & 1, gave_up)) break;
      if (!load_walked<VPANELS, false>(&maps.v, panels_at(v_tile, vs), kv_head, unit.begin + key, kWalk,
                                       smem_addr(&sh.v_full[vs]), smem_addr(&sh.own), &state.own_parity, gave_up))
        break;
    }
  } else if (warp == Form::kIssuer) {
    if (elect_one()) {
      const uint32_t wide = mma_shape<T>(kWalk, false), sums = mma_shape<T>(dim16 * 16, true);
      auto scores = [&](int n) {  // Q_m K_m^T
        if (!mbar_wait(smem_addr(&sh.k_full[n % kKStages]), (n / kKStages) & 1, gave_up)) return false;
        for (int m = 0; m < 2; ++m)
          product_tk<4>(tmem + m * 64, q_at + m * 32, maps_at(k_tile, n % kKStages) + m * kPart, wide, dim16);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // dout V^T
        if (!mbar_wait(smem_addr(&sh.v_full[n % kVStages]), (n / kVStages) & 1, gave_up)) return false;
        product_tk<4 * VPANELS>(dp_at(n), do_at, panels_at(v_tile, n % kVStages), wide, value16);
        mma_commit(smem_addr(&sh.dp_full[n & 1]));
        mma_commit(smem_addr(&sh.v_empty[n % kVStages]));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.kept), 0, gave_up);
      tc_fence_after();
      ok = ok && scores(base) && dprob(base);
      for (int n = base; n < end && ok; ++n) {
        if (!(ok = mbar_wait(smem_addr(&sh.s_read), n & 1, gave_up))) break;
        tc_fence_after();
        if (n + 1 < end && !(ok = scores(n + 1) && dprob(n + 1))) break;
        if (!(ok = mbar_wait(smem_addr(&sh.ds_ready[n & 1]), (n >> 1) & 1, gave_up))) break;
        tc_fence_after();
        for (int m = 0; m < 2; ++m)
          for (int h = 0; h < kParts; ++h)
            product_ts<kCols / 16>(dq_at + m * 64, dp_at(n) + h * kCols + m * kCols / 2, maps_at(k_tile, n % kKStages) + m * kPart, h, sums,
                          n > base || h > 0);
        mma_commit(smem_addr(&sh.k_empty[n % kKStages]));
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else if (warp < Form::kIssuer) {
    // thread: query row, a part of the keys of each tile
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane0 = (uint32_t)(warp & 3) << 21;
    const float c = a.scale * kLog2e;
    const bool valid = query + row < unit.length;
    wait_for_delta();
    const float lambda = a.lambda[head];
    const int64_t at = (int64_t)2 * head * a.tokens + unit.begin + query + row;
    Two lse[2], delta[2];
    for (int m = 0; m < 2; ++m) {
      const float l = valid ? -a.lse[at + m * a.tokens] * kLog2e : -INFINITY;
      const float dl = valid ? -a.delta[at + m * a.tokens] * by : 0.f;
      lse[m] = two(l, l);
      delta[m] = two(dl, dl);
    }
    bool ok = true;
    if (FIRST && (ok = mbar_wait(smem_addr(&sh.q_full), 0, gave_up) && mbar_wait(smem_addr(&sh.do_full), 0, gave_up))) {
      for (int i = part; i < 4; i += kParts) {  // half a panel of both
        keep_half(q_tile + (i >> 1) * kPanelBytes, row, i & 1, lane0 + q_at + i * 16);
        if (i < 2 * VPANELS) keep_half(do_tile + (i >> 1) * kPanelBytes, row, i & 1, lane0 + do_at + i * 16);
      }
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.kept));
    }
    bool finite = true;
    float most = 0.f;
    for (int n = base; n < end && ok; ++n) {
      const int key = (n - base) * kWalk;  // the tile's first
      const bool masked = key + kWalk > query;
      auto step = [&](auto mask) {
        constexpr bool kMasked = decltype(mask)::value;
        auto seen = [&](int x) { return key + part * kCols + x <= query + row; };
        if (!mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up)) return false;
        tc_fence_after();
        float p0[kCols], p1[kCols], d[kCols];
        uint32_t packed[kCols / 2];
        tmem_load16(lane0 + tmem + part * kCols, p0);
        tmem_load16(lane0 + tmem + 64 + part * kCols, p1);
        tmem_wait_load();
        tmem_loaded(p0);
        tmem_loaded(p1);
        warp_arrive(smem_addr(&sh.s_read));
        probabilities<kMasked>(p0, c, [&](int) { return lse[0]; }, seen);
        probabilities<kMasked>(p1, c, [&](int) { return lse[1]; }, seen);
        const uint32_t dp = lane0 + dp_at(n) + part * kCols;
        if (!mbar_wait(smem_addr(&sh.dp_full[n & 1]), (n >> 1) & 1, gave_up)) return false;
        tc_fence_after();
        tmem_load16(dp, d);
        tmem_wait_load();
        tmem_loaded(d);
        const float e0 = score_gradients<T, kMasked>(p0, d, packed, by, [&](int) { return delta[0]; });
        store_pairs(dp, packed);
        const float e1 = score_gradients<T, kMasked>(p1, d, packed, by, [&](int) { return delta[1]; });
        store_pairs(dp + kCols / 2, packed);
        tmem_wait_store();
        warp_arrive(smem_addr(&sh.ds_ready[n & 1]));
        if (kScaled<T>) most = fmaxf(most, fmaxf(fabsf(e0), fabsf(e1)));
        return true;
      };
      if (!(ok = masked ? step(std::true_type()) : step(std::false_type()))) break;
    }
    if (ok && mbar_wait(smem_addr(&sh.done), FIRST ? 0 : state.walks & 1, gave_up)) {
      tc_fence_after();
      const int from = query + (warp & 3) * 32;
      for (int i = part; i < 4; i += kParts) {  // 32 columns of one map's
        const int m = i >> 1;
        T* out = static_cast<T*>(const_cast<void*>(a.dq.ptr)) + (int64_t)(unit.begin + from) * a.dq.token_stride +
                 (2 * head + m) * a.dq.head_stride;
        finite &= write_rows<T, 32>(lane0 + dq_at + m * 64, k_tile + warp * 2048, out, a.dq.token_stride,
                                    unit.length - from, (i & 1) * 32, a.dim,
                                    a.scale * (1.f / by) * (m ? -lambda : 1.f));
      }
    }
    if (kScaled<T> && FIRST && ok && !__any_sync(0xFFFFFFFFu, most > 0.f)) {
      // a prompt's queries often have no gradient at all, and need no other power
      ok = mbar_wait(smem_addr(&sh.do_full), 0, gave_up);
      for (int i = part; valid && i < 2 * VPANELS; i += kParts)
        if (any_element(do_tile + (i >> 1) * kPanelBytes + row * 128 + (i & 1) * 64)) most = kUnknown;
    }
    put_most<T>(most, finite, sh.most);
  }
  return leave<T, Form>(&sh.gave_up, warp, tmem, sh.most, state);
}

template <class T, int VPANELS>
__device__ __forceinline__ void dq_block(const Maps& maps, const DiffArgs& a, int block, uint8_t* tiles, SharedQ& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = block % a.heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, block / a.heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == Form::kIssuer) {
    tmem_alloc(smem_addr(&sh.tmem), Form::kColumns);
  } else if (warp == Form::kLoader && lane == 0) {
    init_barriers(sh);
    prefetch_map(&maps.k);
    prefetch_map(&maps.q);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.unit.count == 0) {
    if (warp == Form::kIssuer) tmem_free(sh.tmem, Form::kColumns);
    wait_for_delta();
    return;
  }
  State state;
  if (dq_walk<T, VPANELS, true>(maps, a, head, tiles, sh, state)) {
    if constexpr (kScaled<T>)
      while (dq_walk<T, VPANELS, false>(maps, a, head, tiles, sh, state)) {}
  }
}

// ---- all ----------------------------------------------------------------------------

union Shared {
  SharedKV kv;
  SharedQ q;
  float part[Form::kThreads / 32];
  __device__ Shared() {}
};

// One launch: first the blocks of dk and dv, then those of dq, which fill the
// first ones' last wave, then those of dlambda.
template <class T, int VPANELS>
__global__ void __launch_bounds__(Form::kThreads, 1)
    diff_attention_backward_kernel(const __grid_constant__ Maps maps, const __grid_constant__ DiffArgs a, int kv_blocks,
                                   int q_blocks) {
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ Shared sh;
  const int block = blockIdx.x;
  if (block < kv_blocks) dkv_block<T, VPANELS>(maps, a, block, tiles, sh.kv);
  else if (block - kv_blocks < q_blocks) dq_block<T, VPANELS>(maps, a, block - kv_blocks, tiles, sh.q);
  else dlambda_block(a, block - kv_blocks - q_blocks, sh.part);
}

template <class T, int VPANELS>
cudaError_t run(int dtype, const DiffArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  auto* kernel = diff_attention_backward_kernel<T, VPANELS>;
  cudaError_t e = open_kernel((const void*)kernel, kSmem, false, opened);
  if (e != cudaSuccess) return e;
  Maps maps;
  if (!make_tensor_map(&maps.q, dtype, a.q, a.tokens, 2 * a.heads, a.dim, kWalk) ||
      !make_tensor_map(&maps.k, dtype, a.k, a.tokens, 2 * a.kv_heads, a.dim, kWalk) ||
      !make_tensor_map(&maps.v, dtype, a.v, a.tokens, a.kv_heads, a.value_dim, kWalk) ||
      !make_tensor_map(&maps.dout, dtype, a.dout, a.tokens, a.heads, a.value_dim, kWalk))
    return cudaErrorInvalidValue;
  constexpr int kLanes = VPANELS * 8, kRows = 256 / kLanes;
  diff_delta_kernel<T, kLanes><<<(unsigned)((a.tokens * a.heads + kRows - 1) / kRows), 256, 0, s>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t most = most_units(a.tokens, a.seqs, kTile);
  const int kv_blocks = (int)(most * a.kv_heads), q_blocks = (int)(most * a.heads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kv_blocks + q_blocks + (a.dlambda ? a.heads : 0)));
  cfg.blockDim = dim3(Form::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, maps, a, kv_blocks, q_blocks);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_diff_attention_backward(int dtype, const DiffArgs& a, cudaStream_t s) {
  if (dtype == BF16) return a.value_dim <= 64 ? run<__nv_bfloat16, 1>(dtype, a, s) : run<__nv_bfloat16, 2>(dtype, a, s);
  return a.value_dim <= 64 ? run<__half, 1>(dtype, a, s) : run<__half, 2>(dtype, a, s);
}

cudaError_t diff_attention_backward_take_status(int* status, cudaStream_t s) { return take_status(status, s); }

}  // namespace ar
