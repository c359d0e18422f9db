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
// memory: two threads have a row's 64 columns.  The difference of probabilities
// has a place of its own (two by turns), so the next scores are computed as soon
// as the current ones have been read; both ds take dp's place, as 16-bit pairs.
//
// lambda may differ from one by any factor, and f16 would lose what it makes
// small: ds_1 is held without it in dq's blocks and relative to the group's
// largest in dk's, and the sums are multiplied by the rest.
#include "ar_attention_backward.cuh"

#include <algorithm>

namespace ar {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

constexpr int kWalk = 64;
constexpr uint32_t kPart = kWalk * 128;       // bytes of a panel of a walked tile
constexpr uint32_t kStageBytes = 2 * kPart;   // of a walked tile
constexpr int kStages = 4;                    // tiles of q and of dout in flight, for dk and dv
constexpr int kKStages = 4, kVStages = 4;     // of k and v, for dq
constexpr int kStats = 8 * 32;                // floats of a worker warp: [turn][lse 0, lse 1, delta 0, delta 1][32]

struct Form {
  static constexpr int kWorkers = 256;  // threads: 128 rows, two halves of the columns
  static constexpr int kIssuer = 8, kLoader = 9;
  static constexpr int kThreads = 320;
  static constexpr int kColumns = 512;
};
// shared memory of both kinds of block
constexpr uint32_t kTilesKV = 4 * kPanelBytes + 2 * kStages * kStageBytes;
constexpr uint32_t kTilesQ = 4 * kPanelBytes + (kKStages + kVStages) * kStageBytes;
constexpr uint32_t kSmem = kTilesKV + Form::kWorkers / 32 * kStats * 4;
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

// The kept tile of both maps (PANELS 2, a panel each), or of v or dout.
template <int PANELS, bool BOTH_MAPS>
__device__ __forceinline__ void load_kept(const CUtensorMap* map, uint32_t dst, int head, int token, uint32_t bar) {
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

// ---- a worker's arithmetic ----------------------------------------------------------

// 32 scores become probabilities 2^(c s - lse) in place.
template <class L, class S>
__device__ __forceinline__ void probabilities(float (&p)[32], float c, L lse, bool masked, S seen) {
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
}

// Pairs of ds = p (by d + minus_delta).  What is not seen has p = 0 and no ds,
// whatever d holds there.  The first is returned, where f16 looks at it.
template <class T, class L>
__device__ __forceinline__ float score_gradients(const float (&p)[32], const float (&d)[32], uint32_t (&packed)[16],
                                                 float by, L minus_delta, bool masked) {
  const Two by2 = two(by, by);
  float first = 0.f;
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    float lo, hi;
    split(mul2(two(p[x], p[x + 1]), fma2(two(d[x], d[x + 1]), by2, minus_delta(x))), lo, hi);
    if (masked) {
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
  alignas(8) uint64_t kv_full, q_full[kStages], do_full[kStages], empty[kStages], s_full, s_read, dp_full, p_ready[2],
      ds_ready[2], done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
  float most[Form::kWorkers / 32];  // what each worker warp has seen of the score gradients
};

__device__ __forceinline__ void init_barriers(SharedKV& sh) {
  uint64_t* const one[] = {&sh.kv_full, &sh.s_full, &sh.dp_full, &sh.done, &sh.own};
  for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
  for (int i = 0; i < kStages; ++i) {
    mbar_init(smem_addr(&sh.q_full[i]), 1);
    mbar_init(smem_addr(&sh.do_full[i]), 1);
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
  if (FIRST && warp == Form::kLoader && lane == 0) {
    const uint32_t bar = smem_addr(&sh.kv_full);
    mbar_expect(bar, (2 + VPANELS) * kPanelBytes);
    load_kept<2, true>(&maps.k, k_tile, kv_head, unit.begin + unit.index * kTile, bar);
    load_kept<VPANELS, false>(&maps.v, v_tile, kv_head, unit.begin + unit.index * kTile, bar);
  }
  // Tensor memory: both maps' scores, their difference (two places by turns),
  // dout v^T, dv, both dk.  Both ds take dout v^T's place, of each half's 32
  // columns 16 each.
  const uint32_t tmem = sh.tmem, dp_at = tmem + 192, dv_at = tmem + 256, dk_at = tmem + 384;
  auto diff_at = [&](int n) { return tmem + 128 + (n & 1) * 32; };

  if (warp == Form::kLoader) {
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
      bool ok = mbar_wait(smem_addr(&sh.kv_full), 0, gave_up) && scores(base) && dprob(base);
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
          for (int h = 0; h < 2; ++h)
            product_ts<2>(dk_at + m * 64, dp_at + h * 32 + m * 16, maps_at(q_tile, n % kStages) + m * kPart, h, keys,
                          n > base || h > 0);
        mma_commit(smem_addr(&sh.empty[n % kStages]));
        if (more) ok = dprob(n + 1);
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: key row, queries [32 half, 32 half + 32) of each tile
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const int left = unit.length - unit.index * kTile;  // queries from the first key to the sequence's end
    const uint32_t lane0 = (uint32_t)(warp & 3) << 21, s_at = tmem + lane0 + half * 32;
    const float c = a.scale * kLog2e;
    float* stats = reinterpret_cast<float*>(tiles + kTilesKV) + warp * kStats;
    // The group's largest lambda; f16 holds probabilities times a power of two
    // that leaves their difference, at most 1 + |lambda| in size, below 2^15.
    float largest = 0.f;
    for (int h = 0; h < group; ++h) largest = fmaxf(largest, fabsf(a.lambda[kv_head * group + h]));
    float shift = 0.f;
    if (kScaled<T>) shift = 14.f - (float)max(0, min(100, (__float_as_int(0.5f * (1.f + largest)) >> 23) - 126));
    const float unshift = exp2f(-shift), by_unshift = by * unshift, unscale = 1.f / by;
    // Each warp fetches its 32 queries' numbers for itself: four warps that
    // shared them would meet at every step.
    int next_tile = 0, next_head = kv_head * group;
    float next_lambda = 0.f;
    auto fetch = [&]() {  // of the next step, and on
      const int query = (first + next_tile) * kWalk + half * 32 + lane;
      const int64_t at = (int64_t)2 * next_head * a.tokens + unit.begin + query;
      const float l = a.lambda[next_head], relative = largest > 0.f ? -l / largest : 0.f;
      next_lambda = l;
      if (++next_tile == per) next_tile = 0, ++next_head;
      if (query >= unit.length) return make_float4(0.f, 0.f, 0.f, 0.f);  // masked
      return make_float4(fmaf(-a.lse[at], kLog2e, shift), fmaf(-a.lse[at + a.tokens], kLog2e, shift),
                         -a.delta[at] * by_unshift, -a.delta[at + a.tokens] * by_unshift * relative);
    };
    auto put = [&](int n, float4 v) {
      float* to = stats + (n & 1) * 128 + lane;
      to[0] = v.x;
      to[32] = v.y;
      to[64] = v.z;
      to[96] = v.w;
      __syncwarp();
    };
    wait_for_delta();
    put(base, fetch());
    float lambda = next_lambda;
    int tile = 0;
    bool ok = true, finite = true;
    float most = kUnknown;
    for (int n = base; n < end; ++n) {
      const float4 next = n + 1 < end ? fetch() : make_float4(0.f, 0.f, 0.f, 0.f);
      const int from = tile * kWalk;  // the tile's first query, counted from the first key
      const bool masked = from < kTile || from + kWalk > left;
      auto seen = [&](int x) { return from + half * 32 + x >= row && from + half * 32 + x < left; };
      const float* at = stats + (n & 1) * 128;
      if (!(ok = mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up))) break;
      tc_fence_after();
      float p0[32], p1[32], d[32];
      uint32_t packed[16];
      tmem_load32(s_at, p0);
      tmem_load32(s_at + 64, p1);
      tmem_wait_load();
      tmem_loaded(p0);
      tmem_loaded(p1);
      warp_arrive(smem_addr(&sh.s_read));
      probabilities(p0, c, [&](int x) { return two_of(at, x); }, masked, seen);
      probabilities(p1, c, [&](int x) { return two_of(at + 32, x); }, masked, seen);
      const Two less = two(-lambda, -lambda);
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        float lo, hi;
        split(fma2(two(p1[x], p1[x + 1]), less, two(p0[x], p0[x + 1])), lo, hi);
        packed[x / 2] = pack2<T>(lo, hi);
      }
      // (dv's product of the step before last, which read this place, came before these scores)
      tmem_store16(lane0 + diff_at(n) + half * 16, packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.p_ready[n & 1]));
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full), n & 1, gave_up))) break;
      tc_fence_after();
      tmem_load32(lane0 + dp_at + half * 32, d);
      tmem_wait_load();
      tmem_loaded(d);
      const float e0 = score_gradients<T>(p0, d, packed, by_unshift, [&](int x) { return two_of(at + 64, x); }, masked);
      tmem_store16(lane0 + dp_at + half * 32, packed);
      const float e1 = score_gradients<T>(p1, d, packed, largest > 0.f ? by_unshift * (-lambda / largest) : 0.f,
                                          [&](int x) { return two_of(at + 96, x); }, masked);
      tmem_store16(lane0 + dp_at + half * 32 + 16, packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.ds_ready[n & 1]));
      if (kScaled<T>) most = fmaxf(most, fmaxf(fabsf(e0), fabsf(e1)));
      put(n + 1, next);
      lambda = next_lambda;
      if (++tile == per) tile = 0;
    }
    if (ok && mbar_wait(smem_addr(&sh.done), FIRST ? 0 : state.walks & 1, gave_up)) {
      tc_fence_after();
      // half: dv, or both dk
      const int key = unit.index * kTile + (warp & 3) * 32;
      const uint32_t stage = q_tile + warp * 4096;
      auto place = [&](const AttnTensor& to, int head) {
        return static_cast<T*>(const_cast<void*>(to.ptr)) + (int64_t)(unit.begin + key) * to.token_stride +
               head * to.head_stride;
      };
      if (half == 0) {
        for (int p = 0; p < VPANELS; ++p)
          write_rows<T, 64>(lane0 + dv_at, stage, place(a.dv, kv_head), a.dv.token_stride, unit.length - key, p * 64,
                            a.value_dim, unshift);
      } else {
        for (int m = 0; m < 2; ++m)
          finite &= write_rows<T, 64>(lane0 + dk_at + m * 64, stage, place(a.dk, 2 * kv_head + m), a.dk.token_stride,
                                      unit.length - key, 0, a.dim, a.scale * unscale * (m ? largest : 1.f));
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
  alignas(8) uint64_t q_full, k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], s_full, s_read,
      dp_full[2], ds_ready[2], done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
  float most[Form::kWorkers / 32];
};

__device__ __forceinline__ void init_barriers(SharedQ& sh) {
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
  if (FIRST && warp == Form::kLoader && lane == 0) {
    const uint32_t bar = smem_addr(&sh.q_full);
    mbar_expect(bar, (2 + VPANELS) * kPanelBytes);
    load_kept<2, true>(&maps.q, q_tile, head, unit.begin + query, bar);
    load_kept<VPANELS, false>(&maps.dout, do_tile, head, unit.begin + query, bar);
  }
  // Tensor memory: both maps' scores, dout v^T (in two places by turns), both
  // dq.  The next tile's scores and dout v^T are under way while this one's ds
  // are made.  So a warp may have finished the next step before another has this
  // one, though not one more: ds_ready is two barriers by turns.
  const uint32_t tmem = sh.tmem, dq_at = tmem + 256;
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
          product_ss<4>(tmem + m * 64, q_tile + m * kPanelBytes, maps_at(k_tile, n % kKStages) + m * kPart, wide, dim16);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // dout V^T
        if (!mbar_wait(smem_addr(&sh.v_full[n % kVStages]), (n / kVStages) & 1, gave_up)) return false;
        product_ss<4 * VPANELS>(dp_at(n), do_tile, panels_at(v_tile, n % kVStages), wide, value16);
        mma_commit(smem_addr(&sh.dp_full[n & 1]));
        mma_commit(smem_addr(&sh.v_empty[n % kVStages]));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.q_full), 0, gave_up) && scores(base) && dprob(base);
      for (int n = base; n < end && ok; ++n) {
        if (!(ok = mbar_wait(smem_addr(&sh.s_read), n & 1, gave_up))) break;
        tc_fence_after();
        if (n + 1 < end && !(ok = scores(n + 1) && dprob(n + 1))) break;
        if (!(ok = mbar_wait(smem_addr(&sh.ds_ready[n & 1]), (n >> 1) & 1, gave_up))) break;
        tc_fence_after();
        for (int m = 0; m < 2; ++m)
          for (int h = 0; h < 2; ++h)
            product_ts<2>(dq_at + m * 64, dp_at(n) + h * 32 + m * 16, maps_at(k_tile, n % kKStages) + m * kPart, h, sums,
                          n > base || h > 0);
        mma_commit(smem_addr(&sh.k_empty[n % kKStages]));
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: query row, keys [32 half, 32 half + 32) of each tile
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane0 = (uint32_t)(warp & 3) << 21;
    const float c = a.scale * kLog2e;
    const bool valid = query + row < unit.length;
    wait_for_delta();
    const int64_t at = (int64_t)2 * head * a.tokens + unit.begin + query + row;
    Two lse[2], delta[2];
    for (int m = 0; m < 2; ++m) {
      const float l = valid ? -a.lse[at + m * a.tokens] * kLog2e : -INFINITY;
      const float dl = valid ? -a.delta[at + m * a.tokens] * by : 0.f;
      lse[m] = two(l, l);
      delta[m] = two(dl, dl);
    }
    bool ok = true, finite = true;
    float most = 0.f;
    for (int n = base; n < end; ++n) {
      const int key = (n - base) * kWalk;  // the tile's first
      const bool masked = key + kWalk > query;
      auto seen = [&](int x) { return key + half * 32 + x <= query + row; };
      if (!(ok = mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up))) break;
      tc_fence_after();
      float p0[32], p1[32], d[32];
      uint32_t packed[16];
      tmem_load32(lane0 + tmem + half * 32, p0);
      tmem_load32(lane0 + tmem + 64 + half * 32, p1);
      tmem_wait_load();
      tmem_loaded(p0);
      tmem_loaded(p1);
      warp_arrive(smem_addr(&sh.s_read));
      probabilities(p0, c, [&](int) { return lse[0]; }, masked, seen);
      probabilities(p1, c, [&](int) { return lse[1]; }, masked, seen);
      const uint32_t dp = lane0 + dp_at(n) + half * 32;
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full[n & 1]), (n >> 1) & 1, gave_up))) break;
      tc_fence_after();
      tmem_load32(dp, d);
      tmem_wait_load();
      tmem_loaded(d);
      const float e0 = score_gradients<T>(p0, d, packed, by, [&](int) { return delta[0]; }, masked);
      tmem_store16(dp, packed);
      const float e1 = score_gradients<T>(p1, d, packed, by, [&](int) { return delta[1]; }, masked);
      tmem_store16(dp + 16, packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.ds_ready[n & 1]));
      if (kScaled<T>) most = fmaxf(most, fmaxf(fabsf(e0), fabsf(e1)));
    }
    if (ok && mbar_wait(smem_addr(&sh.done), FIRST ? 0 : state.walks & 1, gave_up)) {
      tc_fence_after();
      // half: which map
      const int from = query + (warp & 3) * 32;
      T* out = static_cast<T*>(const_cast<void*>(a.dq.ptr)) + (int64_t)(unit.begin + from) * a.dq.token_stride +
               (2 * head + half) * a.dq.head_stride;
      finite = write_rows<T, 64>(lane0 + dq_at + half * 64, k_tile + warp * 4096, out, a.dq.token_stride,
                                 unit.length - from, 0, a.dim, a.scale * (1.f / by) * (half ? -a.lambda[head] : 1.f));
    }
    if (kScaled<T> && FIRST && ok && !__any_sync(0xFFFFFFFFu, most > 0.f)) {
      // a prompt's queries often have no gradient at all, and need no other power
      ok = mbar_wait(smem_addr(&sh.q_full), 0, gave_up);
      if (valid)
        for (int p = 0; p < VPANELS; ++p)
          if (any_element(do_tile + p * kPanelBytes + row * 128 + half * 64)) most = kUnknown;
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
