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
// In both, sixteen warps take the exponentials: four threads share a row of
// the tile, 32 columns each.  p and ds take the places of the scores and of
// dout v^T in tensor memory, as 16-bit pairs, and are the left operands of the
// sums' products there.  The next tiles' products are issued between the
// current one's sums, so the tensor cores work while exponentials are taken.
#include "ar_tcgen05.cuh"

#include <algorithm>

#include "../../include/ar.h"

namespace ar {
namespace {

__device__ int g_status;  // AR_ERR_TIMEOUT once a wait has run out

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 576;
constexpr int kIssuer = 16, kLoader = 17;  // warps
constexpr int kWorkers = 512;              // threads of the others

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

// Writes 16 columns of a thread's row of sums, times `scale`, rounded.
template <class T>
__device__ __forceinline__ void write16(uint32_t from, T* row, int column, int dim, float scale, bool valid) {
  float o[16];
  tmem_load16(from + column, o);
  tmem_wait_load();
  tmem_loaded(o);
  if (!valid) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (column + h * 8 >= dim) break;
    *reinterpret_cast<uint4*>(row + column + h * 8) =
        make_uint4(pack2<T>(o[h * 8] * scale, o[h * 8 + 1] * scale), pack2<T>(o[h * 8 + 2] * scale, o[h * 8 + 3] * scale),
                   pack2<T>(o[h * 8 + 4] * scale, o[h * 8 + 5] * scale), pack2<T>(o[h * 8 + 6] * scale, o[h * 8 + 7] * scale));
  }
}

__device__ __forceinline__ void leave(int* gave_up, int warp, uint32_t tmem) {
  tc_fence_before();
  __syncthreads();
  if (*(volatile int*)gave_up) {
    // copies and products in flight end by themselves: give them time
    for (int i = 0; i < 100; ++i) __nanosleep(100000);
    if (threadIdx.x == 0) g_status = AR_ERR_TIMEOUT;
    __syncthreads();
  }
  if (warp == kIssuer) tmem_free(tmem, 512);
}

// 32 scores of a thread become probabilities 2^(c s - lse) in place, and pairs
// of them in `packed`; `seen` is asked in the tile on the diagonal alone.
template <class T, class L, class S>
__device__ __forceinline__ void probabilities(float (&p)[32], uint32_t (&packed)[16], float c, L lse, bool diagonal,
                                              S seen) {
  const Two c2 = two(c, c);
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    split(fma2(two(p[x], p[x + 1]), c2, lse(x)), p[x], p[x + 1]);
    p[x] = exp2_approx(p[x]);
    p[x + 1] = exp2_approx(p[x + 1]);
  }
  if (diagonal) {
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (!seen(x)) p[x] = 0.f;
  }
#pragma unroll
  for (int x = 0; x < 32; x += 2) packed[x / 2] = pack2<T>(p[x], p[x + 1]);
}

// Pairs of ds = p (d - delta).  What is not seen has p = 0 and no ds, whatever
// d holds there (tokens of another sequence, in the tile on the diagonal).
template <class T, class L>
__device__ __forceinline__ void score_gradients(float (&p)[32], float (&d)[32], uint32_t (&packed)[16], L minus_delta,
                                                bool diagonal) {
  if (diagonal) {
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (p[x] == 0.f) d[x] = 0.f;
  }
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    float lo, hi;
    split(mul2(two(p[x], p[x + 1]), add2(two(d[x], d[x + 1]), minus_delta(x))), lo, hi);
    packed[x / 2] = pack2<T>(lo, hi);
  }
}

struct Maps {
  CUtensorMap q, k, v, dout;
};

// ---- dk and dv ---------------------------------------------------------------------

constexpr int kMostStages = 4;

// Tiles of queries (q and dout) in flight: as many as fit beside k and v.
__host__ __device__ constexpr int query_stages(int panels) { return panels == 1 ? kMostStages : 2; }

struct SharedKV {
  alignas(8) uint64_t kv_full, q_full[kMostStages], do_full[kMostStages], empty[kMostStages], s_full, s_read, dp_full,
      dp_read, p_ready, ds_ready, dv_done, dk_done, done, own;
  alignas(16) float lse[2][4][32], delta[2][4][32];  // [turn][quarter]
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
};

template <class T, int PANELS>
__device__ __forceinline__ void dkv_block(const Maps& maps, const AttnArgs& a, int block, uint8_t* tiles, SharedKV& sh) {
  constexpr int kStages = query_stages(PANELS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv_head = block % a.kv_heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, block / a.kv_heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == kLoader && lane == 0) {
    uint64_t* const one[] = {&sh.kv_full, &sh.s_full, &sh.dp_full, &sh.dv_done, &sh.dk_done, &sh.done, &sh.own};
    for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&sh.q_full[i]), 1);
      mbar_init(smem_addr(&sh.do_full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    uint64_t* const all[] = {&sh.s_read, &sh.dp_read, &sh.p_ready, &sh.ds_ready};
    for (uint64_t* b : all) mbar_init(smem_addr(b), kWorkers / 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (sh.unit.count == 0) return;
  SeqUnit unit = sh.unit;
  unit.index = unit.count - 1 - unit.index;  // the first keys are seen by the most queries

  constexpr uint32_t kTileBytes = PANELS * kPanelBytes;
  const uint32_t k_tile = smem_addr(tiles), v_tile = k_tile + kTileBytes, q_tile = v_tile + kTileBytes,
                 do_tile = q_tile + kStages * kTileBytes;
  volatile int* gave_up = &sh.gave_up;
  if (warp == kIssuer) tmem_alloc(smem_addr(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // Tensor memory: scores 0, dout v^T 128, dv 256.  Heads of up to 64 leave
  // room for p and ds beside them, so that the next tile's products run as
  // soon as the current scores and dout v^T have been read; otherwise they
  // take those places, each quarter's 16 columns of pairs at the front of the
  // 32 that it read.
  constexpr bool kApart = PANELS == 1;
  const uint32_t dv_at = tmem + 256, dk_at = tmem + (kApart ? 320 : 384);
  auto p_at = [&](int quarter) { return tmem + (kApart ? 384 + quarter * 16 : quarter * 32); };
  auto ds_at = [&](int quarter) { return tmem + (kApart ? 448 + quarter * 16 : 128 + quarter * 32); };

  // step n: head n / per of the group, tile of queries unit.index + n % per
  const int group = a.heads / a.kv_heads, per = unit.count - unit.index, steps = group * per;
  const int dim16 = (a.dim + 15) / 16;

  if (warp == kLoader) {
    if (lane == 0) {
      const uint32_t bar = smem_addr(&sh.kv_full);
      mbar_expect(bar, 2 * kTileBytes);
      for (int p = 0; p < PANELS; ++p) {
        tma_load(k_tile + p * kPanelBytes, &maps.k, p * 64, kv_head, unit.begin + unit.index * kTile, bar);
        tma_load(v_tile + p * kPanelBytes, &maps.v, p * 64, kv_head, unit.begin + unit.index * kTile, bar);
      }
    }
    uint32_t own_parity = 0;
    for (int n = 0; n < steps; ++n) {
      const int stage = n % kStages;
      if (n >= kStages && !mbar_wait(smem_addr(&sh.empty[stage]), (n / kStages - 1) & 1, gave_up)) break;
      const int head = kv_head * group + n / per, query = (unit.index + n % per) * kTile;
      if (!load_tile(&maps.q, q_tile + stage * kTileBytes, PANELS, head, unit.begin + query, unit.length - query,
                     smem_addr(&sh.q_full[stage]), smem_addr(&sh.own), &own_parity, gave_up) ||
          !load_tile(&maps.dout, do_tile + stage * kTileBytes, PANELS, head, unit.begin + query, unit.length - query,
                     smem_addr(&sh.do_full[stage]), smem_addr(&sh.own), &own_parity, gave_up))
        break;
    }
  } else if (warp == kIssuer) {
    if (elect_one()) {
      const uint32_t wide = mma_shape<T>(kTile, false), sums = mma_shape<T>(dim16 * 16, true);
      auto at = [&](uint32_t tile, int n) { return tile + (n % kStages) * kTileBytes; };
      auto scores = [&](int n) {  // K Q^T
        if (!mbar_wait(smem_addr(&sh.q_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(tmem, k_tile, at(q_tile, n), wide, dim16);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // V dout^T
        if (!mbar_wait(smem_addr(&sh.do_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(tmem + 128, v_tile, at(do_tile, n), wide, dim16);
        mma_commit(smem_addr(&sh.dp_full));
        return true;
      };
      auto ready = [&](uint64_t& bar, int n) {
        if (!mbar_wait(smem_addr(&bar), n & 1, gave_up)) return false;
        tc_fence_after();
        return true;
      };
      auto sum_dv = [&](int n) {
        if (!ready(sh.p_ready, n)) return false;
        for (int h = 0; h < 4; ++h) product_ts<2>(dv_at, p_at(h), at(do_tile, n), h, sums, n > 0 || h > 0);
        if (kApart) mma_commit(smem_addr(&sh.dv_done));
        return true;
      };
      auto sum_dk = [&](int n) {
        if (!ready(sh.ds_ready, n)) return false;
        for (int h = 0; h < 4; ++h) product_ts<2>(dk_at, ds_at(h), at(q_tile, n), h, sums, n > 0 || h > 0);
        if (kApart) mma_commit(smem_addr(&sh.dk_done));
        mma_commit(smem_addr(&sh.empty[n % kStages]));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.kv_full), 0, gave_up) && scores(0) && dprob(0);
      for (int n = 0; n < steps && ok; ++n) {
        const bool more = n + 1 < steps;
        if constexpr (kApart) {
          ok = (!more || (ready(sh.s_read, n) && scores(n + 1))) && sum_dv(n) &&
               (!more || (ready(sh.dp_read, n) && dprob(n + 1))) && sum_dk(n);
        } else {
          ok = sum_dv(n) && (!more || scores(n + 1)) && sum_dk(n) && (!more || dprob(n + 1));
        }
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: key row, queries [32 quarter, 32 quarter + 32) of each tile
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane, t = threadIdx.x & 127;
    const uint32_t lane0 = (uint32_t)(warp & 3) << 21, s_at = tmem + lane0 + quarter * 32;
    const float c = a.scale * kLog2e;
    // threads 0..31 of a quarter fetch its queries' -lse in powers of two, the next 32 their -delta
    auto fetch = [&](int n) {
      const int query = (unit.index + n % per) * kTile + quarter * 32 + (t & 31);
      if (t >= 64) return 0.f;
      if (query >= unit.length) return t < 32 ? -INFINITY : 0.f;  // p = 0 after the sequence's end
      const int64_t at = (int64_t)(kv_head * group + n / per) * a.tokens + unit.begin + query;
      return t < 32 ? -a.lse[at] * kLog2e : -a.delta[at];
    };
    auto put = [&](int n, float v) {
      if (t < 64) (t < 32 ? sh.lse : sh.delta)[n & 1][quarter][t & 31] = v;
      named_barrier(1 + quarter, 128);
    };
    put(0, fetch(0));
    bool ok = true;
    for (int n = 0; n < steps; ++n) {
      const float next = n + 1 < steps ? fetch(n + 1) : 0.f;
      const bool diagonal = n % per == 0;
      if (!(ok = mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up))) break;
      tc_fence_after();
      float p[32], d[32];
      uint32_t packed[16];
      tmem_load32(s_at, p);
      tmem_wait_load();
      tmem_loaded(p);
      if constexpr (kApart) {
        warp_arrive(smem_addr(&sh.s_read));
      }
      const float* lse = sh.lse[n & 1][quarter];
      probabilities<T>(p, packed, c, [&](int x) { return Two{*reinterpret_cast<const uint64_t*>(lse + x)}; }, diagonal,
                       [&](int x) { return quarter * 32 + x >= row; });
      if (kApart && n > 0) {
        // the last sums have read what these replace
        if (!(ok = mbar_wait(smem_addr(&sh.dv_done), (n - 1) & 1, gave_up))) break;
        tc_fence_after();
      }
      tmem_store16(lane0 + p_at(quarter), packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.p_ready));
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full), n & 1, gave_up))) break;
      tc_fence_after();
      tmem_load32(s_at + 128, d);
      tmem_wait_load();
      tmem_loaded(d);
      if constexpr (kApart) {
        warp_arrive(smem_addr(&sh.dp_read));
      }
      const float* delta = sh.delta[n & 1][quarter];
      score_gradients<T>(p, d, packed, [&](int x) { return Two{*reinterpret_cast<const uint64_t*>(delta + x)}; }, diagonal);
      if (kApart && n > 0) {
        if (!(ok = mbar_wait(smem_addr(&sh.dk_done), (n - 1) & 1, gave_up))) break;
        tc_fence_after();
      }
      tmem_store16(lane0 + ds_at(quarter), packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.ds_ready));
      put(n + 1, next);
    }
    if (ok && mbar_wait(smem_addr(&sh.done), 0, gave_up)) {
      tc_fence_after();
      const int key = unit.index * kTile + row;
      const bool is_dk = quarter & 1;
      const AttnTensor& to = is_dk ? a.dk : a.dv;
      T* out = static_cast<T*>(const_cast<void*>(to.ptr)) + (int64_t)(unit.begin + key) * to.token_stride +
               kv_head * to.head_stride;
      for (int x = quarter >> 1; x < dim16; x += 2)
        write16<T>(lane0 + (is_dk ? dk_at : dv_at), out, x * 16, a.dim, is_dk ? a.scale : 1.f, key < unit.length);
    }
  }
  leave(&sh.gave_up, warp, tmem);
}

// ---- dq ---------------------------------------------------------------------------

constexpr int kKStages = 3, kVStages = 2;

struct SharedQ {
  alignas(8) uint64_t q_full, k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], s_full, s_read,
      dp_full[2], ds_ready, done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
};

template <class T, int PANELS>
__device__ __forceinline__ void dq_block(const Maps& maps, const AttnArgs& a, int block, uint8_t* tiles, SharedQ& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = block % a.heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, block / a.heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == kLoader && lane == 0) {
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
    mbar_init(smem_addr(&sh.s_read), kWorkers / 32);
    mbar_init(smem_addr(&sh.ds_ready), kWorkers / 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (sh.unit.count == 0) return;
  const SeqUnit unit = sh.unit;

  constexpr uint32_t kTileBytes = PANELS * kPanelBytes;
  const uint32_t q_tile = smem_addr(tiles), do_tile = q_tile + kTileBytes, k_tile = do_tile + kTileBytes,
                 v_tile = k_tile + kKStages * kTileBytes;
  volatile int* gave_up = &sh.gave_up;
  if (warp == kIssuer) tmem_alloc(smem_addr(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Tensor memory: scores 0, dout v^T 128 and 256 (by turns), dq 384.  The
  // next tile's scores and dout v^T are under way while this one's ds is made.
  const uint32_t tmem = sh.tmem;

  const int steps = unit.index + 1, query = unit.index * kTile;
  const int dim16 = (a.dim + 15) / 16;

  if (warp == kLoader) {
    const int kv_head = head / (a.heads / a.kv_heads);
    if (lane == 0) {
      const uint32_t bar = smem_addr(&sh.q_full);
      mbar_expect(bar, 2 * kTileBytes);
      for (int p = 0; p < PANELS; ++p) {
        tma_load(q_tile + p * kPanelBytes, &maps.q, p * 64, head, unit.begin + query, bar);
        tma_load(do_tile + p * kPanelBytes, &maps.dout, p * 64, head, unit.begin + query, bar);
      }
    }
    uint32_t own_parity = 0;
    for (int n = 0; n < steps; ++n) {
      const int ks = n % kKStages, vs = n % kVStages, key = n * kTile;
      if (n >= kKStages && !mbar_wait(smem_addr(&sh.k_empty[ks]), (n / kKStages - 1) & 1, gave_up)) break;
      // dq sums over the rows of K: those of another sequence are cleared
      if (!load_tile(&maps.k, k_tile + ks * kTileBytes, PANELS, kv_head, unit.begin + key, unit.length - key,
                     smem_addr(&sh.k_full[ks]), smem_addr(&sh.own), &own_parity, gave_up))
        break;
      if (n >= kVStages && !mbar_wait(smem_addr(&sh.v_empty[vs]), (n / kVStages - 1) & 1, gave_up)) break;
      if (!load_tile(&maps.v, v_tile + vs * kTileBytes, PANELS, kv_head, unit.begin + key, kTile,
                     smem_addr(&sh.v_full[vs]), smem_addr(&sh.own), &own_parity, gave_up))
        break;
    }
  } else if (warp == kIssuer) {
    if (elect_one()) {
      const uint32_t wide = mma_shape<T>(kTile, false), sums = mma_shape<T>(dim16 * 16, true);
      auto scores = [&](int n) {  // Q K^T
        if (!mbar_wait(smem_addr(&sh.k_full[n % kKStages]), (n / kKStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(tmem, q_tile, k_tile + (n % kKStages) * kTileBytes, wide, dim16);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // dout V^T
        if (!mbar_wait(smem_addr(&sh.v_full[n % kVStages]), (n / kVStages) & 1, gave_up)) return false;
        product_ss<4 * PANELS>(tmem + 128 + (n & 1) * 128, do_tile, v_tile + (n % kVStages) * kTileBytes, wide, dim16);
        mma_commit(smem_addr(&sh.dp_full[n & 1]));
        mma_commit(smem_addr(&sh.v_empty[n % kVStages]));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.q_full), 0, gave_up) && scores(0) && dprob(0);
      for (int n = 0; n < steps && ok; ++n) {
        if (n + 1 < steps) {
          if (!(ok = mbar_wait(smem_addr(&sh.s_read), n & 1, gave_up))) break;
          tc_fence_after();
          if (!(ok = scores(n + 1) && dprob(n + 1))) break;
        }
        if (!(ok = mbar_wait(smem_addr(&sh.ds_ready), n & 1, gave_up))) break;
        tc_fence_after();
        for (int h = 0; h < 4; ++h)
          product_ts<2>(tmem + 384, tmem + 128 + (n & 1) * 128 + h * 32, k_tile + (n % kKStages) * kTileBytes, h, sums,
                        n > 0 || h > 0);
        mma_commit(smem_addr(&sh.k_empty[n % kKStages]));
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: query row, keys [32 quarter, 32 quarter + 32) of each tile
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const float c = a.scale * kLog2e;
    const bool valid = query + row < unit.length;
    const int64_t at = (int64_t)head * a.tokens + unit.begin + query + row;
    const float l = valid ? -a.lse[at] * kLog2e : -INFINITY, dl = valid ? -a.delta[at] : 0.f;
    const Two lse = two(l, l), delta = two(dl, dl);
    bool ok = true;
    for (int n = 0; n < steps; ++n) {
      const bool diagonal = n == steps - 1;
      if (!(ok = mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up))) break;
      tc_fence_after();
      float p[32], d[32];
      uint32_t packed[16];
      tmem_load32(lanes + quarter * 32, p);
      tmem_wait_load();
      tmem_loaded(p);
      warp_arrive(smem_addr(&sh.s_read));
      probabilities<T>(p, packed, c, [&](int) { return lse; }, diagonal, [&](int x) { return quarter * 32 + x <= row; });
      const uint32_t dp_at = lanes + 128 + (n & 1) * 128 + quarter * 32;
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full[n & 1]), (n >> 1) & 1, gave_up))) break;
      tc_fence_after();
      tmem_load32(dp_at, d);
      tmem_wait_load();
      tmem_loaded(d);
      score_gradients<T>(p, d, packed, [&](int) { return delta; }, diagonal);
      tmem_store16(dp_at, packed);
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.ds_ready));
    }
    if (ok && mbar_wait(smem_addr(&sh.done), 0, gave_up)) {
      tc_fence_after();
      T* out = static_cast<T*>(const_cast<void*>(a.dq.ptr)) + (int64_t)(unit.begin + query + row) * a.dq.token_stride +
               head * a.dq.head_stride;
      for (int x = quarter; x < dim16; x += 4) write16<T>(lanes + 384, out, x * 16, a.dim, a.scale, valid);
    }
  }
  leave(&sh.gave_up, warp, tmem);
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
__global__ void __launch_bounds__(kThreads, 1)
    attention_backward_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, int kv_blocks) {
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ Shared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for delta
  const int block = blockIdx.x;
  if (block < kv_blocks) dkv_block<T, PANELS>(maps, a, block, tiles, sh.kv);
  else dq_block<T, PANELS>(maps, a, block - kv_blocks, tiles, sh.q);
}

template <class T, int PANELS>
cudaError_t run(int dtype, const AttnArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  constexpr int tiles = std::max(2 + 2 * query_stages(PANELS), 2 + kKStages + kVStages);
  constexpr int smem = tiles * PANELS * (int)kPanelBytes;
  auto* kernel = attention_backward_kernel<T, PANELS>;
  cudaError_t e = open_kernel((const void*)kernel, smem, false, opened);
  if (e != cudaSuccess) return e;
  Maps maps;
  if (!make_tensor_map(&maps.q, dtype, a.q, a.tokens, a.heads, a.dim) ||
      !make_tensor_map(&maps.k, dtype, a.k, a.tokens, a.kv_heads, a.dim) ||
      !make_tensor_map(&maps.v, dtype, a.v, a.tokens, a.kv_heads, a.dim) ||
      !make_tensor_map(&maps.dout, dtype, a.dout, a.tokens, a.heads, a.dim))
    return cudaErrorInvalidValue;
  constexpr int kLanes = PANELS * 8, kRows = 256 / kLanes;
  attention_delta_kernel<T, kLanes><<<(unsigned)((a.tokens * a.heads + kRows - 1) / kRows), 256, 0, s>>>(a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // at most this many tiles, however the tokens are split
  const int64_t most = a.tokens / kTile + std::min<int64_t>(a.seqs, a.tokens);
  const int kv_blocks = (int)(most * a.kv_heads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kv_blocks + most * a.heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, maps, a, kv_blocks);
  count_launch();
  return e;
}

}  // namespace

cudaError_t launch_attention_backward(int dtype, const AttnArgs& a, cudaStream_t s) {
  if (dtype == BF16) return a.dim <= 64 ? run<__nv_bfloat16, 1>(dtype, a, s) : run<__nv_bfloat16, 2>(dtype, a, s);
  return a.dim <= 64 ? run<__half, 1>(dtype, a, s) : run<__half, 2>(dtype, a, s);
}

cudaError_t attention_forward_take_status(int* status);

cudaError_t attention_take_status(int* status) {
  cudaError_t e = attention_forward_take_status(status);
  int v = 0;
  if (e != cudaSuccess || (e = cudaMemcpyFromSymbol(&v, g_status, sizeof(int))) != cudaSuccess || !v) return e;
  *status = v;
  v = 0;
  return cudaMemcpyToSymbol(g_status, &v, sizeof(int));
}

}  // namespace ar
