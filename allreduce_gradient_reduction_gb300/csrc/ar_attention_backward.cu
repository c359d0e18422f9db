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
// In both, eight warps take the exponentials: two threads share a row of the
// tile, 64 columns each.  p and ds take the places of the scores and of
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
constexpr int kThreads = 320;

// delta[head][token] = dout . out: 16 threads to a row, 16 bytes each.
template <class T>
__global__ void __launch_bounds__(256) attention_delta_kernel(const AttnArgs a) {
  const int64_t rows = a.tokens * a.heads;
  const int64_t r = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  const int c = threadIdx.x % 16 * 8;
  float s = 0.f;
  const int64_t token = r / a.heads, head = r % a.heads;
  if (r < rows && c < a.dim) {
    const Pack<T, 8> x = *reinterpret_cast<const Pack<T, 8>*>(static_cast<const T*>(a.out.ptr) + token * a.out.token_stride +
                                                              head * a.out.head_stride + c);
    const Pack<T, 8> y = *reinterpret_cast<const Pack<T, 8>*>(static_cast<const T*>(a.dout.ptr) + token * a.dout.token_stride +
                                                              head * a.dout.head_stride + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(Conv<T>::up(x.v[i]), Conv<T>::up(y.v[i]), s);
  }
#pragma unroll
  for (int m = 8; m; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
  if (r < rows && c == 0) a.delta[head * a.tokens + token] = s;
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
  if (warp == 8) tmem_free(tmem, 512);
}

// ---- dk and dv ---------------------------------------------------------------------

constexpr int kStages = 2;  // tiles of queries (q and dout) in flight

struct SharedKV {
  alignas(8) uint64_t kv_full, q_full[kStages], do_full[kStages], empty[kStages], s_full, dp_full, p_ready, ds_ready,
      done, own;
  alignas(16) float lse[2][2][64], delta[2][2][64];  // [buffer][half]
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
};

template <class T, int PANELS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_dkv_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap do_map,
                         const AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ SharedKV sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv_head = blockIdx.x % a.kv_heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, blockIdx.x / a.kv_heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  }
  __syncthreads();
  if (sh.unit.count == 0) return;
  const SeqUnit unit = sh.unit;

  constexpr uint32_t kTileBytes = PANELS * kPanelBytes;
  const uint32_t k_tile = smem_addr(tiles), v_tile = k_tile + kTileBytes, q_tile = v_tile + kTileBytes,
                 do_tile = q_tile + kStages * kTileBytes;
  volatile int* gave_up = &sh.gave_up;
  if (warp == 8) tmem_alloc(smem_addr(&sh.tmem), 512);
  if (threadIdx.x == 0) {
    uint64_t* const one[] = {&sh.kv_full, &sh.q_full[0], &sh.q_full[1], &sh.do_full[0], &sh.do_full[1], &sh.empty[0],
                             &sh.empty[1], &sh.s_full, &sh.dp_full, &sh.done, &sh.own};
    for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
    mbar_init(smem_addr(&sh.p_ready), 256);
    mbar_init(smem_addr(&sh.ds_ready), 256);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;  // columns: scores 0, dout v^T 128, dv 256, dk 384

  // step n: head n / per of the group, tile of queries unit.index + n % per
  const int group = a.heads / a.kv_heads, per = unit.count - unit.index, steps = group * per;
  const int dim16 = (a.dim + 15) / 16;

  if (warp == 9) {
    if (lane == 0) {
      const uint32_t bar = smem_addr(&sh.kv_full);
      mbar_expect(bar, 2 * kTileBytes);
      for (int p = 0; p < PANELS; ++p) {
        tma_load(k_tile + p * kPanelBytes, &k_map, p * 64, kv_head, unit.begin + unit.index * kTile, bar);
        tma_load(v_tile + p * kPanelBytes, &v_map, p * 64, kv_head, unit.begin + unit.index * kTile, bar);
      }
    }
    uint32_t own_parity = 0;
    for (int n = 0; n < steps; ++n) {
      const int stage = n % kStages;
      if (n >= kStages && !mbar_wait(smem_addr(&sh.empty[stage]), (n / kStages - 1) & 1, gave_up)) break;
      const int head = kv_head * group + n / per, query = (unit.index + n % per) * kTile;
      if (!load_tile(&q_map, q_tile + stage * kTileBytes, PANELS, head, unit.begin + query, unit.length - query,
                     smem_addr(&sh.q_full[stage]), smem_addr(&sh.own), &own_parity, gave_up) ||
          !load_tile(&do_map, do_tile + stage * kTileBytes, PANELS, head, unit.begin + query, unit.length - query,
                     smem_addr(&sh.do_full[stage]), smem_addr(&sh.own), &own_parity, gave_up))
        break;
    }
  } else if (warp == 8) {
    if (lane == 0) {
      const uint32_t wide = mma_shape<T>(kTile, false), sums = mma_shape<T>(dim16 * 16, true);
      auto at = [&](uint32_t tile, int n) { return tile + (n % kStages) * kTileBytes; };
      auto scores = [&](int n) {  // K Q^T
        if (!mbar_wait(smem_addr(&sh.q_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        for (int s = 0; s < dim16; ++s) mma_ss(tmem, k_major(k_tile, s), k_major(at(q_tile, n), s), wide, s > 0);
        mma_commit(smem_addr(&sh.s_full));
        return true;
      };
      auto dprob = [&](int n) {  // V dout^T
        if (!mbar_wait(smem_addr(&sh.do_full[n % kStages]), (n / kStages) & 1, gave_up)) return false;
        for (int s = 0; s < dim16; ++s) mma_ss(tmem + 128, k_major(v_tile, s), k_major(at(do_tile, n), s), wide, s > 0);
        mma_commit(smem_addr(&sh.dp_full));
        return true;
      };
      // a half's 32 columns of pairs lie at the front of the 64 that it read
      auto sum = [&](uint32_t to, uint32_t from, uint32_t right, bool add) {
        for (int s = 0; s < kTile / 16; ++s)
          mma_ts(to, from + (s >> 2) * 64 + (s & 3) * 8, mn_major(right, s), sums, add || s > 0);
      };
      bool ok = mbar_wait(smem_addr(&sh.kv_full), 0, gave_up) && scores(0) && dprob(0);
      for (int n = 0; n < steps && ok; ++n) {
        if (!(ok = mbar_wait(smem_addr(&sh.p_ready), n & 1, gave_up))) break;
        tc_fence_after();
        sum(tmem + 256, tmem, at(do_tile, n), n > 0);
        if (n + 1 < steps && !(ok = scores(n + 1))) break;
        if (!(ok = mbar_wait(smem_addr(&sh.ds_ready), n & 1, gave_up))) break;
        tc_fence_after();
        sum(tmem + 384, tmem + 128, at(q_tile, n), n > 0);
        mma_commit(smem_addr(&sh.empty[n % kStages]));
        if (n + 1 < steps && !(ok = dprob(n + 1))) break;
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: key row, queries [64 half, 64 half + 64) of each tile
    const int half = warp >> 2, row = (warp & 3) * 32 + lane, t = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const float c = a.scale * kLog2e;
    // threads 0..63 of a half fetch its queries' lse, the others their delta
    auto fetch = [&](int n) {
      const int query = (unit.index + n % per) * kTile + half * 64 + (t & 63);
      if (query >= unit.length) return t < 64 ? INFINITY : 0.f;  // p = 0 after the sequence's end
      const int64_t at = (int64_t)(kv_head * group + n / per) * a.tokens + unit.begin + query;
      return t < 64 ? a.lse[at] * kLog2e : a.delta[at];
    };
    auto put = [&](int n, float v) {
      (t < 64 ? sh.lse : sh.delta)[n & 1][half][t & 63] = v;
      named_barrier(1 + half, 128);
    };
    put(0, fetch(0));
    bool ok = true;
    for (int n = 0; n < steps; ++n) {
      const float next = n + 1 < steps ? fetch(n + 1) : 0.f;
      const bool diagonal = n % per == 0;
      if (!(ok = mbar_wait(smem_addr(&sh.s_full), n & 1, gave_up))) break;
      tc_fence_after();
      float p[2][32];
      tmem_load32(lanes + half * 64, p[0]);
      tmem_load32(lanes + half * 64 + 32, p[1]);
      tmem_wait_load();
      tmem_loaded(p[0]);
      tmem_loaded(p[1]);
      uint32_t packed[32];
#pragma unroll
      for (int x = 0; x < 64; x += 4) {
        const float4 l = *reinterpret_cast<const float4*>(&sh.lse[n & 1][half][x]);
        const float ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float& e = p[x >> 5][(x & 31) + y];
          e = exp2_approx(fmaf(e, c, -ls[y]));
          if (diagonal && half * 64 + x + y < row) e = 0.f;
        }
        packed[x / 2] = pack2<T>(p[x >> 5][x & 31], p[x >> 5][(x & 31) + 1]);
        packed[x / 2 + 1] = pack2<T>(p[x >> 5][(x & 31) + 2], p[x >> 5][(x & 31) + 3]);
      }
      tmem_store32(lanes + half * 64, packed);
      tmem_wait_store();
      tc_fence_before();
      mbar_arrive(smem_addr(&sh.p_ready));
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full), n & 1, gave_up))) break;
      tc_fence_after();
      float d[2][32];
      tmem_load32(lanes + 128 + half * 64, d[0]);
      tmem_load32(lanes + 128 + half * 64 + 32, d[1]);
      tmem_wait_load();
      tmem_loaded(d[0]);
      tmem_loaded(d[1]);
#pragma unroll
      for (int x = 0; x < 64; x += 4) {
        const float4 l = *reinterpret_cast<const float4*>(&sh.delta[n & 1][half][x]);
        const float ls[4] = {l.x, l.y, l.z, l.w};
        float v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float e = p[x >> 5][(x & 31) + y];
          v[y] = e == 0.f ? 0.f : e * (d[x >> 5][(x & 31) + y] - ls[y]);
        }
        packed[x / 2] = pack2<T>(v[0], v[1]);
        packed[x / 2 + 1] = pack2<T>(v[2], v[3]);
      }
      tmem_store32(lanes + 128 + half * 64, packed);
      tmem_wait_store();
      tc_fence_before();
      mbar_arrive(smem_addr(&sh.ds_ready));
      put(n + 1, next);
    }
    if (ok && mbar_wait(smem_addr(&sh.done), 0, gave_up)) {
      tc_fence_after();
      const int key = unit.index * kTile + row;
      const AttnTensor& to = half ? a.dk : a.dv;
      T* out = static_cast<T*>(const_cast<void*>(to.ptr)) + (int64_t)(unit.begin + key) * to.token_stride +
               kv_head * to.head_stride;
      for (int d = 0; d < dim16; ++d)
        write16<T>(lanes + (half ? 384 : 256), out, d * 16, a.dim, half ? a.scale : 1.f, key < unit.length);
    }
  }
  leave(&sh.gave_up, warp, tmem);
}

// ---- dq ---------------------------------------------------------------------------

constexpr int kKStages = 3, kVStages = 2;

struct SharedQ {
  alignas(8) uint64_t q_full, k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], s_full[2],
      dp_full, ds_ready, done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
};

template <class T, int PANELS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_dq_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap do_map,
                        const AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ SharedQ sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % a.heads;
  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, blockIdx.x / a.heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  }
  __syncthreads();
  if (sh.unit.count == 0) return;
  const SeqUnit unit = sh.unit;

  constexpr uint32_t kTileBytes = PANELS * kPanelBytes;
  const uint32_t q_tile = smem_addr(tiles), do_tile = q_tile + kTileBytes, k_tile = do_tile + kTileBytes,
                 v_tile = k_tile + kKStages * kTileBytes;
  volatile int* gave_up = &sh.gave_up;
  if (warp == 8) tmem_alloc(smem_addr(&sh.tmem), 512);
  if (threadIdx.x == 0) {
    uint64_t* const one[] = {&sh.q_full, &sh.s_full[0], &sh.s_full[1], &sh.dp_full, &sh.done, &sh.own};
    for (uint64_t* b : one) mbar_init(smem_addr(b), 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(smem_addr(&sh.k_full[i]), 1);
      mbar_init(smem_addr(&sh.k_empty[i]), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(smem_addr(&sh.v_full[i]), 1);
      mbar_init(smem_addr(&sh.v_empty[i]), 1);
    }
    mbar_init(smem_addr(&sh.ds_ready), 256);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;  // columns: scores 0 and 128, dout v^T 256, dq 384

  const int tile = unit.count - 1 - unit.index;  // the longest rows of a sequence first
  const int steps = tile + 1, query = tile * kTile;
  const int dim16 = (a.dim + 15) / 16;

  if (warp == 9) {
    const int kv_head = head / (a.heads / a.kv_heads);
    if (lane == 0) {
      const uint32_t bar = smem_addr(&sh.q_full);
      mbar_expect(bar, 2 * kTileBytes);
      for (int p = 0; p < PANELS; ++p) {
        tma_load(q_tile + p * kPanelBytes, &q_map, p * 64, head, unit.begin + query, bar);
        tma_load(do_tile + p * kPanelBytes, &do_map, p * 64, head, unit.begin + query, bar);
      }
    }
    uint32_t own_parity = 0;
    for (int n = 0; n < steps; ++n) {
      const int ks = n % kKStages, vs = n % kVStages, key = n * kTile;
      if (n >= kKStages && !mbar_wait(smem_addr(&sh.k_empty[ks]), (n / kKStages - 1) & 1, gave_up)) break;
      // dq sums over the rows of K: those of another sequence are cleared
      if (!load_tile(&k_map, k_tile + ks * kTileBytes, PANELS, kv_head, unit.begin + key, unit.length - key,
                     smem_addr(&sh.k_full[ks]), smem_addr(&sh.own), &own_parity, gave_up))
        break;
      if (n >= kVStages && !mbar_wait(smem_addr(&sh.v_empty[vs]), (n / kVStages - 1) & 1, gave_up)) break;
      if (!load_tile(&v_map, v_tile + vs * kTileBytes, PANELS, kv_head, unit.begin + key, kTile,
                     smem_addr(&sh.v_full[vs]), smem_addr(&sh.own), &own_parity, gave_up))
        break;
    }
  } else if (warp == 8) {
    if (lane == 0) {
      const uint32_t wide = mma_shape<T>(kTile, false), sums = mma_shape<T>(dim16 * 16, true);
      auto scores = [&](int n) {  // Q K^T
        if (!mbar_wait(smem_addr(&sh.k_full[n % kKStages]), (n / kKStages) & 1, gave_up)) return false;
        for (int s = 0; s < dim16; ++s)
          mma_ss(tmem + (n & 1) * 128, k_major(q_tile, s), k_major(k_tile + (n % kKStages) * kTileBytes, s), wide, s > 0);
        mma_commit(smem_addr(&sh.s_full[n & 1]));
        return true;
      };
      auto dprob = [&](int n) {  // dout V^T
        if (!mbar_wait(smem_addr(&sh.v_full[n % kVStages]), (n / kVStages) & 1, gave_up)) return false;
        for (int s = 0; s < dim16; ++s)
          mma_ss(tmem + 256, k_major(do_tile, s), k_major(v_tile + (n % kVStages) * kTileBytes, s), wide, s > 0);
        mma_commit(smem_addr(&sh.dp_full));
        mma_commit(smem_addr(&sh.v_empty[n % kVStages]));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&sh.q_full), 0, gave_up) && scores(0) && dprob(0) && (steps < 2 || scores(1));
      for (int n = 0; n < steps && ok; ++n) {
        if (!(ok = mbar_wait(smem_addr(&sh.ds_ready), n & 1, gave_up))) break;
        tc_fence_after();
        const uint32_t k = k_tile + (n % kKStages) * kTileBytes;
        for (int s = 0; s < kTile / 16; ++s)
          mma_ts(tmem + 384, tmem + 256 + (s >> 2) * 64 + (s & 3) * 8, mn_major(k, s), sums, n > 0 || s > 0);
        mma_commit(smem_addr(&sh.k_empty[n % kKStages]));
        if (n + 1 < steps && !(ok = dprob(n + 1))) break;
        if (n + 2 < steps && !(ok = scores(n + 2))) break;
      }
      if (ok) mma_commit(smem_addr(&sh.done));
    }
    __syncwarp();
  } else {
    // thread: query row, keys [64 half, 64 half + 64) of each tile
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const float c = a.scale * kLog2e;
    const bool valid = query + row < unit.length;
    const int64_t at = (int64_t)head * a.tokens + unit.begin + query + row;
    const float lse = valid ? a.lse[at] * kLog2e : INFINITY, delta = valid ? a.delta[at] : 0.f;
    bool ok = true;
    for (int n = 0; n < steps; ++n) {
      if (!(ok = mbar_wait(smem_addr(&sh.s_full[n & 1]), (n >> 1) & 1, gave_up))) break;
      tc_fence_after();
      float p[2][32], d[2][32];
      tmem_load32(lanes + (n & 1) * 128 + half * 64, p[0]);
      tmem_load32(lanes + (n & 1) * 128 + half * 64 + 32, p[1]);
      tmem_wait_load();
      tmem_loaded(p[0]);
      tmem_loaded(p[1]);
#pragma unroll
      for (int x = 0; x < 64; ++x) {
        float& e = p[x >> 5][x & 31];
        e = exp2_approx(fmaf(e, c, -lse));
        if (n == steps - 1 && half * 64 + x > row) e = 0.f;
      }
      if (!(ok = mbar_wait(smem_addr(&sh.dp_full), n & 1, gave_up))) break;
      tc_fence_after();
      tmem_load32(lanes + 256 + half * 64, d[0]);
      tmem_load32(lanes + 256 + half * 64 + 32, d[1]);
      tmem_wait_load();
      tmem_loaded(d[0]);
      tmem_loaded(d[1]);
      uint32_t packed[32];
#pragma unroll
      for (int x = 0; x < 64; x += 2) {
        const float e = p[x >> 5][x & 31], f = p[x >> 5][(x & 31) + 1];
        packed[x / 2] = pack2<T>(e == 0.f ? 0.f : e * (d[x >> 5][x & 31] - delta),
                                 f == 0.f ? 0.f : f * (d[x >> 5][(x & 31) + 1] - delta));
      }
      tmem_store32(lanes + 256 + half * 64, packed);
      tmem_wait_store();
      tc_fence_before();
      mbar_arrive(smem_addr(&sh.ds_ready));
    }
    if (ok && mbar_wait(smem_addr(&sh.done), 0, gave_up)) {
      tc_fence_after();
      T* out = static_cast<T*>(const_cast<void*>(a.dq.ptr)) + (int64_t)(unit.begin + query + row) * a.dq.token_stride +
               head * a.dq.head_stride;
      for (int d = half; d < dim16; d += 2) write16<T>(lanes + 384, out, d * 16, a.dim, a.scale, valid);
    }
  }
  leave(&sh.gave_up, warp, tmem);
}

template <class T, int PANELS>
cudaError_t run(int dtype, const AttnArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> opened_kv[256], opened_q[256];
  constexpr int smem_kv = (2 + 2 * kStages) * PANELS * (int)kPanelBytes;
  constexpr int smem_q = (2 + kKStages + kVStages) * PANELS * (int)kPanelBytes;
  cudaError_t e = open_kernel((const void*)attention_dkv_kernel<T, PANELS>, smem_kv, false, opened_kv);
  if (e != cudaSuccess) return e;
  if ((e = open_kernel((const void*)attention_dq_kernel<T, PANELS>, smem_q, false, opened_q)) != cudaSuccess) return e;
  CUtensorMap q, k, v, d;
  if (!make_tensor_map(&q, dtype, a.q, a.tokens, a.heads, a.dim) ||
      !make_tensor_map(&k, dtype, a.k, a.tokens, a.kv_heads, a.dim) ||
      !make_tensor_map(&v, dtype, a.v, a.tokens, a.kv_heads, a.dim) ||
      !make_tensor_map(&d, dtype, a.dout, a.tokens, a.heads, a.dim))
    return cudaErrorInvalidValue;
  attention_delta_kernel<T><<<(unsigned)((a.tokens * a.heads + 15) / 16), 256, 0, s>>>(a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // at most this many tiles, however the tokens are split
  const int64_t most = a.tokens / kTile + std::min<int64_t>(a.seqs, a.tokens);
  attention_dkv_kernel<T, PANELS><<<(unsigned)(most * a.kv_heads), kThreads, smem_kv, s>>>(q, k, v, d, a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  attention_dq_kernel<T, PANELS><<<(unsigned)(most * a.heads), kThreads, smem_q, s>>>(q, k, v, d, a);
  count_launch();
  return cudaGetLastError();
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
