// Causal attention over packed sequences, forward.
//
//   a_ij = scale q_i . k_j (j <= i, same sequence), out_i = sum_j p_ij v_j with
//   p = softmax(a_i), lse_i = log sum_j exp(a_ij).
//
// Bound by the tensor cores at head sizes near 128 (4 dim operations a pair of
// tokens), by the exponentials and what goes with them at 64 and below.  One
// pass over the keys with a running maximum and sum, the scores and the output
// in tensor memory.  Four warps to a tile of queries take the exponentials,
// one issues the products, one loads.  The probabilities go back to tensor
// memory as 16-bit pairs and are the second product's left operand there:
// rounded to the type of v, as the tensor cores need, an error of half a unit
// in the last place of each; the sum that divides them is of the unrounded.
//
// Measured: 8192 tokens of one sequence, 32 heads of 128 over 8 K/V heads, 350
// us (1.57 PFLOP/s, 82% of the rate of a plain matrix product on the same
// device); 32 heads of 64, 284 us, of which the products alone are half (the
// exponentials of a tile take as long as its products, and one block's do not
// cover the other's products whole).
//
// The running maximum that scales the output is moved only when a row's true
// maximum has grown by more than 8 in the exponent of two: until then the
// probabilities stay below 2^8, exact enough in either 16-bit type, and the
// output need not be touched.  f16 holds them times 2^7, below 2^15 then, so that
// one of 2^-32 of the row's largest is not lost yet: thousands of keys may have
// no more each and a value that counts.  The power is part of the exponential's
// argument and of the sum that divides.
#include "ar_tcgen05.cuh"

#include <algorithm>

namespace ar {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;  // powers of two that a row's maximum may grow by before the output is rescaled
constexpr int kStages = 4;     // tiles of K or V in flight
template <class T>
constexpr float kShift = __is_same(T, __half) ? 7.f : 0.f;  // powers of two that probabilities are held times

// What differs with the head size.  A tensor core product of 128 x 128 scores
// takes 4 cycles for each element of the head, the exponentials of a tile at
// least 512 cycles whatever the head.
//
// Up to 64 elements (one panel) the exponentials bound it, and what counts is
// that they never wait: a block takes one tile of 128 queries, and two blocks
// share a multiprocessor (8192 tokens, 32 heads of 64: 286 us, and 308 us with
// the layout below).  Tensor memory has room for the probabilities beside the
// scores, so the next scores are computed as soon as the current ones have
// been read.
//
// Beyond, the products bound it: a block takes two tiles, so that K and V are
// fetched once for 256 queries and one tile's products run while the other's
// exponentials are taken.  The outputs fill tensor memory and the
// probabilities take the scores' place.
//
// A thread has one query's whole row, so its maximum and sum need no exchange.
template <int PANELS>
struct Form {
  static constexpr int kTiles = PANELS == 1 ? 1 : 2;
  static constexpr bool kApart = PANELS == 1;
  static constexpr int kThreads = PANELS == 1 ? 192 : 384;
  static constexpr int kIssuer = 4 * kTiles, kLoader = kIssuer + 1;  // warps; those before them take exponentials
  static constexpr int kBlocks = PANELS == 1 ? 2 : 1;  // on a multiprocessor
  static constexpr int kColumns = PANELS == 1 ? 256 : 512;
  static constexpr int kQueries = kTiles * kTile;
};

struct Shared {
  alignas(8) uint64_t q_full[2], kv_full[kStages], kv_empty[kStages], s_full[2], s_read[2], p_full[2][2], o_done[2], own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
};

template <class T, int PANELS>
__global__ void __launch_bounds__(Form<PANELS>::kThreads, Form<PANELS>::kBlocks)
    attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const AttnArgs a) {
  using F = Form<PANELS>;
  constexpr int kTiles = F::kTiles;
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % a.heads;

  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, F::kQueries, blockIdx.x / a.heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == F::kIssuer) {
    tmem_alloc(smem_addr(&sh.tmem), F::kColumns);
  } else if (warp == F::kLoader && lane == 0) {
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(smem_addr(&sh.q_full[i]), 1);
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.s_read[i]), 4);
      mbar_init(smem_addr(&sh.p_full[i][0]), 4);
      mbar_init(smem_addr(&sh.p_full[i][1]), 4);
      mbar_init(smem_addr(&sh.o_done[i]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&sh.kv_full[i]), 1);
      mbar_init(smem_addr(&sh.kv_empty[i]), 1);
    }
    mbar_init(smem_addr(&sh.own), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.unit.count == 0) {
    if (warp == F::kIssuer) tmem_free(sh.tmem, F::kColumns);
    return;
  }
  const SeqUnit unit = sh.unit;

  constexpr uint32_t kTileBytes = PANELS * kPanelBytes;
  const uint32_t q_tile = smem_addr(tiles), kv_tile = q_tile + kTiles * kTileBytes;
  volatile int* gave_up = &sh.gave_up;

  const int first = unit.index * F::kQueries;  // first query, within the sequence
  int blocks[kTiles];                          // tiles of keys that each tile of queries sees
  for (int i = 0; i < kTiles; ++i) blocks[i] = first + i * kTile < unit.length ? first / kTile + 1 + i : 0;
  const int most = max(blocks[0], blocks[kTiles - 1]);
  const int dim16 = (a.dim + 15) / 16;

  // loads: Q tiles first, then K 0, V 0, K 1, V 1, ...
  const int kv_head = head / (a.heads / a.kv_heads);
  uint32_t own_parity = 0;
  auto load = [&](int n) {
    const int stage = n % kStages, key = (n >> 1) * kTile;
    return load_tile<PANELS, kTile>(n & 1 ? &v_map : &k_map, kv_tile + stage * kTileBytes, kv_head, unit.begin + key,
                                    n & 1 ? unit.length - key : kTile, smem_addr(&sh.kv_full[stage]),
                                    smem_addr(&sh.own), &own_parity, gave_up);
  };
  // tensor memory: each tile's scores, then probabilities where they are apart, then outputs
  const uint32_t tmem = sh.tmem;
  auto p_at = [&](int i, int half) { return tmem + (F::kApart ? 128 + half * 32 : i * 128 + half * 32); };
  auto out_at = [&](int i) { return tmem + (F::kApart ? 192 : 256 + i * 128); };

  if (warp >= F::kIssuer) {
    if constexpr (F::kThreads == 384) give_registers();
    if (warp == F::kLoader) {
      if (lane == 0) {
        for (int i = 0; i < kTiles; ++i) {
          if (!blocks[i]) continue;
          const uint32_t bar = smem_addr(&sh.q_full[i]);
          mbar_expect(bar, kTileBytes);
          for (int p = 0; p < PANELS; ++p)
            tma_load(q_tile + i * kTileBytes + p * kPanelBytes, &q_map, p * 64, head, unit.begin + first + i * kTile, bar);
        }
      }
      for (int n = 0; n < 2 * most; ++n) {
        if (n >= kStages && !mbar_wait(smem_addr(&sh.kv_empty[n % kStages]), (n / kStages - 1) & 1, gave_up)) break;
        if (!load(n)) break;
      }
    } else if (warp == F::kIssuer) {
      // ---- products, all issued by one thread
      if (elect_one()) {
        const uint32_t qk = mma_shape<T>(kTile, false), pv = mma_shape<T>(dim16 * 16, true);
        auto full = [&](int n) {
          return mbar_wait(smem_addr(&sh.kv_full[n % kStages]), (n / kStages) & 1, gave_up);
        };
        auto scores = [&](int i, int j) {
          product_ss<4 * PANELS>(tmem + i * 128, q_tile + i * kTileBytes, kv_tile + (2 * j % kStages) * kTileBytes, qk, dim16);
          mma_commit(smem_addr(&sh.s_full[i]));
        };
        auto output = [&](int i, int j) {
          const uint32_t v = kv_tile + ((2 * j + 1) % kStages) * kTileBytes;
          for (int h = 0; h < 2; ++h) {
            if (!mbar_wait(smem_addr(&sh.p_full[i][h]), j & 1, gave_up)) return false;
            tc_fence_after();
            product_ts<4>(out_at(i), p_at(i, h), v, h, pv, j > 0 || h > 0);
          }
          mma_commit(smem_addr(&sh.o_done[i]));
          return true;
        };
        bool ok = full(0);
        for (int i = 0; i < kTiles && ok; ++i)
          if (blocks[i] && (ok = mbar_wait(smem_addr(&sh.q_full[i]), 0, gave_up))) scores(i, 0);
        if (ok) mma_commit(smem_addr(&sh.kv_empty[0]));
        for (int j = 0; j < most && ok; ++j) {
          const int vn = 2 * j + 1, kn = vn + 1;
          const bool more = j + 1 < most;
          if constexpr (F::kApart) {
            if (more) {
              if (!(ok = full(kn) && mbar_wait(smem_addr(&sh.s_read[0]), j & 1, gave_up))) break;
              tc_fence_after();
              scores(0, j + 1);
              mma_commit(smem_addr(&sh.kv_empty[kn % kStages]));
            }
            if (!(ok = full(vn) && output(0, j))) break;
          } else {
            ok = full(vn) && (!more || full(kn));
            for (int i = 0; i < kTiles && ok; ++i)
              if (j < blocks[i] && (ok = output(i, j)) && j + 1 < blocks[i]) scores(i, j + 1);
            if (!ok) break;
            if (more) mma_commit(smem_addr(&sh.kv_empty[kn % kStages]));
          }
          mma_commit(smem_addr(&sh.kv_empty[vn % kStages]));
        }
      }
      __syncwarp();
    }
  } else {
    if constexpr (F::kThreads == 384) take_registers();
    // ---- softmax: a thread has one query of tile i
    const int i = warp >> 2, n = blocks[i];
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = lanes + tmem + i * 128, o_at = lanes + out_at(i);
    const int row = (warp & 3) * 32 + lane;
    const float c = a.scale * kLog2e;
    const Two c2 = two(c, c);
    float m = -INFINITY, sum = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!(ok = mbar_wait(smem_addr(&sh.s_full[i]), j & 1, gave_up))) break;
      tc_fence_after();
      float s[4][32], top[4];
      tmem_load32(s_at, s[0]);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        tmem_wait_load();
        tmem_loaded(s[b]);
        if (b < 3) tmem_load32(s_at + (b + 1) * 32, s[b + 1]);  // on its way while these are looked at
        if (j == n - 1) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (b * 32 + x > row) s[b][x] = -INFINITY;
        }
        float even = fmaxf(s[b][0], s[b][1]), odd = fmaxf(s[b][2], s[b][3]);
#pragma unroll
        for (int x = 4; x < 32; x += 4) {
          even = max3(even, s[b][x], s[b][x + 1]);
          odd = max3(odd, s[b][x + 2], s[b][x + 3]);
        }
        top[b] = fmaxf(even, odd);
      }
      if constexpr (F::kApart) warp_arrive(smem_addr(&sh.s_read[i]));
      const float most_s = fmaxf(max3(top[0], top[1], top[2]), top[3]);
      if (j == 0) {
        m = most_s;
      } else if (__any_sync(0xFFFFFFFFu, (most_s - m) * c > kSlack)) {
        const float moved = fmaxf(m, most_s);
        const float by = m == moved ? 1.f : exp2_approx((m - moved) * c);
        m = moved;
        sum *= by;
        if (!(ok = mbar_wait(smem_addr(&sh.o_done[i]), (j - 1) & 1, gave_up))) break;
        tc_fence_after();
        for (int d = 0; d < dim16; ++d) {
          float o[16];
          tmem_load16(o_at + d * 16, o);
          tmem_wait_load();
          tmem_loaded(o);
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] *= by;
          tmem_store16(o_at + d * 16, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : m * c;
      const Two base2 = two(kShift<T> - base, kShift<T> - base);
      if (F::kApart && j > 0) {
        // the last product has read the probabilities that these replace
        if (!(ok = mbar_wait(smem_addr(&sh.o_done[i]), (j - 1) & 1, gave_up))) break;
        tc_fence_after();
      }
      Two part[2] = {two(0.f, 0.f), two(0.f, 0.f)};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t p[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          float lo, hi;
          split(fma2(two(s[b][2 * x], s[b][2 * x + 1]), c2, base2), lo, hi);
          lo = exp2_approx(lo);
          hi = exp2_approx(hi);
          part[x & 1] = add2(part[x & 1], two(lo, hi));
          p[x] = pack2<T>(lo, hi);
        }
        tmem_store16(lanes + p_at(i, 0) + b * 16, p);
        if (b == 1) {
          tmem_wait_store();
          warp_arrive(smem_addr(&sh.p_full[i][0]));
        }
      }
      tmem_wait_store();
      warp_arrive(smem_addr(&sh.p_full[i][1]));
      float sum_lo, sum_hi;
      split(add2(part[0], part[1]), sum_lo, sum_hi);
      sum += sum_lo + sum_hi;
    }
    if (n && ok && mbar_wait(smem_addr(&sh.o_done[i]), (n - 1) & 1, gave_up)) {
      tc_fence_after();
      const int from = first + i * kTile + (warp & 3) * 32, at = from + lane;  // within the sequence
      const int64_t token = unit.begin + at;
      T* out = static_cast<T*>(const_cast<void*>(a.out.ptr)) + (int64_t)(unit.begin + from) * a.out.token_stride +
               head * a.out.head_stride;
      // through the tile's queries, which nothing reads any more
      for (int p = 0; p < PANELS; ++p)
        write_rows<T, 64>(o_at, q_tile + i * kTileBytes + (warp & 3) * 4096, out, a.out.token_stride,
                          unit.length - from, p * 64, a.dim, 1.f / sum);
      if (a.lse && at < unit.length) a.lse[(int64_t)head * a.tokens + token] = (m * c + (log2f(sum) - kShift<T>)) * kLn2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (sh.gave_up) {
    // copies and products in flight end by themselves: give them time
    for (int i = 0; i < 100; ++i) __nanosleep(100000);
    if (threadIdx.x == 0) g_status = AR_ERR_TIMEOUT;
    __syncthreads();
  }
  if (warp == F::kIssuer) tmem_free(tmem, F::kColumns);
}

template <class T, int PANELS>
cudaError_t run(int dtype, const AttnArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  using F = Form<PANELS>;
  constexpr int smem = (F::kTiles + kStages) * PANELS * (int)kPanelBytes;
  cudaError_t e = open_kernel((const void*)attention_kernel<T, PANELS>, smem, false, opened);
  if (e != cudaSuccess) return e;
  // the warpgroups' shares are sound only if the launch brings them
  static const int registers = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, (const void*)attention_kernel<T, PANELS>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (F::kThreads == 384 && registers != kLaunchRegisters) return cudaErrorInvalidConfiguration;
  CUtensorMap q, k, v;
  if (!make_tensor_map(&q, dtype, a.q, a.tokens, a.heads, a.dim, kTile) ||
      !make_tensor_map(&k, dtype, a.k, a.tokens, a.kv_heads, a.dim, kTile) ||
      !make_tensor_map(&v, dtype, a.v, a.tokens, a.kv_heads, a.dim, kTile))
    return cudaErrorInvalidValue;
  const int64_t units = most_units(a.tokens, a.seqs, F::kQueries);
  attention_kernel<T, PANELS><<<(unsigned)(units * a.heads), F::kThreads, smem, s>>>(q, k, v, a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

bool make_tensor_map(CUtensorMap* map, int dtype, const AttnTensor& t, int64_t tokens, int heads, int dim, int rows) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)t.head_stride * 2, (cuuint64_t)t.token_stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, unit[3] = {1, 1, 1};
  return encode(map, dtype == BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                const_cast<void*>(t.ptr), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_attention(int dtype, const AttnArgs& a, cudaStream_t s) {
  if (dtype == BF16) return a.dim <= 64 ? run<__nv_bfloat16, 1>(dtype, a, s) : run<__nv_bfloat16, 2>(dtype, a, s);
  return a.dim <= 64 ? run<__half, 1>(dtype, a, s) : run<__half, 2>(dtype, a, s);
}

cudaError_t attention_take_status(int* status, cudaStream_t s) { return take_status(status, s); }

}  // namespace ar
