// Differential attention over packed sequences, forward.
//
//   a_m = scale q_m k_m^T (causal, m = 0, 1), p_m = softmax(a_m),
//   out = (p_0 - lambda p_1) v, second = p_1 v, lse_m = log sum exp(a_m).
//
// Bound by the tensor cores (4 dim + 4 value_dim operations a pair of tokens and
// head) at dim 64.  A block has 128 queries of one head, and both maps of them:
// what one map's products take on the tensor cores is what the other's
// exponentials are taken in, and v, the keys' other half, is fetched once for
// both.  The maps' queries and keys are panels of one tile in shared memory,
// each a map's.
//
// One pass over the keys with a running maximum and sum for each map, scores
// and both outputs in tensor memory; the difference is taken once, of the two
// normalised sums, in binary32.  Four warps to a map take the exponentials, one
// issues the products, one loads.  The probabilities take the scores' place as
// 16-bit pairs: rounded to the type of v, half a unit in the last place of each;
// the sums that divide them are of the unrounded.
//
// Measured: 8192 tokens of one sequence, 16 heads of 2 x 64 over 4, bf16, 297
// to 301 us a call (1.38 PFLOP/s, 73% of the measured rate of a plain matrix
// product; 286 us on the device).  A
// step of 128 keys takes 2260 cycles, of which the products take 1536: a map's
// exponentials (1290) and products (800, with what announces them) follow one
// another, as its scores have no second place in tensor memory, and the other
// map's run meanwhile.  Scores of 64 keys at a time, in two places, took 324 us
// (products of 64 columns wait for shared memory), two threads to a row 358.
//
// As in the ordinary attention, the maximum that scales an output is moved only
// when the true one has grown by more than 8 in the exponent of two, and f16
// holds probabilities times 2^7.  So a half tile's exponentials need not wait for
// its own maximum (307 us).
#include "ar_tcgen05.cuh"

#include <type_traits>

namespace ar {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;  // powers of two that a row's maximum may grow by before the output is rescaled
constexpr int kStages = 4;     // tiles of both maps' keys, or of v, in flight
template <class T>
constexpr float kShift = __is_same(T, __half) ? 7.f : 0.f;  // powers of two that probabilities are held times

constexpr int kThreads = 384, kIssuer = 8, kLoader = 9;  // warps; those before them take exponentials
constexpr int kColumns = 512;                            // of tensor memory

struct Shared {
  alignas(8) uint64_t q_full, kv_full[kStages], kv_empty[kStages], s_full[2], p_full[2][2], o_done[2], all_done, own;
  uint32_t tmem;
  int gave_up;
  SeqUnit unit;
  float by[kTile];  // what the second map's sums are multiplied by
};

// VPANELS: panels of 64 columns of v
template <class T, int VPANELS>
__global__ void __launch_bounds__(kThreads, 1)
    diff_attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map, const DiffArgs a) {
  extern __shared__ __align__(1024) uint8_t tiles[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % a.heads;

  if (warp == 0) {
    const SeqUnit u = find_unit(a.cu_seqlens, a.seqs, (int)a.tokens, kTile, blockIdx.x / a.heads);
    if (lane == 0) {
      sh.unit = u;
      sh.gave_up = 0;
    }
  } else if (warp == kIssuer) {
    tmem_alloc(smem_addr(&sh.tmem), kColumns);
  } else if (warp == kLoader && lane == 0) {
    mbar_init(smem_addr(&sh.q_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_full[i][0]), 4);
      mbar_init(smem_addr(&sh.p_full[i][1]), 4);
      mbar_init(smem_addr(&sh.o_done[i]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&sh.kv_full[i]), 1);
      mbar_init(smem_addr(&sh.kv_empty[i]), 1);
    }
    mbar_init(smem_addr(&sh.all_done), 1);
    mbar_init(smem_addr(&sh.own), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.unit.count == 0) {
    if (warp == kIssuer) tmem_free(sh.tmem, kColumns);
    return;
  }
  const SeqUnit unit = sh.unit;

  constexpr uint32_t kTileBytes = 2 * kPanelBytes;
  const uint32_t q_tile = smem_addr(tiles), kv_tile = q_tile + kTileBytes;
  volatile int* gave_up = &sh.gave_up;

  const int first = unit.index * kTile;  // first query, within the sequence
  const int n = unit.index + 1;          // tiles of keys that the queries see
  const int dim16 = (a.dim + 15) / 16, value16 = (a.value_dim + 15) / 16;
  const int kv_head = head / (a.heads / a.kv_heads);
  // tensor memory: each map's scores, then each map's output
  const uint32_t tmem = sh.tmem;
  auto out_at = [&](int i) { return tmem + 256 + i * 128; };

  if (warp >= kIssuer) {
    give_registers();
    if (warp == kLoader) {
      // loads: both maps' queries, then K 0, V 0, K 1, V 1, ...
      uint32_t own_parity = 0;
      auto load_maps = [&](const CUtensorMap* map, uint32_t dst, int head, int token, uint32_t bar) {
        if (lane) return;
        mbar_expect(bar, kTileBytes);
        for (int m = 0; m < 2; ++m) tma_load(dst + m * kPanelBytes, map, 0, 2 * head + m, token, bar);
      };
      load_maps(&q_map, q_tile, head, unit.begin + first, smem_addr(&sh.q_full));
      for (int i = 0; i < 2 * n; ++i) {
        const int stage = i % kStages, key = (i >> 1) * kTile;
        if (i >= kStages && !mbar_wait(smem_addr(&sh.kv_empty[stage]), (i / kStages - 1) & 1, gave_up)) break;
        const uint32_t dst = kv_tile + stage * kTileBytes, full = smem_addr(&sh.kv_full[stage]);
        if (!(i & 1)) load_maps(&k_map, dst, kv_head, unit.begin + key, full);
        else if (!load_tile<VPANELS, kTile>(&v_map, dst, kv_head, unit.begin + key, unit.length - key, full,
                                            smem_addr(&sh.own), &own_parity, gave_up))
          break;
      }
    } else if (warp == kIssuer) {
      // ---- products, all issued by one thread
      if (elect_one()) {
        const uint32_t qk = mma_shape<T>(kTile, false), pv = mma_shape<T>(value16 * 16, true);
        auto full = [&](int i) { return mbar_wait(smem_addr(&sh.kv_full[i % kStages]), (i / kStages) & 1, gave_up); };
        auto scores = [&](int i, int j) {
          product_ss<4>(tmem + i * 128, q_tile + i * kPanelBytes, kv_tile + (2 * j % kStages) * kTileBytes + i * kPanelBytes,
                        qk, dim16);
          mma_commit(smem_addr(&sh.s_full[i]));
        };
        auto output = [&](int i, int j) {
          const uint32_t v = kv_tile + ((2 * j + 1) % kStages) * kTileBytes;
          for (int h = 0; h < 2; ++h) {
            if (!mbar_wait(smem_addr(&sh.p_full[i][h]), j & 1, gave_up)) return false;
            tc_fence_after();
            product_ts<4>(out_at(i), tmem + i * 128 + h * 32, v, h, pv, j > 0 || h > 0);
            mma_commit(smem_addr(&sh.o_done[i]));
          }
          return true;
        };
        bool ok = full(0) && mbar_wait(smem_addr(&sh.q_full), 0, gave_up);
        if (ok) {
          scores(0, 0);
          scores(1, 0);
          mma_commit(smem_addr(&sh.kv_empty[0]));
        }
        for (int j = 0; j < n && ok; ++j) {
          const int vn = 2 * j + 1, kn = vn + 1;
          const bool more = j + 1 < n;
          ok = full(vn) && (!more || full(kn));
          for (int i = 0; i < 2 && ok; ++i)
            if ((ok = output(i, j)) && more) scores(i, j + 1);
          if (!ok) break;
          if (more) mma_commit(smem_addr(&sh.kv_empty[kn % kStages]));
          mma_commit(smem_addr(&sh.kv_empty[vn % kStages]));
        }
        if (ok) mma_commit(smem_addr(&sh.all_done));
      }
      __syncwarp();
    }
  } else {
    take_registers();
    // ---- softmax: a thread has one query's whole row of map i
    const int i = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = lanes + tmem + i * 128, o_at = lanes + out_at(i);
    const int row = (warp & 3) * 32 + lane;
    const float c = a.scale * kLog2e;
    const Two c2 = two(c, c);
    float m = -INFINITY, sum = 0.f;
    auto hide = [&](float (&s)[32], int from) {  // what comes after the row's own key, on the diagonal
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if (from + x > row) s[x] = -INFINITY;
    };
    auto most_of = [&](const float (&s)[32]) {
      float even = fmaxf(s[0], s[1]), odd = fmaxf(s[2], s[3]);
#pragma unroll
      for (int x = 4; x < 32; x += 4) {
        even = max3(even, s[x], s[x + 1]);
        odd = max3(odd, s[x + 2], s[x + 3]);
      }
      return fmaxf(even, odd);
    };
    // 32 scores become 16 columns of pairs; their sum
    auto powers = [&](const float (&s)[32], float m, uint32_t to) {
      const float base = m == -INFINITY ? 0.f : m * c;
      const Two base2 = two(kShift<T> - base, kShift<T> - base);
      Two part[2] = {two(0.f, 0.f), two(0.f, 0.f)};
      uint32_t p[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        float lo, hi;
        split(fma2(two(s[2 * x], s[2 * x + 1]), c2, base2), lo, hi);
        lo = exp2_approx(lo);
        hi = exp2_approx(hi);
        part[x & 1] = add2(part[x & 1], two(lo, hi));
        p[x] = pack2<T>(lo, hi);
      }
      tmem_store16(to, p);
      float lo, hi;
      split(add2(part[0], part[1]), lo, hi);
      return lo + hi;
    };
    // Half a tile at a time.  Its exponentials are taken with the maximum so far
    // while its own is looked for, and once more in the rare case that a row's has
    // grown by too much: they do not wait for it.
    auto step = [&](int j, auto last) {
      if (!mbar_wait(smem_addr(&sh.s_full[i]), j & 1, gave_up)) return false;
      tc_fence_after();
      float s[4][32];
      tmem_load32(s_at, s[0]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float part = 0.f, top[2];
#pragma unroll
        for (int b = 2 * h; b < 2 * h + 2; ++b) {
          tmem_wait_load();
          tmem_loaded(s[b]);
          if (b < 3) tmem_load32(s_at + (b + 1) * 32, s[b + 1]);  // on its way meanwhile
          if constexpr (decltype(last)::value) hide(s[b], b * 32);
          top[b & 1] = most_of(s[b]);
          part += powers(s[b], m, s_at + b * 16);  // (in the place of scores that have been read)
        }
        const float most_s = fmaxf(top[0], top[1]);
        if (__any_sync(0xFFFFFFFFu, (most_s - m) * c > kSlack)) {
          const float moved = fmaxf(m, most_s);
          const float by = m == moved ? 1.f : exp2_approx((m - moved) * c);
          m = moved;
          sum *= by;
          // (these scores are later products than the last tile's outputs: the half before is the current phase or just over)
          const int before = 2 * j + h - 1;
          if (before >= 0) {
            if (!mbar_wait(smem_addr(&sh.o_done[i]), before & 1, gave_up)) return false;
            tc_fence_after();
            for (int d = 0; d < value16; ++d) {
              float o[16];
              tmem_load16(o_at + d * 16, o);
              tmem_wait_load();
              tmem_loaded(o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] *= by;
              tmem_store16(o_at + d * 16, o);
            }
          }
          if (h == 0) tmem_loaded(s[2]);  // it has arrived with the others
          tmem_wait_store();              // the first ones stand where these go
          part = 0.f;
#pragma unroll
          for (int b = 2 * h; b < 2 * h + 2; ++b) part += powers(s[b], m, s_at + b * 16);
        }
        sum += part;
        tmem_wait_store();
        warp_arrive(smem_addr(&sh.p_full[i][h]));
      }
      return true;
    };
    // the first maximum is that of the first 64 keys
    bool ok = mbar_wait(smem_addr(&sh.s_full[i]), 0, gave_up);
    if (ok) {
      tc_fence_after();
      float s[2][32];
      tmem_load32(s_at, s[0]);
      tmem_load32(s_at + 32, s[1]);
      tmem_wait_load();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        tmem_loaded(s[b]);
        if (n == 1) hide(s[b], b * 32);
        m = fmaxf(m, most_of(s[b]));
      }
    }
    // the tile on the diagonal is compiled apart: the others compare nothing
    for (int j = 0; j + 1 < n && ok; ++j) ok = step(j, std::false_type());
    ok = ok && step(n - 1, std::true_type());
    const float by = 1.f / sum;
    if (i) sh.by[row] = by * a.lambda[head];
    named_barrier(1, 256);
    if (ok && mbar_wait(smem_addr(&sh.all_done), 0, gave_up)) {
      tc_fence_after();
      const int from = first + (warp & 3) * 32, at = from + lane;  // within the sequence
      if (a.lse && at < unit.length)
        a.lse[(int64_t)(2 * head + i) * a.tokens + unit.begin + at] = (m * c + (log2f(sum) - kShift<T>)) * kLn2;
      // the first map's warps write the difference, the second's their own
      const AttnTensor& to = i ? a.second : a.out;
      if (to.ptr) {
        if (!i) {
          const float less = sh.by[row];
          const uint32_t other = lanes + out_at(1);
          for (int d = 0; d < value16; ++d) {
            float o[16], l[16];
            tmem_load16(o_at + d * 16, o);
            tmem_load16(other + d * 16, l);
            tmem_wait_load();
            tmem_loaded(o);
            tmem_loaded(l);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = o[x] * by - l[x] * less;
            tmem_store16(o_at + d * 16, o);
          }
          tmem_wait_store();
        }
        T* out = static_cast<T*>(const_cast<void*>(to.ptr)) + (int64_t)(unit.begin + from) * to.token_stride +
                 head * to.head_stride;
        // through the map's queries, which nothing reads any more
        for (int p = 0; p < VPANELS; ++p)
          write_rows<T, 64>(o_at, q_tile + i * kPanelBytes + (warp & 3) * 4096, out, to.token_stride, unit.length - from,
                            p * 64, a.value_dim, i ? by : 1.f);
      }
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
  if (warp == kIssuer) tmem_free(tmem, kColumns);
}

template <class T, int VPANELS>
cudaError_t run(int dtype, const DiffArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> opened[256];
  constexpr int smem = (1 + kStages) * 2 * (int)kPanelBytes;
  cudaError_t e = open_kernel((const void*)diff_attention_kernel<T, VPANELS>, smem, false, opened);
  if (e != cudaSuccess) return e;
  // the warpgroups' shares are sound only if the launch brings them
  static const int registers = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, (const void*)diff_attention_kernel<T, VPANELS>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (registers != kLaunchRegisters) return cudaErrorInvalidConfiguration;
  CUtensorMap q, k, v;
  if (!make_tensor_map(&q, dtype, a.q, a.tokens, 2 * a.heads, a.dim, kTile) ||
      !make_tensor_map(&k, dtype, a.k, a.tokens, 2 * a.kv_heads, a.dim, kTile) ||
      !make_tensor_map(&v, dtype, a.v, a.tokens, a.kv_heads, a.value_dim, kTile))
    return cudaErrorInvalidValue;
  const int64_t units = most_units(a.tokens, a.seqs, kTile);
  diff_attention_kernel<T, VPANELS><<<(unsigned)(units * a.heads), kThreads, smem, s>>>(q, k, v, a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_attention(int dtype, const DiffArgs& a, cudaStream_t s) {
  if (dtype == BF16) return a.value_dim <= 64 ? run<__nv_bfloat16, 1>(dtype, a, s) : run<__nv_bfloat16, 2>(dtype, a, s);
  return a.value_dim <= 64 ? run<__half, 1>(dtype, a, s) : run<__half, 2>(dtype, a, s);
}

cudaError_t diff_attention_take_status(int* status, cudaStream_t s) { return take_status(status, s); }

}  // namespace ar
