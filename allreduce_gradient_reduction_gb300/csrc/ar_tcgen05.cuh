// Blackwell's asynchronous units, as the attention kernels use them: mbarriers
// with bounded waits, tiled TMA loads, and the tensor cores' products from
// shared and tensor memory (tcgen05) with their descriptors.
//
// Tiles in shared memory are 128 (or 64) rows of 64 16-bit elements ("panels"
// of 16 KB), in the 128-byte swizzle: row r is the 128 bytes at r * 128, its
// 16-byte pieces permuted within the row by r mod 8.  A row-major matrix of
// 128 columns is two panels, of 128 rows each.  The same panel serves a product in both readings:
// rows as the M or N axis and columns as K ("K-major"), or rows as K and
// columns as the N axis ("MN-major").
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "ar_ops.cuh"

namespace ar {

constexpr int kTile = 128;                        // rows of a tile
constexpr uint32_t kPanelBytes = kTile * 64 * 2;  // 128 rows of 128 bytes

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarriers -------------------------------------------------------------------

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// For a whole warp, after tensor memory accesses that must come before: one
// arrival.  (A barrier takes arrivals one by one, some five cycles each: 128
// threads' own arrivals took 600 cycles.)
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits up to `ns` for the phase of the given parity to end, the thread asleep
// meanwhile.  (Without a time the instruction returns at once, and a warp that
// looks again and again takes every fourth issue slot from the others on its
// quarter of the multiprocessor; it wakes no sooner, 90 cycles after the
// arrival.)
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}
constexpr uint32_t kSleepNs = 10000000;  // one look: as long as the instruction sleeps at most (3.8 us)

// Waits for the phase of the given parity to end.  Every wait is bounded: one
// that runs out (no correct launch does) sets the block's `gave_up`, which
// ends the other threads' waits too, and the caller returns.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  if (mbar_try(bar, parity, kSleepNs)) return true;
  const uint64_t until = global_ns() + kWaitLimitNs;
  for (;;) {
    if (mbar_try(bar, parity, kSleepNs)) return true;
    if (*gave_up) return false;
    if (global_ns() > until) {
      *gave_up = 1;
      return false;
    }
  }
}

// ---- TMA ----------------------------------------------------------------------------

// The box of one panel at (column, head, token); columns are a multiple of 64
// elements, so every copy starts on a 16-byte boundary.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int column, int head, int token,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(map), "r"(column), "r"(head), "r"(token), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One warp loads the panels of a tile of ROWS rows, of which the first `rows`
// belong to the sequence.  The rows after them are another sequence's: they
// are overwritten with zeros before the tile is announced on `full`, so that
// what they hold (an infinity, a NaN) cannot reach a sum through a zero
// weight.  `own` is a barrier of this warp's alone for that case.
template <int PANELS, int ROWS>
__device__ __forceinline__ bool load_tile(const CUtensorMap* map, uint32_t dst, int head, int token, int rows,
                                          uint32_t full, uint32_t own, uint32_t* own_parity, volatile int* gave_up) {
  constexpr uint32_t kBytes = ROWS * 128;
  const int lane = threadIdx.x & 31;
  const bool cut = rows < ROWS;
  if (lane == 0) {
    const uint32_t bar = cut ? own : full;
    mbar_expect(bar, PANELS * kBytes);
    for (int p = 0; p < PANELS; ++p) tma_load(dst + p * kBytes, map, p * 64, head, token, bar);
  }
  if (!cut) return true;
  if (!mbar_wait(own, *own_parity, gave_up)) return false;
  *own_parity ^= 1;
  for (int p = 0; p < PANELS; ++p)
    for (uint32_t b = rows * 128 + lane * 16; b < kBytes; b += 512)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + p * kBytes + b), "r"(0) : "memory");
  fence_async_shared();
  __syncwarp();
  if (lane == 0) mbar_arrive(full);
  return true;
}

// ---- tensor memory -----------------------------------------------------------------

// 128 lanes x 512 columns of 32 bits; an address is lane << 16 | column.  Warp
// w reaches lanes 32 (w mod 4) ... + 31.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 or 16 columns of the thread's lane.  The registers hold the values after
// tmem_wait_load; the empty statement there keeps uses behind it.
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(at)
      : "memory");
}
// Ties the registers to the wait before them.
template <int N>
__device__ __forceinline__ void tmem_loaded(float (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i])::"memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t at, const float (&r)[16]) {
  uint32_t bits[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) bits[i] = __float_as_uint(r[i]);
  tmem_store16(at, bits);
}

// A warp writes COLS columns of its 32 rows of sums from tensor memory, times
// `scale`, rounded: `rows` of them, `dim` columns in all, from `column` on.
// The rows go through 64 COLS bytes of shared memory at `stage`, so that the
// lanes write runs of 2 COLS bytes and not 32 rows at a time.  Whether all sums
// of the lane's row, if it is one of the `rows`, are finite.
template <class T, int COLS>
__device__ __forceinline__ bool write_rows(uint32_t sums, uint32_t stage, T* out, int64_t stride, int rows, int column,
                                           int dim, float scale) {
  constexpr int kPieces = COLS / 8;  // 16-byte pieces of a row
  const int lane = threadIdx.x & 31;
  Two nothing = two(0.f, 0.f);  // NaN once a sum is not finite
  __syncwarp();
  auto place = [&](int row, int piece) {  // pieces of a row change places, so that eight lanes reach all banks
    return stage + row * (COLS * 2) + ((piece ^ (row / (8 / kPieces) & (kPieces - 1))) << 4);
  };
#pragma unroll
  for (int c = 0; c < COLS; c += 16) {
    if (column + c >= dim) break;
    float o[16];
    tmem_load16(sums + column + c, o);
    tmem_wait_load();
    tmem_loaded(o);
#pragma unroll
    for (int i = 0; i < 16; i += 2) nothing = fma2(two(o[i], o[i + 1]), two(0.f, 0.f), nothing);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(lane, c / 8 + h)),
                   "r"(pack2<T>(o[h * 8] * scale, o[h * 8 + 1] * scale)),
                   "r"(pack2<T>(o[h * 8 + 2] * scale, o[h * 8 + 3] * scale)),
                   "r"(pack2<T>(o[h * 8 + 4] * scale, o[h * 8 + 5] * scale)),
                   "r"(pack2<T>(o[h * 8 + 6] * scale, o[h * 8 + 7] * scale))
                   : "memory");
  }
  __syncwarp();
  const int piece = lane % kPieces, at = column + piece * 8;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = lane / kPieces + i * (32 / kPieces);
    if (row >= rows || at >= dim) continue;
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(place(row, piece)) : "memory");
    *reinterpret_cast<uint4*>(out + row * stride + at) = v;
  }
  float lo, hi;
  split(nothing, lo, hi);
  return lane >= rows || lo + hi == 0.f;
}

// ---- products -------------------------------------------------------------------------

// Instruction descriptor: f32 sums, A and B of the same 16-bit type, M = 128.
template <class T>
__device__ __forceinline__ uint32_t mma_shape(int n, bool b_mn_major) {
  const uint32_t type = sizeof(T) == 2 && __is_same(T, __nv_bfloat16) ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | (b_mn_major ? 1u << 16 : 0) | (uint32_t)(n >> 3) << 17 | (kTile >> 4) << 24;
}

// Shared-memory descriptors of a panel (128-byte swizzle): groups of eight
// rows are 1024 bytes apart; MN-major operands wider than a panel find the
// next one kPanelBytes on.
__device__ __forceinline__ uint64_t panel_desc(uint32_t at, bool mn_major) {
  const uint64_t lead = mn_major ? kPanelBytes >> 4 : 1;
  return (uint64_t)((at & 0x3FFFF) >> 4) | lead << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// What the k-th 16 elements along K add to it.
__host__ __device__ constexpr uint32_t k_major_step(int k) { return ((k >> 2) * kPanelBytes + (k & 3) * 32) >> 4; }
__host__ __device__ constexpr uint32_t mn_major_step(int k) { return k * 16 * 128 >> 4; }

// One thread of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
      : "memory");
}
// D = A B^T over `steps` times 16 columns of two K-major tiles.  Issuing is
// one thread's work and has to stay ahead of the tensor cores (64 cycles a
// product of 128 x 128 x 16), so the loop is unrolled and a step's
// descriptors are one addition each.
template <int MAX>
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a_tile, uint32_t b_tile, uint32_t shape, int steps) {
  const uint64_t a = panel_desc(a_tile, false), b = panel_desc(b_tile, false);
#pragma unroll
  for (int k = 0; k < MAX; ++k)
    if (k < steps) mma_ss(d, a + k_major_step(k), b + k_major_step(k), shape, k > 0);
}
// D (+)= P B over STEPS times 16 rows of B, the `part`-th such part of its
// rows; P's pairs of that part, eight columns a step, in tensor memory.
template <int STEPS>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t p, uint32_t b_tile, int part, uint32_t shape, bool add) {
  const uint64_t b = panel_desc(b_tile, true) + part * mn_major_step(STEPS);
#pragma unroll
  for (int k = 0; k < STEPS; ++k) mma_ts(d, p + k * 8, b + mn_major_step(k), shape, k > 0 || add);
}
// Arrives on the barrier when every product issued by this thread so far is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- registers ---------------------------------------------------------------------------

// Blocks of 384 threads are launched with 168 registers each, 64512 in all;
// two warpgroups that hold rows of scores take 208 and the third, which
// issues and loads, keeps 88: 256 * 208 + 128 * 88 = 64512.  Every warp of a
// warpgroup has to say so.
constexpr int kLaunchRegisters = 168;
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;"); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 88;"); }

// ---- packed sequences ------------------------------------------------------------------

// Every sequence is split into ceil(length / size) units, the i-th of which
// (from 0) stands for work in proportion to i + 1; where the first unit is the
// longest, the caller counts from the end.  A launch takes the units of all
// sequences with the most work first, so that no long one starts last.  Every
// block looks at all sequences for that, so with more of them than a warp has
// lanes it takes them in the sequences' order instead, each one's longest first
// (gradient, 12 heads of 64, by work and in order: 24 sequences of 8179 tokens
// 62.8 and 64.0 us, 48 of 8169 68.3 and 61.6, 192 of 8087 172 and 95, 8192 of
// 9182 168 ms and 3.1 ms).
constexpr int kFewSequences = 32;
struct SeqUnit {
  int begin, length;  // the sequence
  int index;          // the unit's place in it
  int count;          // its units; 0: there is no such unit
};

// The unit of place `place` among places that lie closer than units can: sequence
// s has those from floor(begin / size) + s to its successor's, which are its
// ceil(length / size) units or more, whatever begin and length.  So the sequence
// is found by looking at 32 of them at a time, once for every five bits of
// their number.  By one warp.
__device__ __forceinline__ SeqUnit find_unit_in_order(const int32_t* cu_seqlens, int seqs, int tokens, int size,
                                                      int place) {
  const int lane = threadIdx.x & 31;
  auto first_place = [&](int s) { return min(max(cu_seqlens[s], 0), tokens) / size + s; };
  int s = 0;
  for (int range = seqs;;) {
    const int step = (range + 31) / 32, mine = s + lane * step;
    const uint32_t before = __ballot_sync(0xFFFFFFFFu, lane * step < range && first_place(mine) <= place);
    if (!before) return SeqUnit{0, 0, 0, 0};  // it lies before the first sequence
    const int last = 31 - __clz(before);
    s += last * step;
    range = min(step, range - last * step);
    if (step == 1) break;
  }
  const int begin = min(max(cu_seqlens[s], 0), tokens), length = min(max(cu_seqlens[s + 1], begin), tokens) - begin;
  const int n = (length + size - 1) / size, i = place - first_place(s);
  if (i < 0 || i >= n) return SeqUnit{0, 0, 0, 0};
  return SeqUnit{begin, length, n - 1 - i, n};
}

// The `unit`-th unit with the most work first, by one warp.  There are
// sum_s max(0, n_s - w) units with more work than w, n_s being the units of
// sequence s.  The work of the one asked for is found by looking at 32 values
// of w at a time, one to a lane; then the sequence, which is the next one in
// order that has a unit of that work.  Entries of cu_seqlens are clamped, so
// that no value in it leads outside the tensors.
__device__ __forceinline__ SeqUnit find_unit(const int32_t* cu_seqlens, int seqs, int tokens, int size, int unit) {
  if (seqs > kFewSequences) return find_unit_in_order(cu_seqlens, seqs, tokens, size, unit);
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31;
  int begin = 0, length = 0, first = -1;
  auto look = [&](int s0) {  // this lane's sequence of the 32 from s0; its units
    if (s0 != first) {
      const int s = s0 + lane;
      begin = length = 0;
      if (s < seqs) {
        begin = min(max(cu_seqlens[s], 0), tokens);
        length = min(max(cu_seqlens[s + 1], begin), tokens) - begin;
      }
      first = s0;
    }
    return (length + size - 1) / size;
  };
  int w = 0, range = (tokens + size - 1) / size;  // the work less one is in [w, w + range)
  int after;                                      // units with more work than that and one
  for (;;) {
    const int step = (range + 30) / 31;
    const int mine = w + lane * step;
    int above = 0;
    for (int s0 = 0; s0 < seqs; s0 += 32) {
      const int n = look(s0), here = min(32, seqs - s0);
      for (int k = 0; k < here; k += 8)  // lanes without a sequence have no units
#pragma unroll
        for (int i = 0; i < 8; ++i) above += max(__shfl_sync(kAll, n, k + i) - mine, 0);
    }
    const uint32_t more = __ballot_sync(kAll, above > unit);
    if (!more) return SeqUnit{0, 0, 0, 0};
    const int last = 31 - __clz(more);
    w += last * step;
    if (step == 1) {
      after = __shfl_sync(kAll, above, min(last + 1, 31));
      break;
    }
    range = step;
  }
  int place = unit - after;
  for (int s0 = 0; s0 < seqs; s0 += 32) {
    const int n = look(s0);
    const uint32_t has = __ballot_sync(kAll, n > w);
    const int here = __popc(has);
    if (place < here) {
      const bool it = n > w && __popc(has & ((1u << lane) - 1)) == place;
      const int from = __ffs(__ballot_sync(kAll, it)) - 1;
      return SeqUnit{__shfl_sync(kAll, begin, from), __shfl_sync(kAll, length, from), w, __shfl_sync(kAll, n, from)};
    }
    place -= here;
  }
  return SeqUnit{0, 0, 0, 0};
}

// Host: at most this many units (or places), however the tokens are split.
inline int64_t most_units(int64_t tokens, int64_t seqs, int size) {
  return tokens / size + (seqs > kFewSequences || seqs < tokens ? seqs : tokens);
}

// Host: the tensor map of a [tokens][heads][dim] operand, `rows` rows of one
// panel to a box.  False if the driver refuses it.
bool make_tensor_map(CUtensorMap* map, int dtype, const AttnTensor& t, int64_t tokens, int heads, int dim, int rows);

}  // namespace ar
