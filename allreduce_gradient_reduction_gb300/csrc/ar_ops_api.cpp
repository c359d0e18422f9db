// C ABI of the training-step operators: argument checks and launches.
// Declarations and the contract of every entry point are in include/ar.h.
#include "../../include/ar.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>
#include <vector>

#include "ar_internal.h"
#include "ar_ops.h"

namespace {

int esize_of(int dtype) { return dtype == AR_BF16 || dtype == AR_F16 ? 2 : 4; }
bool is_float(int dtype) { return dtype == AR_F32 || dtype == AR_BF16 || dtype == AR_F16; }

// Rows of `width` bytes, `stride` bytes apart; with `pitch`, each of them is
// pieces of `piece` bytes, `pitch` bytes apart, and what lies between those is
// not the operand's.
struct Rows {
  uintptr_t lo;
  uint64_t width, stride, n;
  uint64_t piece = 0, pitch = 0;
  uintptr_t hi() const { return lo + (n - 1) * stride + width; }
};

// False for NULL, a misaligned pointer, or an end past the address space.
bool make_rows(const void* p, int64_t rows, int64_t width, int64_t stride, int esize, Rows* out) {
  const uintptr_t lo = (uintptr_t)p;
  if (!lo || lo % (uintptr_t)esize) return false;
  if (rows == 1) stride = width;
  const __int128 bytes = ((__int128)(rows - 1) * stride + width) * esize;
  if (bytes >= ((__int128)1 << 62) || lo > UINTPTR_MAX - (uintptr_t)bytes) return false;
  *out = Rows{lo, (uint64_t)width * esize, (uint64_t)stride * esize, (uint64_t)rows, 0, 0};
  return true;
}

// Whether b, of `b_width` bytes in each period, comes to lie on a's.
bool meet(uintptr_t a, uint64_t a_width, uintptr_t b, uint64_t b_width, uint64_t period) {
  const uint64_t d = a <= b ? (b - a) % period : period - (a - b) % period;
  const uint64_t at = d % period;  // where b begins within a's period
  return !(at >= a_width && at + b_width <= period);
}

// Whether two sets of rows share a byte (or may: not every arrangement is told
// apart).  Column ranges of the same wide buffer lie between each other's rows
// and do not; nor do parts that alternate piece by piece, where every piece of
// both begins a whole number of pitches from its operand's first.
bool overlap(const Rows& a, const Rows& b) {
  if (a.hi() <= b.lo || b.hi() <= a.lo) return false;
  auto on_pitch = [](const Rows& r) { return r.n == 1 || r.stride % r.pitch == 0; };
  if (a.pitch && a.pitch == b.pitch && on_pitch(a) && on_pitch(b) && !meet(a.lo, a.piece, b.lo, b.piece, a.pitch))
    return false;
  if (a.n == 1 || b.n == 1 || a.stride != b.stride) return true;
  return meet(a.lo, a.width, b.lo, b.width, a.stride);
}

bool same(const Rows& a, const Rows& b) {
  return a.lo == b.lo && a.width == b.width && a.n == b.n && (a.n == 1 || a.stride == b.stride) && a.piece == b.piece &&
         a.pitch == b.pitch;
}

// The operands of a call: what it writes overlaps nothing else, except where
// a result may stand in the place of one input.
struct Operands {
  std::vector<Rows> in, out;
  std::vector<std::pair<size_t, size_t>> shared;  // an output that may be exactly this input
  bool bad = false;
  Rows add(const void* p, int64_t rows, int64_t width, int64_t stride, int esize, std::vector<Rows>* to) {
    Rows r{};
    if (!make_rows(p, rows, width, stride, esize, &r)) bad = true;
    else to->push_back(r);
    return r;
  }
  void read(const void* p, int64_t rows, int64_t width, int64_t stride, int esize) { add(p, rows, width, stride, esize, &in); }
  void write(const void* p, int64_t rows, int64_t width, int64_t stride, int esize) { add(p, rows, width, stride, esize, &out); }
  bool may_share(size_t i, size_t j, int in_place) const {
    if (i == 0 && (int)j < in_place) return true;
    return std::find(shared.begin(), shared.end(), std::make_pair(i, j)) != shared.end();
  }
  // in_place: the first output may be exactly one of the first `in_place` inputs
  int check(int in_place) const {
    if (bad) return AR_ERR_INVALID_ARG;
    for (size_t i = 0; i < out.size(); ++i) {
      for (size_t j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return AR_ERR_INVALID_ARG;
      for (size_t j = 0; j < in.size(); ++j)
        if (overlap(out[i], in[j]) && !(may_share(i, j, in_place) && same(out[i], in[j]))) return AR_ERR_INVALID_ARG;
    }
    std::vector<ar::AddressRange> rs;
    for (const Rows& r : in) rs.push_back({r.lo, r.hi()});
    for (const Rows& r : out) rs.push_back({r.lo, r.hi()});
    return ar::check_device_ranges(rs);
  }
};

int status_of(cudaError_t e) {
  if (e == cudaSuccess) return AR_OK;
  (void)cudaGetLastError();  // the next call's launch must not find this one's failure
  return ar::note_cuda_failure(e);
}

// Nothing may unwind through the C ABI.
template <class F>
int guarded(F f) noexcept {
  try {
    return f();
  } catch (...) {
    return AR_ERR_HOST;
  }
}

constexpr int64_t kMaxRows = INT32_MAX;   // one or more rows to a block of a launch
constexpr int64_t kMaxWidth = 1 << 30;    // columns are counted in 32 bits

int check_layer_norm(int64_t rows, int64_t cols, int dtype, int pdtype) {
  if (rows < 0 || cols < 1 || rows > AR_MAX_COUNT || cols > AR_MAX_COUNT) return AR_ERR_INVALID_ARG;
  if (dtype < AR_F32 || dtype > AR_F16 || pdtype < AR_F32 || pdtype > AR_F16) return AR_ERR_INVALID_ARG;
  if (!is_float(dtype) || (pdtype != AR_F32 && pdtype != dtype)) return AR_ERR_UNSUPPORTED;
  if (rows > kMaxRows || cols > kMaxWidth) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

int check_distill(int64_t rows, int64_t vocab, int64_t top, float temperature, int dtype, int vdtype) {
  if (rows < 0 || vocab < 1 || top < 0 || rows > AR_MAX_COUNT || vocab > AR_MAX_COUNT) return AR_ERR_INVALID_ARG;
  if (dtype < AR_F32 || dtype > AR_F16 || vdtype < AR_F32 || vdtype > AR_F16) return AR_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return AR_ERR_INVALID_ARG;
  if (!is_float(dtype) || (vdtype != AR_F32 && vdtype != dtype)) return AR_ERR_UNSUPPORTED;
  if (rows > kMaxRows || vocab > kMaxWidth || top > ar::kDistillMaxTop) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

int distill(bool backward, const void* logits, int64_t logits_stride, const int32_t* index, const void* value,
            const float* scale, float* loss, float* lse, void* dlogits, int64_t dlogits_stride, int64_t rows,
            int64_t vocab, int64_t top, float temperature, int dtype, int vdtype, cudaStream_t s) {
  int rc = check_distill(rows, vocab, top, temperature, dtype, vdtype);
  if (rc) return rc;
  if (rows > 1 && (logits_stride < vocab || (dlogits && dlogits_stride < vocab))) return AR_ERR_INVALID_ARG;
  if (rows == 0) return AR_OK;
  const int es = esize_of(dtype);
  Operands o;
  o.read(logits, rows, vocab, logits_stride, es);
  if (top > 0) {
    o.read(index, 1, rows * top, 0, 4);
    o.read(value, 1, rows * top, 0, esize_of(vdtype));
  }
  if (scale || backward) o.read(scale, 1, rows, 0, 4);
  if (dlogits || backward) o.write(dlogits, rows, vocab, dlogits_stride, es);
  int in_place = dlogits ? 1 : 0;
  if (backward) {
    o.read(lse, 1, rows, 0, 4);
  } else {
    o.write(loss, 1, rows, 0, 4);
    o.write(lse, 1, rows, 0, 4);
  }
  if ((rc = o.check(in_place))) return rc;
  ar::DistillArgs a{};
  a.logits = logits;
  a.index = index;
  a.value = value;
  a.scale = scale;
  a.loss = loss;
  a.lse = lse;
  a.dlogits = dlogits;
  a.logits_stride = logits_stride;
  a.dlogits_stride = dlogits_stride;
  a.rows = rows;
  a.vocab = vocab;
  a.top = (int32_t)top;
  a.temperature = temperature;
  return status_of(ar::launch_distill(dtype, vdtype, backward, a, s));
}

int check_attention(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t dim, float scale, int dtype) {
  if (tokens < 0 || seqs < 0 || heads < 1 || kv_heads < 1 || dim < 1 || heads % kv_heads) return AR_ERR_INVALID_ARG;
  if (dtype < AR_F32 || dtype > AR_F16 || !(scale > 0.f) || !std::isfinite(scale)) return AR_ERR_INVALID_ARG;
  if ((dtype != AR_BF16 && dtype != AR_F16) || dim % 8 || dim > AR_ATTENTION_MAX_DIM) return AR_ERR_UNSUPPORTED;
  if (tokens > (1 << 30) || seqs > (1 << 24) || heads > 4096 || (tokens / 128 + seqs) * (heads + kv_heads) > INT32_MAX ||
      tokens * heads > INT32_MAX)
    return AR_ERR_TOO_LARGE;
  return AR_OK;
}

// A [tokens][heads][dim] operand: tokens outside heads or heads outside
// tokens, every row of `dim` elements on a 16-byte boundary.  Strides of
// an axis of length one are not looked at.
bool add_tensor(Operands& o, ar::AttnTensor& t, const ar_attention_tensor& p, int64_t tokens, int64_t heads,
                int64_t dim, bool written) {
  int64_t ts = p.token_stride, hs = p.head_stride;
  if (heads == 1) hs = dim;
  if (tokens == 1) ts = heads * (hs > dim ? hs : dim);
  if (ts < dim || hs < dim || ts > AR_MAX_COUNT || hs > AR_MAX_COUNT || ts % 8 || hs % 8) return false;
  if ((uintptr_t)p.data % 16) return false;
  const bool token_major = ts >= (__int128)(heads - 1) * hs + dim;
  const bool head_major = hs >= (__int128)(tokens - 1) * ts + dim;
  if (!token_major && !head_major) return false;
  std::vector<Rows>* to = written ? &o.out : &o.in;
  if (token_major) o.add(p.data, tokens, (heads - 1) * hs + dim, ts, 2, to);
  else o.add(p.data, heads, (tokens - 1) * ts + dim, hs, 2, to);
  if (!o.bad && (token_major ? heads : tokens) > 1) {
    to->back().piece = (uint64_t)dim * 2;
    to->back().pitch = (uint64_t)(token_major ? hs : ts) * 2;
  }
  t = ar::AttnTensor{p.data, ts, hs};
  return true;
}

int64_t attention_workspace(int64_t tokens, int64_t heads) { return (tokens * heads * 4 + 15) / 16 * 16; }

int check_diff_attention(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t dim, int64_t value_dim,
                         float scale, int dtype) {
  const int rc = check_attention(tokens, seqs, heads, kv_heads, dim, scale, dtype);
  if (value_dim < 1) return AR_ERR_INVALID_ARG;
  if (rc) return rc;
  if (dim > AR_DIFF_ATTENTION_MAX_DIM || value_dim % 8 || value_dim > AR_ATTENTION_MAX_DIM) return AR_ERR_UNSUPPORTED;
  // every head twice, and blocks of their own for the gradient of lambda
  if (heads > 2048 || (tokens / 128 + seqs) * (heads + kv_heads) > INT32_MAX - heads || 2 * tokens * heads > INT32_MAX)
    return AR_ERR_TOO_LARGE;
  return AR_OK;
}

// ---- norm and rotation of queries and keys

int check_qk(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim) {
  if (tokens < 0 || heads < 1 || kv_heads < 0 || dim < 1) return AR_ERR_INVALID_ARG;
  if (dim % 2 || dim > AR_QK_MAX_DIM) return AR_ERR_UNSUPPORTED;
  if (tokens > kMaxRows || heads > (1 << 20) || kv_heads > (1 << 20)) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

// A [tokens][heads][dim] operand of any strides with tokens or heads as the
// outer axis.
bool add_heads(Operands& o, ar::QkTensor& t, const ar_attention_tensor* p, int64_t tokens, int64_t heads, int64_t dim,
               int esize, bool written) {
  if (!p) return false;
  int64_t ts = p->token_stride, hs = p->head_stride;
  if (heads == 1) hs = dim;
  if (tokens == 1) ts = heads * (hs > dim ? hs : dim);
  if (ts < dim || hs < dim || ts > AR_MAX_COUNT || hs > AR_MAX_COUNT) return false;
  const bool token_major = ts >= (__int128)(heads - 1) * hs + dim;
  const bool head_major = hs >= (__int128)(tokens - 1) * ts + dim;
  if (!token_major && !head_major) return false;
  std::vector<Rows>* to = written ? &o.out : &o.in;
  if (token_major) o.add(p->data, tokens, (heads - 1) * hs + dim, ts, esize, to);
  else o.add(p->data, heads, (tokens - 1) * ts + dim, hs, esize, to);
  if (!o.bad && (token_major ? heads : tokens) > 1) {
    to->back().piece = (uint64_t)dim * esize;
    to->back().pitch = (uint64_t)(token_major ? hs : ts) * esize;
  }
  t = ar::QkTensor{p->data, ts, hs};
  return true;
}

// 1 / (2 pi), its bits after the point (by Machin's formula).
constexpr uint64_t kInverseTurn[] = {
    0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull, 0x7f9458eaf7aef158ull,
    0x6dc91b8e909374b8ull, 0x01924bba82746487ull, 0x3f877ac72c4a69cfull, 0xba208d7d4baed121ull,
    0x3a671c09ad17df90ull, 0x4e64758e60d4ce7dull, 0x272117e2ef7e4a0eull, 0xc7fe25fff7816603ull,
    0xfbcbc462d6829b47ull, 0xdb4d9fb3c9f2c26dull, 0xd3d18fd9a797fa8bull, 0x5d49eeb1faf97c5eull,
    0xcf41ce7de294a4baull, 0x9afed7ec47e35742ull, 0x1580cc11bf1edaeaull,
};

// A finite frequency in turns, its part below one times 2^64, to the nearest: the
// binary64 is whole / 2^k, and of the constant's bits only those matter that give
// neither whole turns nor less than is asked for (Payne and Hanek's reduction).
// A quotient in binary64 loses as many bits as its turns have: at position 2^31 a
// frequency of 10 was 2e-6 radians off, one of 1e9 anything.
uint64_t fraction_of_turn(double frequency) {
  int shift;
  const double half = std::frexp(std::fabs(frequency), &shift);  // below one
  const uint64_t whole = (uint64_t)std::ldexp(half, 53);
  shift -= 53;  // the frequency is whole * 2^shift
  // the constant's 64 bits after the first `skip`, which is at most 971 + 128
  auto bits = [](int skip) -> uint64_t {
    if (skip <= -64) return 0;
    if (skip < 0) return kInverseTurn[0] >> -skip;
    const uint64_t* at = kInverseTurn + skip / 64;
    return skip % 64 ? at[0] << skip % 64 | at[1] >> (64 - skip % 64) : at[0];
  };
  // whole times 192 bits, modulo 2^192: what is cut off is below whole, 2^-139 turns
  unsigned __int128 part = (unsigned __int128)whole * bits(shift + 128);
  part = (unsigned __int128)whole * bits(shift + 64) + (uint64_t)(part >> 64);
  const uint64_t round = (uint64_t)part >> 63;
  const uint64_t turn = whole * bits(shift) + (uint64_t)(part >> 64) + round;
  return std::signbit(frequency) ? 0 - turn : turn;
}

// Turns per position of each pair, times 2^64, or NULL.  A training loop asks for
// the same ones in every call, and powers take longer than the rest of it, so a
// thread has those of its last base at hand.  Those of frequencies are put into
// `turn`.
const uint64_t* turns_of(uint64_t* turn, int64_t rotary, double base, const double* frequencies) {
  if (frequencies) {
    for (int64_t i = 0; i < rotary / 2; ++i) {
      if (!std::isfinite(frequencies[i])) return nullptr;
      turn[i] = fraction_of_turn(frequencies[i]);
    }
    return turn;
  }
  struct Last {
    double base = 0;
    int64_t rotary = 0;
    uint64_t turn[ar::kQkMaxDim / 2];
  };
  static thread_local Last last;
  if (last.base != base || last.rotary != rotary) {
    last.rotary = -1;
    for (int64_t i = 0; i < rotary / 2; ++i) {
      const double f = std::pow(base, -2.0 * (double)i / (double)rotary);
      if (!std::isfinite(f)) return nullptr;
      last.turn[i] = fraction_of_turn(f);
    }
    last.base = base;
    last.rotary = rotary;
  }
  return last.turn;
}

int64_t qk_workspace(int64_t dim) { return (int64_t)ar::kQkMaxBlocks * dim * (int64_t)sizeof(float); }

int qk_norm_rope(bool backward, const ar_attention_tensor* q_up, const ar_attention_tensor* k_up,
                 const ar_attention_tensor* q, const ar_attention_tensor* k, const void* q_weight, const void* k_weight,
                 const int32_t* positions, const ar_attention_tensor* q_out, const ar_attention_tensor* k_out,
                 void* dq_weight, void* dk_weight, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim,
                 int64_t rotary, double base, const double* frequencies, bool interleaved, float eps, int dtype,
                 int wdtype, void* workspace, int64_t workspace_bytes, cudaStream_t s) {
  int rc = check_qk(tokens, heads, kv_heads, dim);
  if (rc == AR_ERR_INVALID_ARG) return rc;
  if (rotary < 0 || rotary > dim || rotary % 2 || !(eps >= 0.f) || !std::isfinite(eps)) return AR_ERR_INVALID_ARG;
  if (!frequencies && (!(base > 0.0) || !std::isfinite(base))) return AR_ERR_INVALID_ARG;
  if (dtype < AR_F32 || dtype > AR_F16 || wdtype < AR_F32 || wdtype > AR_F16) return AR_ERR_INVALID_ARG;
  if (!is_float(dtype) || (wdtype != AR_F32 && wdtype != dtype)) return AR_ERR_UNSUPPORTED;
  if (rc) return rc;
  const int es = esize_of(dtype), ws = esize_of(wdtype);
  ar::QkArgs a{};
  uint64_t turn[ar::kQkMaxDim / 2];
  if (!(a.turn = turns_of(turn, rotary, base, frequencies))) return AR_ERR_INVALID_ARG;
  if (kv_heads == 0) k_weight = nullptr;
  Operands o;
  void* const dweight[2] = {dq_weight, dk_weight};
  if (tokens == 0) {
    // empty sums
    for (void* w : dweight)
      if (w) o.write(w, 1, dim, 0, ws);
    if (o.out.empty() && !o.bad) return AR_OK;
    if ((rc = o.check(0))) return rc;
    for (void* w : dweight)
      if (w && (rc = status_of(cudaMemsetAsync(w, 0, (size_t)dim * ws, s)))) return rc;
    return AR_OK;
  }
  const ar_attention_tensor* const x[2] = {q, k};
  const ar_attention_tensor* const up[2] = {q_up, k_up};
  const ar_attention_tensor* const y[2] = {q_out, k_out};
  const int64_t n[2] = {heads, kv_heads};
  for (int t = 0; t < 2; ++t) {
    if (!n[t]) continue;
    if (!add_heads(o, a.x[t], x[t], tokens, n[t], dim, es, false)) return AR_ERR_INVALID_ARG;
    o.shared.push_back({(size_t)t, o.in.size() - 1});
    if (backward) {
      if (!add_heads(o, a.dy[t], up[t], tokens, n[t], dim, es, false)) return AR_ERR_INVALID_ARG;
      o.shared.push_back({(size_t)t, o.in.size() - 1});
    }
    if (!add_heads(o, a.y[t], y[t], tokens, n[t], dim, es, true)) return AR_ERR_INVALID_ARG;
  }
  if (q_weight) o.read(q_weight, 1, dim, 0, ws);
  if (k_weight) o.read(k_weight, 1, dim, 0, ws);
  o.read(positions, 1, tokens, 0, 4);
  if (dq_weight || dk_weight) {
    if (workspace_bytes < qk_workspace(dim)) return AR_ERR_INVALID_ARG;
    for (void* w : dweight)
      if (w) o.write(w, 1, dim, 0, ws);
    o.write(workspace, 1, qk_workspace(dim) / 4, 0, 4);
    a.partial = static_cast<float*>(workspace);
  }
  if ((rc = o.check(0))) return rc;
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.dweight[0] = dq_weight;
  a.dweight[1] = dk_weight;
  a.positions = positions;
  a.tokens = tokens;
  a.heads[0] = (int32_t)heads;
  a.heads[1] = (int32_t)kv_heads;
  a.dim = (int32_t)dim;
  a.rotary = (int32_t)rotary;
  a.eps = eps;
  return status_of(backward ? ar::launch_qk_norm_rope_backward(dtype, wdtype, interleaved, a, s)
                            : ar::launch_qk_norm_rope(dtype, wdtype, interleaved, a, s));
}

// ---- activation kept in 8 bits

int check_activation8(int64_t rows, int64_t cols, int kind, int dtype) {
  if (rows < 0 || cols < 1 || rows > AR_MAX_COUNT || cols > AR_MAX_COUNT) return AR_ERR_INVALID_ARG;
  if (dtype < AR_F32 || dtype > AR_F16 || kind < AR_ACT_IDENTITY || kind > AR_ACT_GELU) return AR_ERR_INVALID_ARG;
  if (!is_float(dtype)) return AR_ERR_UNSUPPORTED;
  // blocks are counted in 31 bits, past the last by as many as a launch's last threads go
  const int64_t blocks = (cols + AR_ACTIVATION8_BLOCK - 1) / AR_ACTIVATION8_BLOCK;
  if (rows > kMaxRows || cols > kMaxWidth || rows * blocks > INT32_MAX - 4096) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

ar::Activation8Args activation8_args(int64_t rows, int64_t cols) {
  ar::Activation8Args a{};
  a.cols = (int32_t)cols;
  a.blocks = (int32_t)((cols + AR_ACTIVATION8_BLOCK - 1) / AR_ACTIVATION8_BLOCK);
  a.total = (uint32_t)(rows * a.blocks);
  return a;
}

}  // namespace

extern "C" {

int ar_layer_norm(const void* x, int64_t x_stride, const void* weight, const void* bias, void* y, int64_t y_stride,
                  float* mean, float* rstd, int64_t rows, int64_t cols, float eps, ar_dtype dtype,
                  ar_dtype param_dtype, ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_layer_norm(rows, cols, dtype, param_dtype);
    if (rc) return rc;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return AR_ERR_INVALID_ARG;
    if (rows > 1 && (x_stride < cols || y_stride < cols)) return AR_ERR_INVALID_ARG;
    if (rows == 0) return AR_OK;
    const int es = esize_of(dtype), ps = esize_of(param_dtype);
    Operands o;
    o.read(x, rows, cols, x_stride, es);
    o.read(weight, 1, cols, 0, ps);
    if (bias) o.read(bias, 1, cols, 0, ps);
    o.write(y, rows, cols, y_stride, es);
    if (mean) o.write(mean, 1, rows, 0, 4);
    if (rstd) o.write(rstd, 1, rows, 0, 4);
    if ((rc = o.check(1))) return rc;
    ar::LayerNormArgs a{x, weight, bias, y, mean, rstd, x_stride, y_stride, rows, cols, eps};
    return status_of(ar::launch_layer_norm(dtype, param_dtype, a, (cudaStream_t)stream));
  });
}

int64_t ar_layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || rows > kMaxRows || cols > kMaxWidth) return AR_ERR_INVALID_ARG;
  return ar::layer_norm_partial_rows(rows, cols) * 2 * cols * (int64_t)sizeof(float);
}

int ar_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, const void* weight,
                           const float* mean, const float* rstd, void* dx, int64_t dx_stride, void* dweight,
                           void* dbias, int64_t rows, int64_t cols, ar_dtype dtype, ar_dtype param_dtype,
                           void* workspace, int64_t workspace_bytes, ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_layer_norm(rows, cols, dtype, param_dtype);
    if (rc) return rc;
    if (rows > 1 && (x_stride < cols || dy_stride < cols || dx_stride < cols)) return AR_ERR_INVALID_ARG;
    const int es = esize_of(dtype), ps = esize_of(param_dtype);
    Operands o;
    if (rows == 0) {
      // no rows: the parameters' gradients are empty sums
      o.write(dweight, 1, cols, 0, ps);
      if (dbias) o.write(dbias, 1, cols, 0, ps);
      if ((rc = o.check(0))) return rc;
      if ((rc = status_of(cudaMemsetAsync(dweight, 0, (size_t)cols * ps, (cudaStream_t)stream)))) return rc;
      return dbias ? status_of(cudaMemsetAsync(dbias, 0, (size_t)cols * ps, (cudaStream_t)stream)) : AR_OK;
    }
    const int64_t need = ar_layer_norm_workspace_bytes(rows, cols);
    if (workspace_bytes < need) return AR_ERR_INVALID_ARG;
    o.read(dy, rows, cols, dy_stride, es);
    o.read(x, rows, cols, x_stride, es);
    o.read(weight, 1, cols, 0, ps);
    o.read(mean, 1, rows, 0, 4);
    o.read(rstd, 1, rows, 0, 4);
    o.write(dx, rows, cols, dx_stride, es);
    o.write(dweight, 1, cols, 0, ps);
    if (dbias) o.write(dbias, 1, cols, 0, ps);
    o.write(workspace, 1, need / 4, 0, 4);
    if ((rc = o.check(2))) return rc;
    ar::LayerNormBackwardArgs a{dy, x, weight, mean, rstd, dx, dweight, dbias, static_cast<float*>(workspace),
                                dy_stride, x_stride, dx_stride, rows, cols};
    return status_of(ar::launch_layer_norm_backward(dtype, param_dtype, a, (cudaStream_t)stream));
  });
}

int ar_distill_loss(const void* logits, int64_t logits_stride, const int32_t* teacher_index,
                    const void* teacher_logits, const float* scale, float* loss, float* lse, void* dlogits,
                    int64_t dlogits_stride, int64_t rows, int64_t vocab, int64_t top, float temperature,
                    ar_dtype dtype, ar_dtype teacher_dtype, ar_stream_t stream) {
  return guarded([&]() -> int {
    return distill(false, logits, logits_stride, teacher_index, teacher_logits, scale, loss, lse, dlogits,
                   dlogits_stride, rows, vocab, top, temperature, dtype, teacher_dtype, (cudaStream_t)stream);
  });
}

int ar_distill_loss_backward(const void* logits, int64_t logits_stride, const int32_t* teacher_index,
                             const void* teacher_logits, const float* lse, const float* dloss, void* dlogits,
                             int64_t dlogits_stride, int64_t rows, int64_t vocab, int64_t top, float temperature,
                             ar_dtype dtype, ar_dtype teacher_dtype, ar_stream_t stream) {
  return guarded([&]() -> int {
    return distill(true, logits, logits_stride, teacher_index, teacher_logits, dloss, nullptr,
                   const_cast<float*>(lse), dlogits, dlogits_stride, rows, vocab, top, temperature, dtype,
                   teacher_dtype, (cudaStream_t)stream);
  });
}

int ar_attention(const ar_attention_tensor* q, const ar_attention_tensor* k, const ar_attention_tensor* v,
                 const int32_t* cu_seqlens, const ar_attention_tensor* out, float* lse, int64_t tokens, int64_t seqs,
                 int64_t heads, int64_t kv_heads, int64_t dim, float scale, ar_dtype dtype, ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_attention(tokens, seqs, heads, kv_heads, dim, scale, dtype);
    if (rc) return rc;
    if (!q || !k || !v || !out) return AR_ERR_INVALID_ARG;
    if (tokens == 0 || seqs == 0) return AR_OK;
    ar::AttnArgs a{};
    Operands o;
    if (!add_tensor(o, a.q, *q, tokens, heads, dim, false) || !add_tensor(o, a.k, *k, tokens, kv_heads, dim, false) ||
        !add_tensor(o, a.v, *v, tokens, kv_heads, dim, false) || !add_tensor(o, a.out, *out, tokens, heads, dim, true))
      return AR_ERR_INVALID_ARG;
    o.read(cu_seqlens, 1, seqs + 1, 0, 4);
    if (lse) o.write(lse, 1, tokens * heads, 0, 4);
    if ((rc = o.check(0))) return rc;
    a.lse = lse;
    a.cu_seqlens = cu_seqlens;
    a.tokens = tokens;
    a.seqs = (int32_t)seqs;
    a.heads = (int32_t)heads;
    a.kv_heads = (int32_t)kv_heads;
    a.dim = (int32_t)dim;
    a.scale = scale;
    return status_of(ar::launch_attention(dtype, a, (cudaStream_t)stream));
  });
}

int64_t ar_attention_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim) {
  const int rc = check_attention(tokens, 1, heads, kv_heads, dim, 1.f, AR_BF16);
  return rc ? rc : attention_workspace(tokens, heads);
}

int ar_attention_backward(const ar_attention_tensor* dout, const ar_attention_tensor* q, const ar_attention_tensor* k,
                          const ar_attention_tensor* v, const ar_attention_tensor* out, const float* lse,
                          const int32_t* cu_seqlens, const ar_attention_tensor* dq, const ar_attention_tensor* dk,
                          const ar_attention_tensor* dv, int64_t tokens, int64_t seqs, int64_t heads,
                          int64_t kv_heads, int64_t dim, float scale, ar_dtype dtype, void* workspace,
                          int64_t workspace_bytes, ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_attention(tokens, seqs, heads, kv_heads, dim, scale, dtype);
    if (rc) return rc;
    if (!dout || !q || !k || !v || !out || !dq || !dk || !dv) return AR_ERR_INVALID_ARG;
    if (tokens == 0 || seqs == 0) return AR_OK;
    const int64_t need = attention_workspace(tokens, heads);
    if (workspace_bytes < need || (uintptr_t)workspace % 16) return AR_ERR_INVALID_ARG;
    ar::AttnArgs a{};
    Operands o;
    if (!add_tensor(o, a.q, *q, tokens, heads, dim, false) || !add_tensor(o, a.k, *k, tokens, kv_heads, dim, false) ||
        !add_tensor(o, a.v, *v, tokens, kv_heads, dim, false) || !add_tensor(o, a.out, *out, tokens, heads, dim, false) ||
        !add_tensor(o, a.dout, *dout, tokens, heads, dim, false) || !add_tensor(o, a.dq, *dq, tokens, heads, dim, true) ||
        !add_tensor(o, a.dk, *dk, tokens, kv_heads, dim, true) || !add_tensor(o, a.dv, *dv, tokens, kv_heads, dim, true))
      return AR_ERR_INVALID_ARG;
    o.read(cu_seqlens, 1, seqs + 1, 0, 4);
    o.read(lse, 1, tokens * heads, 0, 4);
    o.write(workspace, 1, need / 4, 0, 4);
    if ((rc = o.check(0))) return rc;
    a.lse = const_cast<float*>(lse);
    a.delta = static_cast<float*>(workspace);
    a.cu_seqlens = cu_seqlens;
    a.tokens = tokens;
    a.seqs = (int32_t)seqs;
    a.heads = (int32_t)heads;
    a.kv_heads = (int32_t)kv_heads;
    a.dim = (int32_t)dim;
    a.scale = scale;
    return status_of(ar::launch_attention_backward(dtype, a, (cudaStream_t)stream));
  });
}

int ar_qk_norm_rope(const ar_attention_tensor* q, const ar_attention_tensor* k, const void* q_weight,
                    const void* k_weight, const int32_t* positions, const ar_attention_tensor* q_out,
                    const ar_attention_tensor* k_out, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim,
                    int64_t rotary_dim, double base, const double* frequencies, int interleaved, float eps,
                    ar_dtype dtype, ar_dtype weight_dtype, ar_stream_t stream) {
  return guarded([&]() -> int {
    return qk_norm_rope(false, nullptr, nullptr, q, k, q_weight, k_weight, positions, q_out, k_out, nullptr, nullptr,
                        tokens, heads, kv_heads, dim, rotary_dim, base, frequencies, interleaved != 0, eps, dtype,
                        weight_dtype, nullptr, 0, (cudaStream_t)stream);
  });
}

int64_t ar_qk_norm_rope_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim) {
  const int rc = check_qk(tokens, heads, kv_heads, dim);
  return rc ? rc : qk_workspace(dim);
}

int ar_qk_norm_rope_backward(const ar_attention_tensor* dq_out, const ar_attention_tensor* dk_out,
                             const ar_attention_tensor* q, const ar_attention_tensor* k, const void* q_weight,
                             const void* k_weight, const int32_t* positions, const ar_attention_tensor* dq,
                             const ar_attention_tensor* dk, void* dq_weight, void* dk_weight, int64_t tokens,
                             int64_t heads, int64_t kv_heads, int64_t dim, int64_t rotary_dim, double base,
                             const double* frequencies, int interleaved, float eps, ar_dtype dtype,
                             ar_dtype weight_dtype, void* workspace, int64_t workspace_bytes, ar_stream_t stream) {
  return guarded([&]() -> int {
    return qk_norm_rope(true, dq_out, dk_out, q, k, q_weight, k_weight, positions, dq, dk, dq_weight, dk_weight, tokens,
                        heads, kv_heads, dim, rotary_dim, base, frequencies, interleaved != 0, eps, dtype, weight_dtype,
                        workspace, workspace_bytes, (cudaStream_t)stream);
  });
}

int ar_diff_attention(const ar_attention_tensor* q, const ar_attention_tensor* k, const ar_attention_tensor* v,
                      const float* lambda, const int32_t* cu_seqlens, const ar_attention_tensor* out,
                      const ar_attention_tensor* second, float* lse, int64_t tokens, int64_t seqs, int64_t heads,
                      int64_t kv_heads, int64_t dim, int64_t value_dim, float scale, ar_dtype dtype,
                      ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_diff_attention(tokens, seqs, heads, kv_heads, dim, value_dim, scale, dtype);
    if (rc) return rc;
    if (!q || !k || !v || !out) return AR_ERR_INVALID_ARG;
    if (tokens == 0 || seqs == 0) return AR_OK;
    ar::DiffArgs a{};
    Operands o;
    if (!add_tensor(o, a.q, *q, tokens, 2 * heads, dim, false) || !add_tensor(o, a.k, *k, tokens, 2 * kv_heads, dim, false) ||
        !add_tensor(o, a.v, *v, tokens, kv_heads, value_dim, false) ||
        !add_tensor(o, a.out, *out, tokens, heads, value_dim, true) ||
        (second && !add_tensor(o, a.second, *second, tokens, heads, value_dim, true)))
      return AR_ERR_INVALID_ARG;
    o.read(lambda, 1, heads, 0, 4);
    o.read(cu_seqlens, 1, seqs + 1, 0, 4);
    if (lse) o.write(lse, 1, 2 * tokens * heads, 0, 4);
    if ((rc = o.check(0))) return rc;
    a.lambda = lambda;
    a.lse = lse;
    a.cu_seqlens = cu_seqlens;
    a.tokens = tokens;
    a.seqs = (int32_t)seqs;
    a.heads = (int32_t)heads;
    a.kv_heads = (int32_t)kv_heads;
    a.dim = (int32_t)dim;
    a.value_dim = (int32_t)value_dim;
    a.scale = scale;
    return status_of(ar::launch_diff_attention(dtype, a, (cudaStream_t)stream));
  });
}

int64_t ar_diff_attention_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim,
                                          int64_t value_dim) {
  const int rc = check_diff_attention(tokens, 1, heads, kv_heads, dim, value_dim, 1.f, AR_BF16);
  return rc ? rc : attention_workspace(tokens, 2 * heads);
}

int ar_diff_attention_backward(const ar_attention_tensor* dout, const ar_attention_tensor* q,
                               const ar_attention_tensor* k, const ar_attention_tensor* v, const float* lambda,
                               const ar_attention_tensor* out, const ar_attention_tensor* second, const float* lse,
                               const int32_t* cu_seqlens, const ar_attention_tensor* dq, const ar_attention_tensor* dk,
                               const ar_attention_tensor* dv, float* dlambda, int64_t tokens, int64_t seqs,
                               int64_t heads, int64_t kv_heads, int64_t dim, int64_t value_dim, float scale,
                               ar_dtype dtype, void* workspace, int64_t workspace_bytes, ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_diff_attention(tokens, seqs, heads, kv_heads, dim, value_dim, scale, dtype);
    if (rc) return rc;
    if (!dout || !q || !k || !v || !out || !second || !dq || !dk || !dv) return AR_ERR_INVALID_ARG;
    Operands o;
    if (tokens == 0 || seqs == 0) {
      // no tokens: lambda's gradients are empty sums
      if (!dlambda) return AR_OK;
      o.write(dlambda, 1, heads, 0, 4);
      if ((rc = o.check(0))) return rc;
      return status_of(cudaMemsetAsync(dlambda, 0, (size_t)heads * 4, (cudaStream_t)stream));
    }
    const int64_t need = attention_workspace(tokens, 2 * heads);
    if (workspace_bytes < need || (uintptr_t)workspace % 16) return AR_ERR_INVALID_ARG;
    ar::DiffArgs a{};
    if (!add_tensor(o, a.q, *q, tokens, 2 * heads, dim, false) || !add_tensor(o, a.k, *k, tokens, 2 * kv_heads, dim, false) ||
        !add_tensor(o, a.v, *v, tokens, kv_heads, value_dim, false) ||
        !add_tensor(o, a.out, *out, tokens, heads, value_dim, false) ||
        !add_tensor(o, a.second, *second, tokens, heads, value_dim, false) ||
        !add_tensor(o, a.dout, *dout, tokens, heads, value_dim, false) ||
        !add_tensor(o, a.dq, *dq, tokens, 2 * heads, dim, true) || !add_tensor(o, a.dk, *dk, tokens, 2 * kv_heads, dim, true) ||
        !add_tensor(o, a.dv, *dv, tokens, kv_heads, value_dim, true))
      return AR_ERR_INVALID_ARG;
    o.read(lambda, 1, heads, 0, 4);
    o.read(cu_seqlens, 1, seqs + 1, 0, 4);
    o.read(lse, 1, 2 * tokens * heads, 0, 4);
    if (dlambda) o.write(dlambda, 1, heads, 0, 4);
    o.write(workspace, 1, need / 4, 0, 4);
    if ((rc = o.check(0))) return rc;
    a.lambda = lambda;
    a.dlambda = dlambda;
    a.lse = const_cast<float*>(lse);
    a.delta = static_cast<float*>(workspace);
    a.cu_seqlens = cu_seqlens;
    a.tokens = tokens;
    a.seqs = (int32_t)seqs;
    a.heads = (int32_t)heads;
    a.kv_heads = (int32_t)kv_heads;
    a.dim = (int32_t)dim;
    a.value_dim = (int32_t)value_dim;
    a.scale = scale;
    return status_of(ar::launch_diff_attention_backward(dtype, a, (cudaStream_t)stream));
  });
}

int ar_activation8(const void* x, int64_t x_stride, void* y, int64_t y_stride, int8_t* codes, float* scales,
                   int64_t rows, int64_t cols, ar_activation kind, ar_dtype dtype, ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_activation8(rows, cols, kind, dtype);
    if (rc) return rc;
    if (rows > 1 && (x_stride < cols || (y && y_stride < cols))) return AR_ERR_INVALID_ARG;
    if (rows == 0) return AR_OK;
    if ((uintptr_t)codes % 16) return AR_ERR_INVALID_ARG;
    const int es = esize_of(dtype);
    ar::Activation8Args a = activation8_args(rows, cols);
    Operands o;
    o.read(x, rows, cols, x_stride, es);
    if (y) o.write(y, rows, cols, y_stride, es);
    o.write(codes, 1, (int64_t)a.total * AR_ACTIVATION8_BLOCK, 0, 1);
    o.write(scales, 1, a.total, 0, 4);
    if ((rc = o.check(y ? 1 : 0))) return rc;
    a.x = x;
    a.y = y;
    a.codes_out = codes;
    a.scales_out = scales;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    return status_of(ar::launch_activation8(dtype, kind, rows, a, (cudaStream_t)stream));
  });
}

int ar_activation8_backward(const int8_t* codes, const float* scales, const void* dy, int64_t dy_stride, void* dx,
                            int64_t dx_stride, void* y, int64_t y_stride, int64_t rows, int64_t cols,
                            ar_activation kind, ar_dtype dtype, ar_stream_t stream) {
  return guarded([&]() -> int {
    int rc = check_activation8(rows, cols, kind, dtype);
    if (rc) return rc;
    if (rows == 0) return AR_OK;
    if (!dx != !dy || (!dx && !y)) return AR_ERR_INVALID_ARG;
    if (rows > 1 && ((dx && (dy_stride < cols || dx_stride < cols)) || (y && y_stride < cols))) return AR_ERR_INVALID_ARG;
    if ((uintptr_t)codes % 16) return AR_ERR_INVALID_ARG;
    const int es = esize_of(dtype);
    ar::Activation8Args a = activation8_args(rows, cols);
    Operands o;
    if (dx) {
      o.read(dy, rows, cols, dy_stride, es);
      o.write(dx, rows, cols, dx_stride, es);
    }
    o.read(codes, 1, (int64_t)a.total * AR_ACTIVATION8_BLOCK, 0, 1);
    o.read(scales, 1, a.total, 0, 4);
    if (y) o.write(y, rows, cols, y_stride, es);
    if ((rc = o.check(dx ? 1 : 0))) return rc;
    a.x = dy;
    a.y = y;
    a.dx = dx;
    a.codes = codes;
    a.scales = scales;
    a.x_stride = dy_stride;
    a.y_stride = y_stride;
    a.dx_stride = dx_stride;
    return status_of(ar::launch_activation8_backward(dtype, kind, rows, a, (cudaStream_t)stream));
  });
}

}  // extern "C"
