// Internal interface between the C-ABI layer of the training-step operators
// (ar_ops_api.cpp) and their kernels.  Not installed; not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ar_internal.h"

namespace ar {

// ---- layer norm ------------------------------------------------------------------

struct LayerNormArgs {
  const void* x;
  const void* weight;
  const void* bias;  // may be NULL
  void* y;
  float* mean;  // may be NULL
  float* rstd;  // may be NULL
  int64_t x_stride, y_stride;
  int64_t rows, cols;
  float eps;
};

struct LayerNormBackwardArgs {
  const void* dy;
  const void* x;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dweight;
  void* dbias;      // may be NULL
  float* partial;   // [blocks][2][cols]
  int64_t dy_stride, x_stride, dx_stride;
  int64_t rows, cols;
};

// Most blocks whose partial sums of the parameters' gradients are kept, one row
// of them each: eight on each of the 152 multiprocessors; 64 beyond the widest
// rows that a block keeps.
constexpr int kLayerNormMaxBlocks = 1216, kLayerNormMaxSlices = 64;
constexpr int64_t kLayerNormKeptCols = 16384;
inline int64_t layer_norm_partial_rows(int64_t rows, int64_t cols) {
  const int64_t most = cols > kLayerNormKeptCols ? kLayerNormMaxSlices : kLayerNormMaxBlocks;
  return rows < most ? rows : most;
}

// pdtype: the parameters' type, `dtype` itself or F32
cudaError_t launch_layer_norm(int dtype, int pdtype, const LayerNormArgs& a, cudaStream_t stream);
cudaError_t launch_layer_norm_backward(int dtype, int pdtype, const LayerNormBackwardArgs& a, cudaStream_t stream);

// ---- distillation loss -------------------------------------------------------------

struct DistillArgs {
  const void* logits;
  const int32_t* index;   // [rows][top]
  const void* value;      // [rows][top], `vdtype`
  const float* scale;     // [rows]; NULL: 1
  float* loss;            // forward
  float* lse;             // forward: written; backward: read
  void* dlogits;          // NULL: no gradient
  int64_t logits_stride, dlogits_stride;
  int64_t rows;
  int64_t vocab;
  int32_t top;
  float temperature;
};

constexpr int kDistillMaxTop = 1024;

cudaError_t launch_distill(int dtype, int vdtype, bool backward, const DistillArgs& a, cudaStream_t stream);

// ---- attention -----------------------------------------------------------------------

struct AttnTensor {
  const void* ptr;
  int64_t token_stride, head_stride;  // elements
};

struct AttnArgs {
  AttnTensor q, k, v, out;
  AttnTensor dout, dq, dk, dv;  // backward
  float* lse;                   // [heads][tokens]
  float* delta;                 // backward: [heads][tokens], workspace
  const int32_t* cu_seqlens;    // [seqs + 1]
  int64_t tokens;
  int32_t seqs, heads, kv_heads, dim;
  float scale;
};

cudaError_t launch_attention(int dtype, const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attention_backward(int dtype, const AttnArgs& a, cudaStream_t stream);
// What kernels of the current device left when one of their waits ran out:
// AR_ERR_TIMEOUT is stored in *status, and cleared.  Every operation is in
// `stream`, which the caller has synchronised.
cudaError_t layer_norm_take_status(int* status, cudaStream_t stream);
cudaError_t distill_take_status(int* status, cudaStream_t stream);
cudaError_t attention_take_status(int* status, cudaStream_t stream);
cudaError_t attention_backward_take_status(int* status, cudaStream_t stream);

}  // namespace ar
