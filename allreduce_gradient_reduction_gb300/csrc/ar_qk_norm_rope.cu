// Norm and rotation of queries and keys, forward: ar_qk_norm_rope.cuh.
#include "ar_qk_norm_rope.cuh"

namespace ar {

cudaError_t launch_qk_norm_rope(int dtype, int wdtype, bool interleaved, const QkArgs& a, cudaStream_t s) {
  return launch_qk<false>(dtype, wdtype, interleaved, a, s);
}

}  // namespace ar
