// norm_rope_f32.cu -- norm_rope.cuh's kernels for fp32 (a file of their own: they compile beside
// those for bf16).
#include "norm_rope.cuh"

namespace gdn {

cudaError_t launch_rope_f32(const RopeArgs& a, bool append, cudaStream_t stream) {
  return append ? launch<float, true>(a, stream) : launch<float, false>(a, stream);
}

}  // namespace gdn
