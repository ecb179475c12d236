// norm_rope.cu -- norm_rope.cuh's kernels for bf16, and the choice of the type.
#include "norm_rope.cuh"

namespace gdn {

cudaError_t launch_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.d.dtype == GDN_TREE_F32) return launch_rope_f32(a, false, stream);
  return launch<__nv_bfloat16, false>(a, stream);
}

cudaError_t launch_cache_append_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.d.dtype == GDN_TREE_F32) return launch_rope_f32(a, true, stream);
  return launch<__nv_bfloat16, true>(a, stream);
}

}  // namespace gdn
