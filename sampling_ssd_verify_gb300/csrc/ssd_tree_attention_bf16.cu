// ssd_tree_attention_bf16.cu -- attention of drafted nodes, bfloat16.
#include "ssd_tree_attention_kernel.cuh"

namespace ssd {
cudaError_t launch_tree_bf16(const TreeAttnParams& p, cudaStream_t s) {
  return launch_tree_type<__nv_bfloat16>(p, s);
}
}  // namespace ssd
