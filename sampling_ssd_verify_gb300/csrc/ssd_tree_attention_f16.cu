// ssd_tree_attention_f16.cu -- attention of drafted nodes, float16.
#include "ssd_tree_attention_kernel.cuh"

namespace ssd {
cudaError_t launch_tree_f16(const TreeAttnParams& p, cudaStream_t s) {
  return launch_tree_type<__half>(p, s);
}
}  // namespace ssd
