// int8 instantiations of the tree attention on the tensor cores.
#include "pa_tree_mma.cuh"

namespace pa {

cudaError_t launch_tree_mma_int8(const TreeParams& p, int group, int page_size,
                                 cudaStream_t stream, bool use_pdl) {
  return tree::launch<true>(p, group, page_size, stream, use_pdl);
}

}  // namespace pa
