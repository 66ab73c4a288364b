// bf16 instantiations of the tree attention on the tensor cores.
#include "pa_tree_mma.cuh"

namespace pa {

cudaError_t launch_tree_mma_bf16(const TreeParams& p, int group, int page_size,
                                 cudaStream_t stream, bool use_pdl) {
  const bool one = group * p.max_q_len <= tree::kTile;
#define PA_TREE_CASE(P)                                                    \
  case P:                                                                  \
    return one ? tree::launch_one<P, 1>(p, group, stream, use_pdl)         \
               : tree::launch_one<P, 2>(p, group, stream, use_pdl);
  switch (page_size) {
    PA_TREE_CASE(16)
    PA_TREE_CASE(32)
    PA_TREE_CASE(64)
    PA_TREE_CASE(128)
  }
#undef PA_TREE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pa
