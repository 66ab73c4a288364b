// bf16 instantiations of the tree attention on the tensor cores.
#include "pa_tree_mma.cuh"

namespace pa {

cudaError_t launch_tree_mma_bf16(const TreeParams& p, int group, int page_size,
                                 cudaStream_t stream, bool use_pdl) {
  switch (page_size) {
    case 16: return tree::launch_one<16>(p, group, stream, use_pdl);
    case 32: return tree::launch_one<32>(p, group, stream, use_pdl);
    case 64: return tree::launch_one<64>(p, group, stream, use_pdl);
    case 128: return tree::launch_one<128>(p, group, stream, use_pdl);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
