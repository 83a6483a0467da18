// Attention of a tree of drafts on the tensor cores.
#include "sv_attn_tc_kernel.cuh"

namespace sv {

cudaError_t launch_attn_tree_tc(const AttnArgs& A, int dtype, cudaStream_t s) {
  return run_type<true>(A, dtype, s);
}

}  // namespace sv
