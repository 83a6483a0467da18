// Attention of a chain of drafts, or of one token, on the tensor cores.
#include "sv_attn_tc_kernel.cuh"

namespace sv {

cudaError_t launch_attn_tc(const AttnArgs& A, int dtype, cudaStream_t s) {
  return run_type<false>(A, dtype, s);
}

}  // namespace sv
