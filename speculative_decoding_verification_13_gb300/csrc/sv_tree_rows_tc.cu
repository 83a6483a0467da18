// Attention of trees of drafts with many rows a KV head on the tensor cores.
#include "sv_row_tiles_tc.cuh"

namespace sv {
namespace {

template <class T, int D, bool PART>
cudaError_t run(const AttnArgs& A, cudaStream_t s) {
  using C = PtShape<D>;
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(row_tiles_tc_kernel<T, D, PART, AttnArgs>, C::kSmem, configured))
    return e;
  const bool bf16 = Bits<T>::kFmt != 0;
  AttnArgs B = A;
  B.box_rows = box_rows(A.S, C::TN, D, 32);
  CUtensorMap q, kv;
  if (!heads_map(&q, A.q, bf16, A.D, A.Hq, A.Rt, A.q_ts, A.q_hs, A.G, kM / A.G) ||
      !rows_map(&kv, B, bf16))
    return cudaErrorInvalidValue;
  row_tiles_tc_kernel<T, D, PART, AttnArgs>
      <<<unsigned(A.ctas), kPtThreads, C::kSmem, s>>>(q, kv, kv, B);
  return cudaGetLastError();
}

template <class T>
cudaError_t run_dim(const AttnArgs& A, cudaStream_t s) {
  if (A.D == 64) return run<T, 64, false>(A, s);
  return A.D == 128 ? run<T, 128, false>(A, s) : run<T, 128, true>(A, s);
}

}  // namespace

cudaError_t launch_tree_rows_tc(const AttnArgs& A, int dtype, cudaStream_t s) {
  return dtype == SV_BF16 ? run_dim<__nv_bfloat16>(A, s) : run_dim<__half>(A, s);
}

}  // namespace sv
