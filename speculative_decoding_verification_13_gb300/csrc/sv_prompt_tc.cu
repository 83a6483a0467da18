// Causal attention over packed prompts on the tensor cores.
#include "sv_row_tiles_tc.cuh"

namespace sv {
namespace {

template <class T, int D, bool PART>
cudaError_t run(const PromptArgs& A, int sms, cudaStream_t s) {
  using C = PtShape<D>;
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(row_tiles_tc_kernel<T, D, PART, PromptArgs>, C::kSmem, configured))
    return e;
  const bool bf16 = Bits<T>::kFmt != 0;
  CUtensorMap q, k, v;
  if (!heads_map(&q, A.q, bf16, A.D, A.Hq, A.rows, A.q_ts, A.q_hs, A.G, kM / A.G) ||
      !heads_map(&k, A.k, bf16, A.D, A.Hkv, A.rows, A.k_ts, A.k_hs, 1, C::TN) ||
      !heads_map(&v, A.v, bf16, A.D, A.Hkv, A.rows, A.v_ts, A.v_hs, 1, C::TN))
    return cudaErrorInvalidValue;
  row_tiles_tc_kernel<T, D, PART, PromptArgs>
      <<<unsigned(sms), kPtThreads, C::kSmem, s>>>(q, k, v, A);
  return cudaGetLastError();
}

template <class T>
cudaError_t run_dim(const PromptArgs& A, int sms, cudaStream_t s) {
  if (A.D <= 64) return A.D == 64 ? run<T, 64, false>(A, sms, s) : run<T, 64, true>(A, sms, s);
  if (A.D <= 128) return A.D == 128 ? run<T, 128, false>(A, sms, s) : run<T, 128, true>(A, sms, s);
  return A.D == 256 ? run<T, 256, false>(A, sms, s) : run<T, 256, true>(A, sms, s);
}

}  // namespace

// Types, heads and addresses that the copy engine and the products take.  The
// largest score is found before the scaling, so the scale has to be positive.
bool prompt_on_tensor_cores(const PromptArgs& A, int dtype) {
  auto boxes = [&](const void* p, int64_t ts, int64_t hs, int heads) {
    auto stride = [](int64_t x) { return x > 0 && x % 8 == 0 && x < (int64_t(1) << 38); };
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (A.rows == 1 || stride(ts)) &&
           (heads == 1 || stride(hs));
  };
  return dtype != SV_F32 && A.D % 8 == 0 && A.D <= 256 && A.G <= kM && A.scale2 > 0.0f &&
         boxes(A.q, A.q_ts, A.q_hs, A.Hq) && boxes(A.k, A.k_ts, A.k_hs, A.Hkv) &&
         boxes(A.v, A.v_ts, A.v_hs, A.Hkv);
}

cudaError_t launch_prompt_tc(const PromptArgs& A, int dtype, int sms, cudaStream_t s) {
  return dtype == SV_BF16 ? run_dim<__nv_bfloat16>(A, sms, s) : run_dim<__half>(A, sms, s);
}

}  // namespace sv
