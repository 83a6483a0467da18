// Shared parts of the kernels of attention over packed prompts: arguments, and
// the checks of the sequences' offsets.
#pragma once

#include "sv_attn.cuh"

namespace sv {

struct PromptArgs {
  const void *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;   // strides of row and head (elements)
  void* out;                                    // [rows, Hq, D]
  float* lse;                                   // [rows, Hq]
  const int32_t* offsets;                       // [B + 1]
  int32_t B, Hq, Hkv, G, D, window;
  int64_t rows;
  float scale2;                                 // scale * log2(e)
  int32_t q_vec, k_vec, v_vec;                  // four elements at a time (ordinary cores)
  int32_t out_vec;                              // 16-byte aligned output (tensor cores)
  int32_t test_expire;                          // as in AttnArgs
  int32_t* status;                              // [1 + CTAs]: the batch's, then each CTA's
  WsHeader* hdr;
};

#ifdef __CUDACC__

// Row b of the offsets: first row and length of sequence b, false if it is no
// piece of the rows.
__device__ __forceinline__ bool prompt_sequence(const PromptArgs& A, int b, int* first,
                                                int* length) {
  const int lo = __ldg(A.offsets + b), hi = __ldg(A.offsets + b + 1);
  *first = lo;
  *length = hi - lo;
  return lo >= 0 && hi >= lo && hi <= A.rows;
}

// The header of a call whose sequences are `bad` or not, written by one thread.
__device__ __forceinline__ void prompt_header(const PromptArgs& A, bool bad, int ctas) {
  A.hdr->err_code = kStatusList;
  A.hdr->err_row = 0;
  A.hdr->err_req = 1;
  A.hdr->n_active = 1 + ctas;
  A.status[0] = bad ? -SV_ERR_DATA_ROWS : INT32_MAX;
}

// A batch whose sequences cannot be told apart: every output is NaN.
template <class T>
__device__ __noinline__ void prompt_fail(const PromptArgs& A) {
  const float nan = __int_as_float(0x7fc00000);
  const int64_t n = A.rows * A.Hq, at = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x,
                step = int64_t(gridDim.x) * gridDim.y * blockDim.x;
  for (int64_t i = at + threadIdx.x; i < n; i += step) {
    A.lse[i] = nan;
    T* o = static_cast<T*>(A.out) + i * A.D;
    for (int d = 0; d < A.D; ++d) o[d] = from_float<T>(nan);
  }
}

#endif  // __CUDACC__

// The tensor-core kernel's share of a call, and whether it takes one.
bool prompt_on_tensor_cores(const PromptArgs& A, int dtype);
cudaError_t launch_prompt_tc(const PromptArgs& A, int dtype, int sms, cudaStream_t s);

}  // namespace sv
