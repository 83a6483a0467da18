// Causal attention over packed prompts.
//
//   s_ij = scale * q_i . k_j for max(0, i - W + 1) <= j <= i within the sequence
//   lse_i = ln sum_j exp s_ij,  out_i = sum_j exp(s_ij - lse_i) v_j
//
// The kernel here runs on the ordinary cores, in 32 bits, for every type, head
// size and stride, and takes what the tensor-core kernel does not: fp32, heads and
// rows that do not lie on 16 bytes, a scale that is not positive.  A unit is 64 of
// a sequence's rows of one KV head (row r = i * G + g is token i of head h * G + g,
// so that the heads that share keys share the tiles of them).  Tiles of 64
// positions in shared memory, products of 4 x 4 scores and 4 x D / 16 outputs a
// thread, one pass with the running maximum and sum of the softmax.  The work is
// 128 operations a byte and more: the cores' rate bounds it.
#include <type_traits>

#include "sv_prompt.cuh"

namespace sv {
namespace {

constexpr int kPrThreads = 256;
constexpr int kPrRows = 64, kPrKeys = 64;
constexpr int kPrMaxD = 256;
constexpr int kPrP = kPrKeys + 4;                // row stride of the weights
constexpr uint32_t kPrMasked = 0x80000000u;      // weight of a masked position: -0

inline int padded(int D) { return (D + 3) / 4 * 4; }

// [rows][D] of T into shared memory rows of `stride` floats; rows from `live` on
// and columns from D on are zeros.  row(r): where row r begins.
template <class T, class F>
__device__ __forceinline__ void load_rows(const PromptArgs& A, float* dst, int stride, int live,
                                          bool vec, F row) {
  const int per = (A.D + 3) / 4;
  for (int i = threadIdx.x; i < 64 * per; i += kPrThreads) {
    const int r = i / per, d = (i - r * per) * 4;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < live) {
      const T* p = row(r) + d;
      if (vec) {
        if constexpr (sizeof(T) == 4) {
          const float4 w = *reinterpret_cast<const float4*>(p);
          x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(p);
          const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = to_float<T>(e[c]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (d + c < A.D) x[c] = to_float<T>(p[c]);
      }
    }
    *reinterpret_cast<float4*>(dst + r * stride + d) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// NJ: 64-column pieces of the head.
template <class T, int NJ>
__global__ void __launch_bounds__(kPrThreads) prompt_kernel(const PromptArgs A) {
  extern __shared__ __align__(16) float pr_smem[];
  __shared__ int64_t s_w[kPrThreads / 32];
  __shared__ int s_bad, s_first, s_len, s_tile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tx = tid & 15, ty = tid >> 4;
  const int stride = (A.D + 3) / 4 * 4 + 4;
  float* sq = pr_smem;
  float* sk = sq + kPrRows * stride;
  float* sv_ = sk + kPrKeys * stride;
  float* sp = sv_ + kPrKeys * stride;

  // the sequence and tile of this CTA: tiles in the order of the sequences
  if (tid == 0) {
    s_bad = 0;
    s_tile = -1;
  }
  __syncthreads();
  const int per = (A.B + kPrThreads - 1) / kPrThreads;
  const int b0 = min(A.B, tid * per), b1 = min(A.B, b0 + per);
  int64_t tiles = 0;
  for (int b = b0; b < b1; ++b) {
    int first, len;
    if (!prompt_sequence(A, b, &first, &len)) s_bad = 1;
    else tiles += (int64_t(len) * A.G + kPrRows - 1) / kPrRows;
  }
  int64_t at = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += y;
  }
  if (lane == 31) s_w[warp] = at;
  __syncthreads();
  int64_t total = 0;
  at -= tiles;
  for (int w = 0; w < kPrThreads / 32; ++w) {
    if (w < warp) at += s_w[w];
    total += s_w[w];
  }
  const bool bad = s_bad != 0;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) prompt_header(A, bad, 0);
  if (bad) {
    prompt_fail<T>(A);
    return;
  }
  // the last tiles of a sequence, which see most, begin first
  const int64_t u = total - 1 - blockIdx.x;
  if (u < 0) return;
  if (u >= at && u < at + tiles) {
    for (int b = b0; b < b1; ++b) {
      int first, len;
      prompt_sequence(A, b, &first, &len);
      const int64_t n = (int64_t(len) * A.G + kPrRows - 1) / kPrRows;
      if (u < at + n) {
        s_first = first;
        s_len = len;
        s_tile = int(u - at);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int64_t first = s_first;
  const int64_t row0 = int64_t(s_tile) * kPrRows;
  const int rows = int(min(int64_t(kPrRows), int64_t(s_len) * A.G - row0));
  const int h = blockIdx.y;
  const T* q = static_cast<const T*>(A.q);
  load_rows<T>(A, sq, stride, rows, A.q_vec, [&](int r) {
    const int64_t x = row0 + r;
    return q + (first + x / A.G) * A.q_ts + (int64_t(h) * A.G + x % A.G) * A.q_hs;
  });
  int tok[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) tok[i] = int((row0 + ty * 4 + i) / A.G);
  const int tok_first = int(row0 / A.G), tok_last = int((row0 + rows - 1) / A.G);
  const int lo = A.window > 0 ? max(0, tok_first - A.window + 1) : 0;
  const int all_lo = A.window > 0 ? max(0, tok_last - A.window + 1) : 0;
  float m[4], l[4], acc[4][NJ * 4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NJ * 4; ++c) acc[i][c] = 0.f;
  }
  const T* k = static_cast<const T*>(A.k) + first * A.k_ts + int64_t(h) * A.k_hs;
  const T* v = static_cast<const T*>(A.v) + first * A.v_ts + int64_t(h) * A.v_hs;
  for (int p0 = lo / kPrKeys * kPrKeys; p0 <= tok_last; p0 += kPrKeys) {
    const int live = min(kPrKeys, tok_last + 1 - p0);
    __syncthreads();
    load_rows<T>(A, sk, stride, live, A.k_vec,
                 [&](int r) { return k + int64_t(p0 + r) * A.k_ts; });
    load_rows<T>(A, sv_, stride, live, A.v_vec,
                 [&](int r) { return v + int64_t(p0 + r) * A.v_ts; });
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int d = 0; d < A.D; d += 4) {
      float4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<float4*>(sq + (ty * 4 + i) * stride + d);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = *reinterpret_cast<float4*>(sk + (tx + 16 * j) * stride + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(a[i].x, b[j].x,
                         fmaf(a[i].y, b[j].y,
                              fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
    }
    const bool edge = p0 < all_lo || p0 + kPrKeys > tok_first + 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bool see[4];
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = p0 + tx + 16 * j;
        see[j] = !edge || (p <= tok[i] && (A.window <= 0 || p > tok[i] - A.window));
        s[i][j] = see[j] ? s[i][j] * A.scale2 : -INFINITY;
        top = fmax_nan(top, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmax_nan(top, m[i]);
      const float sh = top == -INFINITY ? 0.f : top;
      const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - sh);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = exp2f(s[i][j] - sh);
        sum += w;
        sp[(ty * 4 + i) * kPrP + tx + 16 * j] = see[j] ? w : __uint_as_float(kPrMasked);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int c = 0; c < NJ * 4; ++c) acc[i][c] *= f;
    }
    __syncwarp();   // a row's weights are written and read by the same half of a warp
    auto products = [&](auto masked) {
#pragma unroll 2
      for (int key = 0; key < kPrKeys; ++key) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = sp[(ty * 4 + i) * kPrP + key];
#pragma unroll
        for (int c = 0; c < NJ; ++c) {
          const int d = c * 64 + tx * 4;
          if (d >= A.D) break;
          const float4 x = *reinterpret_cast<float4*>(sv_ + key * stride + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // a masked weight times an infinite value would be NaN
            if (decltype(masked)::value && __float_as_uint(w[i]) == kPrMasked) continue;
            acc[i][c * 4] = fmaf(w[i], x.x, acc[i][c * 4]);
            acc[i][c * 4 + 1] = fmaf(w[i], x.y, acc[i][c * 4 + 1]);
            acc[i][c * 4 + 2] = fmaf(w[i], x.z, acc[i][c * 4 + 2]);
            acc[i][c * 4 + 3] = fmaf(w[i], x.w, acc[i][c * 4 + 3]);
          }
        }
      }
    };
    if (edge) products(std::true_type());
    else products(std::false_type());
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (ty * 4 + i >= rows) break;
    const int64_t x = row0 + ty * 4 + i;
    const int64_t to = (first + x / A.G) * A.Hq + int64_t(h) * A.G + x % A.G;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
    for (int c = 0; c < NJ * 4; ++c) {
      const int d = c / 4 * 64 + tx * 4 + c % 4;
      if (d < A.D) static_cast<T*>(A.out)[to * A.D + d] = from_float<T>(acc[i][c] * inv);
    }
    if (tx == 0) A.lse[to] = (m[i] == -INFINITY ? 0.f : m[i] * kAttnLn2) + logf(l[i]);
  }
}

template <class T, int NJ>
cudaError_t run_nj(const PromptArgs& A, cudaStream_t s) {
  auto bytes = [](int D) {
    return sizeof(float) * ((2 * kPrKeys + kPrRows) * (padded(D) + 4) + kPrRows * kPrP);
  };
  static std::atomic<uint64_t> done{0};
  if (cudaError_t e = allow_smem(prompt_kernel<T, NJ>, bytes(kPrMaxD), done)) return e;
  const int64_t tiles = (A.rows * A.G + kPrRows - 1) / kPrRows + A.B;
  if (tiles > INT32_MAX || A.Hkv > 65535) return cudaErrorInvalidValue;
  prompt_kernel<T, NJ><<<dim3(unsigned(tiles), unsigned(A.Hkv)), kPrThreads, bytes(A.D), s>>>(A);
  return cudaGetLastError();
}

template <class T>
cudaError_t run_prompt(const PromptArgs& A, cudaStream_t s) {
  if (A.D <= 64) return run_nj<T, 1>(A, s);
  return A.D <= 128 ? run_nj<T, 2>(A, s) : run_nj<T, 4>(A, s);
}

}  // namespace

size_t prompt_workspace_bytes(int32_t, int sms) {
  return align256(sizeof(WsHeader)) + align256(sizeof(int32_t) * (1 + size_t(sms)));
}

cudaError_t launch_prompt(PromptArgs A, int dtype, void* workspace, int sms, cudaStream_t s) {
  A.hdr = static_cast<WsHeader*>(workspace);
  A.status = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(sizeof(WsHeader)));
  A.out_vec = reinterpret_cast<uintptr_t>(A.out) % 16 == 0;
  if (prompt_on_tensor_cores(A, dtype)) return launch_prompt_tc(A, dtype, sms, s);
  const size_t es = dtype == SV_F32 ? 4 : 2;
  auto fours = [&](const void* p, int64_t ts, int64_t hs) {
    return A.D % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && ts % 4 == 0 &&
           hs % 4 == 0;
  };
  A.q_vec = fours(A.q, A.q_ts, A.q_hs);
  A.k_vec = fours(A.k, A.k_ts, A.k_hs);
  A.v_vec = fours(A.v, A.v_ts, A.v_hs);
  switch (dtype) {
    case SV_F32: return run_prompt<float>(A, s);
    case SV_BF16: return run_prompt<__nv_bfloat16>(A, s);
    default: return run_prompt<__half>(A, s);
  }
}

}  // namespace sv
