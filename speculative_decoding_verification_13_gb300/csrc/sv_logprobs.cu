// Log probabilities of given tokens, entropy and the most likely alternatives
// of logit rows, and the gradient of the first two.
//
// With z_y = x_y / T, m = max_y x_y and S = sum_y exp((x_y - m) / T):
//   logsum = ln S                      log p_y = (x_y - m) / T - logsum
//   H = logsum - (1/S) sum_y exp((x_y - m) / T) (x_y - m) / T
// and for a loss with gradients g_l of log p_t and g_h of H:
//   dL/dx_y = (1/T) (g_l (1[y = t] - p_y) - g_h p_y (log p_y + H)).
//
// Forward: one CTA per row, one pass over it (HBM-bound).  Every thread keeps
// a running maximum m, sum s and weighted sum t = sum e^y y, rescaled when its
// maximum grows; a group of four 16-byte vectors is loaded ahead and its
// maximum decides whether to rescale.  (x - m) is taken before the scaling, so
// that a row of the type's lowest value is a uniform row.
//
// Alternatives without keeping candidates during the pass: each thread
// remembers the maximum of each quarter of its elements (a cell).  Every one
// of the 8 warps holds ceil(n / 8) cells at or above its ceil(n/8)-th largest
// lane maximum, so the smallest of those 8 values bounds the n-th largest
// element from below; only cells that reach it are read again (about a
// twentieth of the row on random logits, most of it from L2), and the
// elements that reach it are ranked by (logit, index).  Rows where more than
// kCandCap elements reach the bound (long ties) are scanned once more by the
// warps, each keeping its 32 best in order.
#include <cuda_bf16.h>

#include "sv_internal.cuh"

namespace sv {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;    // vectors in flight per thread
constexpr int kLpSegs = 4;      // cells per thread
constexpr int kCandCap = 512;   // elements that may reach the bound
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFloor2 = -1000.0f;  // exponents below 2^-1000 are zero either way

struct LpArgs {
  const void* x;
  int64_t rows, stride;
  int32_t V, n_top;
  const int32_t* tokens;      // may be null
  const float* temperature;   // may be null
  float *logprob, *entropy, *mx, *logsum;
  int32_t* top_tok;
  float* top_lp;
  int32_t* status;            // [rows]
  WsHeader* hdr;
};

template <class T> struct Elem;
template <> struct Elem<float> {
  static constexpr int VE = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  __device__ static float load(const float* p) { return *p; }
  __device__ static void store(float* p, float v) { *p = v; }
  __device__ static void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
  __device__ static float vmax(const uint4& v) {
    return fmax_nan(fmax_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                    fmax_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
};
template <> struct Elem<__nv_bfloat16> {
  static constexpr int VE = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ static float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  __device__ static void unpack(const uint4& v, float (&x)[8]) {
    x[0] = bf16_lo(v.x);
    x[1] = bf16_hi(v.x);
    x[2] = bf16_lo(v.y);
    x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z);
    x[5] = bf16_hi(v.z);
    x[6] = bf16_lo(v.w);
    x[7] = bf16_hi(v.w);
  }
  __device__ static uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static uint4 pack(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  }
  __device__ static float vmax(const uint4& v) {
    const uint32_t w = bmax2_nan(bmax2_nan(v.x, v.y), bmax2_nan(v.z, v.w));
    return fmax_nan(bf16_lo(w), bf16_hi(w));
  }
};

// A row cut into an unaligned head, 16-byte vectors and a tail.
struct RowCut {
  int head, nvec, tail;
};
template <class T>
__device__ __forceinline__ RowCut cut_row(const T* row, int V) {
  const int off = int(reinterpret_cast<uintptr_t>(row) & 15u);
  RowCut c;
  c.head = min(V, ((16 - off) & 15) / int(sizeof(T)));
  c.nvec = (V - c.head) / Elem<T>::VE;
  c.tail = V - c.head - c.nvec * Elem<T>::VE;
  return c;
}

// Log probability of one token, in natural units throughout: the type's lowest
// value times log2(e) would overflow.
__device__ __forceinline__ float token_logprob(float x, float m, float T, float logsum) {
  return (x - m) / T - logsum;
}

__device__ __forceinline__ float temperature_of(const float* temperature, int64_t r) {
  const float T = temperature ? temperature[r] : 1.0f;
  return T == 0.0f ? 1.0f : T;
}

// The inverse temperature times log2(e); NaN for a temperature that is negative,
// NaN, infinite or too small for it to be finite.  0 stands for 1.
__device__ __forceinline__ float scale_log2(const float* temperature, int64_t r) {
  const float T = temperature_of(temperature, r);
  if (!(T >= 1e-30f && T < INFINITY)) return __int_as_float(0x7fc00000);
  return kLog2e / T;
}

struct Running {
  float m = -INFINITY, s = 0.f, t = 0.f;
  // the maximum grows to at least g (NaN stays)
  __device__ __forceinline__ void raise(float g, float c2) {
    if (!(g <= m)) {
      const float mn = fmax_nan(m, g);
      if (m > -INFINITY) {
        const float d = fmaxf((m - mn) * c2, kFloor2);
        const float f = ex2_approx(d);
        t = f * fmaf(s, d, t);
        s *= f;
      }
      m = mn;
    }
  }
  __device__ __forceinline__ float shift() const { return m > -INFINITY ? m : 0.f; }
  __device__ __forceinline__ void add(float x, float sh, float c2) {
    const float y = fmaxf((x - sh) * c2, kFloor2);
    const float e = ex2_approx(y);
    s += e;
    t = fmaf(e, y, t);
  }
};

// Descending bitonic sort of one 64-bit key per lane.
__device__ __forceinline__ uint64_t warp_sort_desc(uint64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const uint64_t o = shfl_xor_u64(v, j);
      const bool keep_max = ((lane & k) == 0) == ((lane & j) == 0);
      v = keep_max ? (v > o ? v : o) : (v < o ? v : o);
    }
  return v;
}

// The 32 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t warp_merge_desc(uint64_t a, uint64_t b) {
  const int lane = threadIdx.x & 31;
  const uint32_t lo = __shfl_sync(0xffffffffu, uint32_t(b), 31 - lane);
  const uint32_t hi = __shfl_sync(0xffffffffu, uint32_t(b >> 32), 31 - lane);
  const uint64_t r = (uint64_t(hi) << 32) | lo;
  uint64_t v = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint64_t o = shfl_xor_u64(v, j);
    v = (lane & j) == 0 ? (v > o ? v : o) : (v < o ? v : o);
  }
  return v;
}

template <class T, bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LpArgs A) {
  using E = Elem<T>;
  constexpr int VE = E::VE;
  __shared__ float s_m[kLpWarps];
  __shared__ double s_s[kLpWarps], s_t[kLpWarps];
  __shared__ uint32_t s_bound[kLpWarps];
  __shared__ int s_ncell, s_ncand;
  __shared__ uint16_t s_cell[TOP ? kLpThreads * kLpSegs : 1];
  __shared__ uint64_t s_cand[TOP ? kCandCap : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x;
  if (r == 0 && tid == 0) {
    A.hdr->err_code = kStatusList;
    A.hdr->err_row = A.rows;
    A.hdr->err_req = 0;  // entries are rows
    A.hdr->n_active = 0;
  }
  const T* row = static_cast<const T*>(A.x) + r * A.stride;
  const int tok = A.tokens ? A.tokens[r] : 0;
  const float c2 = scale_log2(A.temperature, r);
  int code = 0;
  if (!(c2 == c2)) code = SV_ERR_DATA_TEMPERATURE;
  if (tok < -1 || tok >= A.V) code = SV_ERR_DATA_TOKEN;
  const float nan = __int_as_float(0x7fc00000);
  if (code || tok == -1) {  // a row without a token: nothing of it is read
    if (tid == 0) {
      A.status[r] = code;
      if (A.logprob) A.logprob[r] = nan;
      if (A.entropy) A.entropy[r] = nan;
      if (A.mx) A.mx[r] = nan;
      if (A.logsum) A.logsum[r] = nan;
    }
    if (TOP && tid < A.n_top) {
      A.top_tok[r * A.n_top + tid] = -1;
      A.top_lp[r * A.n_top + tid] = nan;
    }
    return;
  }
  float xt = 0.f;
  if (tid == 0) xt = E::load(row + tok);

  const RowCut cut = cut_row(row, A.V);
  const uint4* vec = reinterpret_cast<const uint4*>(row + cut.head);
  const int niter = (cut.nvec + kLpThreads * kLpUnroll - 1) / (kLpThreads * kLpUnroll);
  Running st;
  float cmax[kLpSegs];
#pragma unroll
  for (int q = 0; q < kLpSegs; ++q) {
    float cm = -INFINITY;
    const int it1 = niter * (q + 1) / kLpSegs;
    for (int it = niter * q / kLpSegs; it < it1; ++it) {
      uint4 v[kLpUnroll];
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) {
        const int i = (it * kLpUnroll + u) * kLpThreads + tid;
        v[u] = i < cut.nvec ? __ldcs(vec + i)
                            : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
      }
      float g = E::vmax(v[0]);
#pragma unroll
      for (int u = 1; u < kLpUnroll; ++u) g = fmax_nan(g, E::vmax(v[u]));
      if (TOP) cm = fmaxf(cm, g);
      st.raise(g, c2);
      const float sh = st.shift();
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u) {
        float x[VE];
        E::unpack(v[u], x);
#pragma unroll
        for (int e = 0; e < VE; ++e) st.add(x[e], sh, c2);
      }
    }
    cmax[q] = cm;
  }
  // head and tail: one element per thread
  const int edge = cut.head + cut.tail;
  float xe = -INFINITY;
  int ie = 0;
  if (tid < edge) {
    ie = tid < cut.head ? tid : A.V - edge + tid;
    xe = E::load(row + ie);
    st.raise(xe, c2);
    st.add(xe, st.shift(), c2);
  }

  // ------------------------------------------------ the row's m, S and sum
  float m = st.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_m[warp] = m;
  if (TOP) {
    // this warp's share of the bound: its ceil(n / 8)-th largest lane maximum
    float lm = cmax[0];
#pragma unroll
    for (int q = 1; q < kLpSegs; ++q) lm = fmaxf(lm, cmax[q]);
    uint32_t key = uint32_t(composite_key(lm, 0) >> 32);
    uint32_t b = 0;
    for (int k = 0; k < (A.n_top + kLpWarps - 1) / kLpWarps; ++k) {
      b = __reduce_max_sync(0xffffffffu, key);
      const uint32_t who = __ballot_sync(0xffffffffu, key == b);
      if (lane == __ffs(who) - 1) key = 0;
    }
    if (lane == 0) s_bound[warp] = b;
    if (tid == 0) s_ncell = s_ncand = 0;
  }
  __syncthreads();
  m = s_m[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) m = fmax_nan(m, s_m[w]);
  {
    // a maximum that is NaN or infinite makes the row's sums meaningless: it fails below
    const float d = st.m > -INFINITY ? fmaxf((st.m - m) * c2, kFloor2) : 0.f;
    const float f = ex2_approx(d);
    float t = f * fmaf(st.s, d, st.t), s = f * st.s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if (lane == 0) {
      s_s[warp] = s;
      s_t[warp] = t;
    }
  }
  __syncthreads();
  double S = 0.0, W = 0.0;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    S += s_s[w];
    W += s_t[w];
  }
  const bool bad = !(m > -INFINITY && m < INFINITY);
  const float temp = temperature_of(A.temperature, r);
  const float logsum = bad ? nan : logf(float(S));
  if (tid == 0) {
    A.status[r] = bad ? SV_ERR_DATA_LOGIT : 0;
    if (A.logprob)
      A.logprob[r] = bad || !A.tokens ? nan : token_logprob(xt, m, temp, logsum);
    if (A.entropy) A.entropy[r] = bad ? nan : logsum - kLn2 * float(W / S);
    if (A.mx) A.mx[r] = bad ? nan : m;
    if (A.logsum) A.logsum[r] = logsum;
  }
  if (!TOP) return;
  if (bad) {
    if (tid < A.n_top) {
      A.top_tok[r * A.n_top + tid] = -1;
      A.top_lp[r * A.n_top + tid] = nan;
    }
    return;
  }

  // ------------------------------------------------------- the alternatives
  // the bound as a value: the smallest of the warps', at least the lowest finite float
  uint32_t bk = s_bound[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) bk = min(bk, s_bound[w]);
  const float bound = fmaxf(composite_value(uint64_t(bk) << 32), -3.402823466e38f);
  auto offer = [&](float x, int i) {
    if (x >= bound) {
      const int at = atomicAdd(&s_ncand, 1);
      if (at < kCandCap) s_cand[at] = composite_key(x, uint32_t(i));
    }
  };
  if (tid < edge) offer(xe, ie);
#pragma unroll
  for (int q = 0; q < kLpSegs; ++q)
    if (cmax[q] >= bound) s_cell[atomicAdd(&s_ncell, 1)] = uint16_t(q * kLpThreads + tid);
  __syncthreads();
  const int per = (niter / kLpSegs + 1) * kLpUnroll;  // vectors per cell, at most
  const int total = s_ncell * per;
  for (int i = tid; i < total; i += kLpThreads) {
    const int cell = s_cell[i / per], j = i % per;
    const int q = cell / kLpThreads;
    const int it = niter * q / kLpSegs + j / kLpUnroll;
    if (it >= niter * (q + 1) / kLpSegs) continue;
    const int vi = (it * kLpUnroll + j % kLpUnroll) * kLpThreads + cell % kLpThreads;
    if (vi >= cut.nvec) continue;
    const uint4 v = vec[vi];
    if (!(E::vmax(v) >= bound)) continue;
    float x[VE];
    E::unpack(v, x);
#pragma unroll
    for (int e = 0; e < VE; ++e) offer(x[e], cut.head + vi * VE + e);
  }
  __syncthreads();
  int n = s_ncand;
  if (n > kCandCap) {
    // long ties at the bound: every warp keeps the 32 best of its share in order
    __syncthreads();
    uint64_t list = 0;
    auto visit = [&](uint64_t key) {
      const uint64_t last = (uint64_t(__shfl_sync(0xffffffffu, uint32_t(list >> 32), 31)) << 32) |
                            __shfl_sync(0xffffffffu, uint32_t(list), 31);
      if (key <= last) key = 0;
      if (__any_sync(0xffffffffu, key != 0))
        list = warp_merge_desc(list, warp_sort_desc(key));
    };
    for (int i0 = warp * 32; i0 < cut.nvec; i0 += kLpThreads) {
      const int i = i0 + lane;
      const uint4 v = i < cut.nvec
                          ? vec[i]
                          : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
      float x[VE];
      E::unpack(v, x);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        visit(x[e] >= bound ? composite_key(x[e], uint32_t(cut.head + i * VE + e)) : 0);
    }
    if (warp == 0)  // head and tail hold at most 14 elements: warp 0's lanes have them
      visit(tid < edge && xe >= bound ? composite_key(xe, uint32_t(ie)) : 0);
    s_cand[tid] = list;
    n = kLpThreads;
    __syncthreads();
  }
  // rank by counting: keys are distinct (0 stands for none)
  for (int c = tid; c < n; c += kLpThreads) {
    const uint64_t key = s_cand[c];
    if (!key) continue;
    int rank = 0;
    for (int k = 0; k < n; ++k) rank += s_cand[k] > key;
    if (rank < A.n_top) {
      A.top_tok[r * A.n_top + rank] = composite_index(key);
      A.top_lp[r * A.n_top + rank] = token_logprob(composite_value(key), m, temp, logsum);
    }
  }
  // fewer finite logits than alternatives asked for
  if (tid == 0) s_ncell = 0;
  __syncthreads();
  for (int c = tid; c < n; c += kLpThreads)
    if (s_cand[c]) atomicAdd(&s_ncell, 1);
  __syncthreads();
  if (tid < A.n_top && tid >= s_ncell) {
    A.top_tok[r * A.n_top + tid] = -1;
    A.top_lp[r * A.n_top + tid] = -INFINITY;
  }
}

// ---------------------------------------------------------------- gradient
constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 4;

struct LpGradArgs {
  const void* x;
  void* out;
  int64_t rows, stride, out_stride;
  int32_t V;
  int32_t chunks;             // blocks per row
  const int32_t* tokens;
  const float *temperature, *mx, *logsum, *entropy, *g_lp, *g_ent;
};

// One read and one write of the row, kGradThreads * kGradUnroll vectors a
// block.  d = p (A + B log2 p) + [y = t] g_l / T with p = 2^(log2 p); p = 0
// gives 0 whatever the logit.
template <class T>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const LpGradArgs A) {
  using E = Elem<T>;
  constexpr int VE = E::VE;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / A.chunks;
  const int chunk = int(blockIdx.x % A.chunks);
  const T* row = static_cast<const T*>(A.x) + r * A.stride;
  T* out = static_cast<T*>(A.out) + r * A.out_stride;
  const int tok = A.tokens[r];
  float c2 = scale_log2(A.temperature, r);
  if (tok < -1 || tok >= A.V) c2 = __int_as_float(0x7fc00000);
  const bool off = tok == -1;
  const float m = A.mx[r], ls2 = A.logsum[r] * kLog2e;
  const float invT = c2 * kLn2;
  const float gl = A.g_lp ? A.g_lp[r] * invT : 0.f;
  const float gh = A.g_ent ? A.g_ent[r] * invT : 0.f;
  const float ca = A.g_ent ? -(gl + gh * A.entropy[r]) : -gl;
  const float cb = -gh * kLn2;
  auto one = [&](float x, int i) {
    const float y = fmaxf((x - m) * c2 - ls2, kFloor2);
    const float p = ex2_approx(y);
    float d = p * fmaf(cb, y, ca);
    if (i == tok) d += gl;
    return off ? 0.f : c2 == c2 && m == m ? d : __int_as_float(0x7fc00000);
  };
  const RowCut ci = cut_row(row, A.V);
  const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  if (!same) {  // rows of input and output lie differently in their 16 bytes
    const int per = kGradThreads * kGradUnroll * VE;
    const int end = min(A.V, (chunk + 1) * per);
    for (int i = chunk * per + tid; i < end; i += kGradThreads)
      E::store(out + i, one(E::load(row + i), i));
    return;
  }
  const uint4* vin = reinterpret_cast<const uint4*>(row + ci.head);
  uint4* vout = reinterpret_cast<uint4*>(out + ci.head);
  const int v0 = chunk * kGradThreads * kGradUnroll + tid;
  uint4 v[kGradUnroll];
#pragma unroll
  for (int u = 0; u < kGradUnroll; ++u)
    if (v0 + u * kGradThreads < ci.nvec) v[u] = __ldcs(vin + v0 + u * kGradThreads);
#pragma unroll
  for (int u = 0; u < kGradUnroll; ++u) {
    const int vi = v0 + u * kGradThreads;
    if (vi >= ci.nvec) continue;
    float x[VE];
    E::unpack(v[u], x);
#pragma unroll
    for (int e = 0; e < VE; ++e) x[e] = one(x[e], ci.head + vi * VE + e);
    __stcs(vout + vi, E::pack(x));
  }
  const int edge = ci.head + ci.tail;
  if (chunk == 0 && tid < edge) {
    const int i = tid < ci.head ? tid : A.V - edge + tid;
    E::store(out + i, one(E::load(row + i), i));
  }
}

}  // namespace

size_t logprobs_workspace_bytes(int64_t rows) {
  return align256(sizeof(WsHeader)) + align256(sizeof(int32_t) * size_t(rows > 0 ? rows : 1));
}

cudaError_t launch_logprobs(const sv_logits& x, const int32_t* tokens, const float* temperature,
                            int n_top, float* logprob, float* entropy, float* mx, float* logsum,
                            int32_t* top_tok, float* top_lp, void* workspace, cudaStream_t s) {
  LpArgs A;
  A.x = x.data;
  A.rows = x.rows;
  A.stride = x.row_stride;
  A.V = x.vocab;
  A.n_top = n_top;
  A.tokens = tokens;
  A.temperature = temperature;
  A.logprob = logprob;
  A.entropy = entropy;
  A.mx = mx;
  A.logsum = logsum;
  A.top_tok = top_tok;
  A.top_lp = top_lp;
  A.hdr = static_cast<WsHeader*>(workspace);
  A.status = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(sizeof(WsHeader)));
  const unsigned grid = unsigned(x.rows);
  if (x.dtype == SV_BF16) {
    if (n_top > 0) logprobs_kernel<__nv_bfloat16, true><<<grid, kLpThreads, 0, s>>>(A);
    else logprobs_kernel<__nv_bfloat16, false><<<grid, kLpThreads, 0, s>>>(A);
  } else {
    if (n_top > 0) logprobs_kernel<float, true><<<grid, kLpThreads, 0, s>>>(A);
    else logprobs_kernel<float, false><<<grid, kLpThreads, 0, s>>>(A);
  }
  return cudaGetLastError();
}

int64_t logprobs_grad_blocks(const sv_logits& x) {
  const int ve = x.dtype == SV_BF16 ? 8 : 4;
  const int per = kGradThreads * kGradUnroll * ve;
  return x.rows * ((int64_t(x.vocab) + per - 1) / per);
}

cudaError_t launch_logprobs_grad(const sv_logits& x, const int32_t* tokens,
                                 const float* temperature, const float* mx, const float* logsum,
                                 const float* entropy, const float* g_lp, const float* g_ent,
                                 void* out, int64_t out_stride, cudaStream_t s) {
  LpGradArgs A;
  A.x = x.data;
  A.out = out;
  A.rows = x.rows;
  A.stride = x.row_stride;
  A.out_stride = out_stride;
  A.V = x.vocab;
  A.chunks = int(logprobs_grad_blocks(x) / x.rows);
  A.tokens = tokens;
  A.temperature = temperature;
  A.mx = mx;
  A.logsum = logsum;
  A.entropy = entropy;
  A.g_lp = g_lp;
  A.g_ent = g_ent;
  const unsigned grid = unsigned(x.rows * A.chunks);
  if (x.dtype == SV_BF16) logprobs_grad_kernel<__nv_bfloat16><<<grid, kGradThreads, 0, s>>>(A);
  else logprobs_grad_kernel<float><<<grid, kGradThreads, 0, s>>>(A);
  return cudaGetLastError();
}

}  // namespace sv
