// Attention of the query tokens of a verification pass (or of one new token)
// over the paged KV cache and the speculative entries, and the accumulation of
// its weights.
//
//   s = scale * q . k, masked outside the positions the query sees
//   lse = ln sum exp s,  out = sum exp(s - lse) v,  score[p] += sum exp(s - lse)
//
// The kernels here run on the ordinary cores, in 32 bits, for every type and
// head size, and take what the tensor-core kernels do not: fp32, heads below 64 or
// of no multiple of 16, a scale that is not positive.  K and V tiles of kTn positions in shared memory, kMr rows a unit,
// one pass with the running maximum and sum of the softmax.  Positions outside
// a request's keys are zero-filled, and a masked weight takes no part in the
// product with V, so that what unused slots hold does not matter.
#include <cmath>
#include <numeric>

#include "sv_attn.cuh"

namespace sv {
namespace {

constexpr int kAtThreads = 128;
constexpr int kTn = 64;       // positions per tile
constexpr int kMr = 16;       // rows per unit
constexpr int kMaxD = 256;
constexpr int kRowsPerGroup = kMr / 2;  // score rows per thread: two threads share a key
constexpr uint32_t kMaskedBits = 0x80000000u;  // weight of a masked position: -0

template <class T>
__device__ __forceinline__ void load_rows16(const AttnArgs& A, int b, int n, int hi, int p0, int h,
                                            bool values, char* dst, int stride, int* bad) {
  // [kTn][D] of T into shared memory rows of `stride` bytes, 16 bytes a thread
  const int per = A.D * int(sizeof(T)) / 16;
  for (int i = threadIdx.x; i < kTn * per; i += kAtThreads) {
    const int key = i / per, c = i % per, p = p0 + key;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (p < hi) {
      int64_t voff;
      const char* a = attn_key(A, b, n, p, &voff);
      if (a)
        v = __ldg(reinterpret_cast<const uint4*>(a + (values ? voff : 0) +
                                                 int64_t(h) * A.D * sizeof(T)) + c);
      else
        *bad = 1;
    }
    *reinterpret_cast<uint4*>(dst + key * stride + c * 16) = v;
  }
}

// Scores of one tile: 2 threads per key, kRowsPerGroup rows each, in the log2
// domain; -inf where the row does not see the key.
template <class T>
__device__ __forceinline__ void score_tile(const AttnArgs& A, const AttnReq& R, const char* sk,
                                           int stride, const float* sq, int row0, int rows, int p0,
                                           float (&acc)[kRowsPerGroup]) {
  const int key = threadIdx.x % kTn, grp = threadIdx.x / kTn;
#pragma unroll
  for (int r = 0; r < kRowsPerGroup; ++r) acc[r] = 0.f;
  constexpr int VE = 16 / int(sizeof(T));
  for (int d = 0; d < A.D; d += VE) {
    const uint4 raw = *reinterpret_cast<const uint4*>(sk + key * stride + d * sizeof(T));
    const T* kv = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float kf = to_float<T>(kv[e]);
#pragma unroll
      for (int r = 0; r < kRowsPerGroup; ++r)
        acc[r] = fmaf(sq[(grp * kRowsPerGroup + r) * A.D + d + e], kf, acc[r]);
    }
  }
  const int p = p0 + key;
#pragma unroll
  for (int r = 0; r < kRowsPerGroup; ++r) {
    const int row = grp * kRowsPerGroup + r;
    const int at = R.at0 + (row0 + row) / A.G;
    const bool see = row < rows && p <= at && p < R.hi && (A.window <= 0 || p > at - A.window);
    acc[r] = see ? acc[r] * A.scale2 : -INFINITY;
  }
}

template <class T>
__device__ __forceinline__ void load_q(const AttnArgs& A, int t_off, int h, int row0, int rows,
                                       float* sq) {
  const T* q = static_cast<const T*>(A.q);
  for (int i = threadIdx.x; i < kMr * A.D; i += kAtThreads) {
    const int r = i / A.D, d = i % A.D, row = row0 + r;
    float v = 0.f;
    if (r < rows)
      v = to_float<T>(q[int64_t(t_off + row / A.G) * A.q_ts +
                        int64_t(h * A.G + row % A.G) * A.q_hs + d]);
    sq[i] = v;
  }
}

template <class T>
__global__ void __launch_bounds__(kAtThreads) attn_kernel(const AttnArgs A) {
  extern __shared__ __align__(16) char at_smem[];
  const int stride = A.D * int(sizeof(T)) + 16;
  char* sk = at_smem;
  char* sv_ = sk + kTn * stride;
  float* sq = reinterpret_cast<float*>(sv_ + kTn * stride);  // [kMr][D]
  float* sp = sq + kMr * A.D;                                 // [kMr][kTn]
  float* s_m = sp + kMr * kTn;
  float* s_l = s_m + kMr;
  float* s_f = s_l + kMr;
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnPlan P = attn_plan<kTn, kMr, false, kAtThreads>(A);
  int first_bad = INT32_MAX;
  if (tid == 0) A.split[blockIdx.x].valid = 0;
  if (P.code) {
    if (tid == 0) A.status[A.B + blockIdx.x] = INT32_MAX;
    fail_all<T>(A);
    return;
  }
  int b = P.b, t_off = P.t_off;
  int64_t base = P.base;
  AttnReq R = attn_request<kTn, kMr, false>(A, b);
  for (int64_t pos = P.start; pos < P.end;) {
    int64_t nt = attn_tiles<kTn, kMr, false>(A, R);
    while (pos >= base + nt) {
      base += nt;
      t_off += R.k + 1;
      R = attn_request<kTn, kMr, false>(A, ++b);
      nt = attn_tiles<kTn, kMr, false>(A, R);
    }
    const int64_t local = pos - base;
    const int unit = int(local / R.ntiles), first = int(local % R.ntiles);
    const int64_t left = P.end - pos;
    const int count = int(left < R.ntiles - first ? left : R.ntiles - first);
    const int h = unit / R.mtiles, row0 = (unit % R.mtiles) * kMr;
    const int rows = min(kMr, (R.k + 1) * A.G - row0);
    __syncthreads();
    if (tid == 0) s_bad = R.code != 0;
    load_q<T>(A, t_off, h, row0, rows, sq);
    if (tid < kMr) {
      s_m[tid] = -INFINITY;
      s_l[tid] = 0.f;
    }
    float acc[kMaxD / kAtThreads][kMr];
#pragma unroll
    for (int c = 0; c < kMaxD / kAtThreads; ++c)
#pragma unroll
      for (int r = 0; r < kMr; ++r) acc[c][r] = 0.f;
    const int hi = R.code ? 0 : R.hi;
    for (int t = 0; t < count; ++t) {
      const int p0 = (R.tile0 + first + t) * kTn;
      __syncthreads();
      load_rows16<T>(A, b, R.n, hi, p0, h, false, sk, stride, &s_bad);
      load_rows16<T>(A, b, R.n, hi, p0, h, true, sv_, stride, &s_bad);
      __syncthreads();
      {
        float s[kRowsPerGroup];
        score_tile<T>(A, R, sk, stride, sq, row0, rows, p0, s);
        const int key = tid % kTn, grp = tid / kTn;
#pragma unroll
        for (int r = 0; r < kRowsPerGroup; ++r) sp[(grp * kRowsPerGroup + r) * kTn + key] = s[r];
      }
      __syncthreads();
      for (int r = warp; r < kMr; r += kAtThreads / 32) {
        const float s0 = sp[r * kTn + lane], s1 = sp[r * kTn + lane + 32];
        float m = fmax_nan(s0, s1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float old = s_m[r];
        m = fmax_nan(m, old);
        const float sh = m == -INFINITY ? 0.f : m;
        const float p0v = exp2f(s0 - sh), p1v = exp2f(s1 - sh);
        float l = p0v + p1v;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        // a masked score is exactly -inf; so is that of an infinite product,
        // whose weight is 0 as well
        sp[r * kTn + lane] = s0 == -INFINITY ? __uint_as_float(kMaskedBits) : p0v;
        sp[r * kTn + lane + 32] = s1 == -INFINITY ? __uint_as_float(kMaskedBits) : p1v;
        __syncwarp();
        if (lane == 0) {
          const float f = old == -INFINITY ? 0.f : exp2f(old - sh);
          s_f[r] = f;
          s_l[r] = s_l[r] * f + l;
          s_m[r] = m;
        }
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kMaxD / kAtThreads; ++c) {
        const int d = c * kAtThreads + tid;
        if (d >= A.D) break;
#pragma unroll
        for (int r = 0; r < kMr; ++r) acc[c][r] *= s_f[r];
        for (int key = 0; key < kTn; ++key) {
          const float v = to_float<T>(*reinterpret_cast<const T*>(sv_ + key * stride + d * sizeof(T)));
#pragma unroll
          for (int r = 0; r < kMr; ++r) {
            const float p = sp[r * kTn + key];
            if (__float_as_uint(p) != kMaskedBits) acc[c][r] = fmaf(p, v, acc[c][r]);
          }
        }
      }
    }
    __syncthreads();
    const bool bad = s_bad != 0;
    if (bad && first_bad == INT32_MAX && !R.code) first_bad = b;
    const float nan = __int_as_float(0x7fc00000);
    const bool whole = first == 0 && count == R.ntiles;
    const int slot = first == 0 ? 1 : 0;
    const int64_t pbase = (int64_t(blockIdx.x) * 2 + slot) * kMr;
#pragma unroll
    for (int c = 0; c < kMaxD / kAtThreads; ++c) {
      const int d = c * kAtThreads + tid;
      if (d >= A.D) break;
#pragma unroll
      for (int r = 0; r < kMr; ++r) {
        if (r >= rows) break;
        if (whole) {
          const int row = row0 + r;
          T* o = static_cast<T*>(A.out) + int64_t(t_off + row / A.G) * A.o_ts +
                 int64_t(h * A.G + row % A.G) * A.o_hs;
          const float l = s_l[r];
          o[d] = from_float<T>(bad ? nan : l == 0.f ? 0.f : acc[c][r] / l);
        } else {
          A.part_o[(pbase + r) * A.D + d] = acc[c][r];
        }
      }
    }
    if (tid < rows) {
      if (whole) {
        const int row = row0 + tid;
        A.lse[int64_t(t_off + row / A.G) * A.Hq + h * A.G + row % A.G] =
            bad ? nan : (s_m[tid] == -INFINITY ? 0.f : s_m[tid] * kAttnLn2) + logf(s_l[tid]);
      } else {
        A.part_ml[pbase + tid] = make_float2(bad ? nan : s_m[tid], s_l[tid]);
      }
    }
    if (!whole && first == 0 && tid == 0) {
      AttnSplit& sp_ = A.split[blockIdx.x];
      sp_.last = attn_owner(A, P, pos + R.ntiles - 1);
      sp_.t_off = t_off;
      sp_.h = h;
      sp_.row0 = row0;
      sp_.rows = rows;
      sp_.valid = 1;
    }
    pos += count;
  }
  if (tid == 0) A.status[A.B + blockIdx.x] = first_bad;
}

// Joins the partials of the unit that CTA blockIdx.x began and later ones
// continued, in order of position.  A warp has a row; where a unit lies in many
// parts, a long context with few rows, the block's warps have a share of one row's
// parts each.  Every lane finds the factor of a part, and the loads of eight
// parts are under way at once: the time is that of a few dependent loads.  36000
// positions, 4 heads of 256 in 38 parts each: the call 100 -> 43 us against one
// warp that takes part after part.
constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinSplit = 16;  // blocks per unit
constexpr int kJoinShare = 8;   // parts from which on the warps share a row
constexpr int kJoinAhead = 8;

template <class T, int MR>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs A) {
  constexpr int kVecs = kMaxD / 4 / 32;   // 16-byte vectors a lane
  __shared__ float4 s_acc[kJoinWarps][kMaxD / 4];
  __shared__ float s_l[kJoinWarps];
  pdl_wait();
  const int c0 = blockIdx.x;
  const AttnSplit u = A.split[c0];
  if (!u.valid) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nseg = (u.last - c0) / A.hg + 1, nvec = A.D / 4;
  const bool share = nseg > kJoinShare;
  const int first = share ? nseg * warp / kJoinWarps : 0;
  const int end = share ? nseg * (warp + 1) / kJoinWarps : nseg;
  for (int r = share ? blockIdx.y : blockIdx.y * kJoinWarps + warp; r < u.rows;
       r += share ? kJoinSplit : kJoinSplit * kJoinWarps) {
    auto slot = [&](int s) { return (int64_t(c0 + s * A.hg) * 2 + (s == 0 ? 1 : 0)) * MR + r; };
    float m = -INFINITY;
    for (int s = lane; s < nseg; s += 32) m = fmax_nan(m, A.part_ml[slot(s)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float sh = m == -INFINITY ? 0.f : m;
    float4 acc[kVecs];
    float l = 0.f;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = first; s0 < end; s0 += 32) {
      const int parts = min(32, end - s0);
      float f = 0.f;   // 0: this part saw nothing
      if (lane < parts) {
        const float2 ml = A.part_ml[slot(s0 + lane)];
        f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - sh);
        l = fmaf(ml.y, f, l);
      }
      for (int j0 = 0; j0 < parts; j0 += kJoinAhead) {
        float4 v[kJoinAhead][kVecs];
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
          const float4* po =
              reinterpret_cast<const float4*>(A.part_o + slot(s0 + min(j0 + j, parts - 1)) * A.D);
#pragma unroll
          for (int c = 0; c < kVecs; ++c)
            v[j][c] = c * 32 + lane < nvec ? po[c * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
          const float fj = __shfl_sync(0xffffffffu, f, j0 + j);
          if (j0 + j >= parts) break;
#pragma unroll
          for (int c = 0; c < kVecs; ++c) {
            acc[c].x = fmaf(v[j][c].x, fj, acc[c].x);
            acc[c].y = fmaf(v[j][c].y, fj, acc[c].y);
            acc[c].z = fmaf(v[j][c].z, fj, acc[c].z);
            acc[c].w = fmaf(v[j][c].w, fj, acc[c].w);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (share) {   // the shares in order
#pragma unroll
      for (int c = 0; c < kVecs; ++c) s_acc[warp][c * 32 + lane] = acc[c];
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) {
          l += s_l[w];
#pragma unroll
          for (int c = 0; c < kVecs; ++c) {
            const float4 x = s_acc[w][c * 32 + lane];
            acc[c].x += x.x;
            acc[c].y += x.y;
            acc[c].z += x.z;
            acc[c].w += x.w;
          }
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const int row = u.row0 + r;
    const int64_t t = u.t_off + row / A.G;
    const int hq = u.h * A.G + row % A.G;
    T* o = static_cast<T*>(A.out) + t * A.o_ts + int64_t(hq) * A.o_hs;
    const bool bad = !(m == m);
    const float inv = bad ? __int_as_float(0x7fc00000) : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
      if (c * 32 + lane >= nvec) break;
      T* to = o + (c * 32 + lane) * 4;
      to[0] = from_float<T>(acc[c].x * inv);
      to[1] = from_float<T>(acc[c].y * inv);
      to[2] = from_float<T>(acc[c].z * inv);
      to[3] = from_float<T>(acc[c].w * inv);
    }
    if (lane == 0) A.lse[t * A.Hq + hq] = bad ? __int_as_float(0x7fc00000) : sh * kAttnLn2 + logf(l);
  }
}

// score[b][p] += sum over the counted tokens and all heads of exp(s - lse): a
// CTA takes whole tiles of a request's positions and walks all heads and rows
// in one order, so a score has one writer and one order of its sum.
template <class T>
__global__ void __launch_bounds__(kAtThreads) attn_weights_kernel(const AttnArgs A) {
  extern __shared__ __align__(16) char at_smem[];
  const int stride = A.D * int(sizeof(T)) + 16;
  char* sk = at_smem;
  float* sq = reinterpret_cast<float*>(sk + kTn * stride);
  float* sl = sq + kMr * A.D;      // [kMr] lse in the log2 domain
  float* sw = sl + kMr;            // [kTn] the second group's sums
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  const AttnPlan P = attn_plan<kTn, kMr, true, kAtThreads>(A);
  int first_bad = INT32_MAX;
  int b = P.b, t_off = P.t_off;
  int64_t base = P.base;
  if (P.code || P.start >= P.end) {
    if (tid == 0) A.status[A.B + blockIdx.x] = INT32_MAX;
    return;
  }
  AttnReq R = attn_request<kTn, kMr, true>(A, b);
  for (int64_t pos = P.start; pos < P.end; ++pos) {
    while (pos >= base + R.ntiles) {
      base += R.ntiles;
      t_off += R.k + 1;
      R = attn_request<kTn, kMr, true>(A, ++b);
    }
    const int p0 = (R.tile0 + int(pos - base)) * kTn;
    const int nrows = R.take * A.G;
    float w = 0.f;
    if (tid == 0) s_bad = 0;
    for (int h = 0; h < A.Hkv; ++h) {
      __syncthreads();
      load_rows16<T>(A, b, R.n, R.hi, p0, h, false, sk, stride, &s_bad);
      for (int row0 = 0; row0 < nrows; row0 += kMr) {
        const int rows = min(kMr, nrows - row0);
        __syncthreads();
        load_q<T>(A, t_off, h, row0, rows, sq);
        if (tid < rows)
          sl[tid] = A.lse[int64_t(t_off + (row0 + tid) / A.G) * A.Hq + h * A.G +
                          (row0 + tid) % A.G] * kAttnLog2e;
        __syncthreads();
        float s[kRowsPerGroup];
        score_tile<T>(A, R, sk, stride, sq, row0, rows, p0, s);
        const int grp = tid / kTn;
#pragma unroll
        for (int r = 0; r < kRowsPerGroup; ++r)
          if (s[r] > -INFINITY || s[r] != s[r]) w += exp2f(s[r] - sl[grp * kRowsPerGroup + r]);
      }
    }
    __syncthreads();
    if (tid >= kTn) sw[tid - kTn] = w;
    __syncthreads();
    if (s_bad && first_bad == INT32_MAX) first_bad = b;
    if (tid < kTn && p0 + tid < R.hi) {
      const int p = p0 + tid;
      int64_t voff;
      if (attn_key(A, b, R.n, p, &voff))
        A.out_score[int64_t(b) * A.out_stride + p] =
            A.score[int64_t(b) * A.score_stride + p] + (w + sw[tid]);
    }
    __syncthreads();
  }
  if (tid == 0) A.status[A.B + blockIdx.x] = first_bad;
}

template <class T>
size_t smem_attn(int D) {
  return size_t(2) * kTn * (D * sizeof(T) + 16) + sizeof(float) * (kMr * D + kMr * kTn + 3 * kMr);
}
template <class T>
size_t smem_weights(int D) {
  return size_t(kTn) * (D * sizeof(T) + 16) + sizeof(float) * (kMr * D + kMr + kTn);
}

template <class Kern>
cudaError_t launch_join(Kern kernel, const AttnArgs& A, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(A.ctas), kJoinSplit);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, A);
}

template <class T>
cudaError_t run_attn(const AttnArgs& A, bool weights, cudaStream_t s) {
  const size_t smem = weights ? smem_weights<T>(A.D) : smem_attn<T>(A.D);
  // the most that any head size takes
  static std::atomic<uint64_t> done_w{0}, done_a{0};
  cudaError_t e = weights ? allow_smem(attn_weights_kernel<T>, smem_weights<T>(kMaxD), done_w)
                          : allow_smem(attn_kernel<T>, smem_attn<T>(kMaxD), done_a);
  if (e != cudaSuccess) return e;
  if (weights) {
    attn_weights_kernel<T><<<A.ctas, kAtThreads, smem, s>>>(A);
    return cudaGetLastError();
  }
  attn_kernel<T><<<A.ctas, kAtThreads, smem, s>>>(A);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join(attn_join_kernel<T, kMr>, A, s);
}

constexpr int kCtasPerSm = 2;  // shared memory of the widest heads
constexpr int kTcRows = 128;   // rows a unit of the tensor-core kernel

// Heads and types that the tensor-core kernels take; they number the cache's
// entries in 32 bits.  Attention finds the largest score before the scaling, so
// the scale has to be positive there.
bool on_tensor_cores(const AttnArgs& A, int dtype, bool weights) {
  return dtype != SV_F32 && A.D >= 64 && A.D % 16 == 0 &&
         (weights || A.scale2 > 0.0f) && (A.num_pages > 0 || A.spec) &&
         A.num_pages * (A.page_bytes / A.entry_bytes) <= INT32_MAX;
}

struct AttnLayout {
  size_t status, split, ml, o, total;
};
AttnLayout attn_layout(int B, int D, int ctas, int mr) {
  AttnLayout L;
  size_t o = align256(sizeof(WsHeader));
  L.status = o;  // right behind the header, as spec_verify_get_error reads it
  o += align256(4 * (size_t(B) + size_t(ctas)));
  L.split = o;
  o += align256(sizeof(AttnSplit) * size_t(ctas));
  L.ml = o;
  o += align256(sizeof(float2) * 2 * size_t(ctas) * mr);
  L.o = o;
  o += align256(sizeof(float) * 2 * size_t(ctas) * mr * size_t(D));
  L.total = o;
  return L;
}

}  // namespace

size_t attn_workspace_bytes(int32_t B, int32_t D, int sms, bool weights) {
  const AttnLayout L = attn_layout(B, D, sms * kCtasPerSm, kMr);
  if (weights) return L.split;
  const AttnLayout T = attn_layout(B, D, sms, kTcRows);
  return L.total > T.total ? L.total : T.total;
}

cudaError_t launch_attn(AttnArgs A, int dtype, bool weights, void* workspace, int sms,
                        cudaStream_t s) {
  const bool tc = on_tensor_cores(A, dtype, weights);
  A.ctas = tc ? sms : sms * kCtasPerSm;
  A.hg = tc && !weights ? std::gcd(A.ctas, A.Hkv) : 1;
  const AttnLayout L = attn_layout(A.B, A.D, A.ctas, tc ? kTcRows : kMr);
  char* w = static_cast<char*>(workspace);
  A.hdr = reinterpret_cast<WsHeader*>(w);
  A.status = reinterpret_cast<int32_t*>(w + L.status);
  A.split = reinterpret_cast<AttnSplit*>(w + L.split);
  A.part_ml = reinterpret_cast<float2*>(w + L.ml);
  A.part_o = reinterpret_cast<float*>(w + L.o);
  if (tc) {
    auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    A.s_shift = -1;
    for (int i = 0; i < 31; ++i)
      if (A.S == 1 << i) A.s_shift = i;
    A.page_rows = int32_t(A.page_bytes / A.entry_bytes);
    A.q_vec = aligned(A.q) && A.q_ts % 8 == 0 && A.q_hs % 8 == 0;
    A.out_vec = aligned(A.out);
    if (weights) return launch_attn_weights_tc(A, dtype, s);
    const cudaError_t e = launch_attn_tc(A, dtype, s);
    if (e != cudaSuccess) return e;
    return dtype == SV_BF16 ? launch_join(attn_join_kernel<__nv_bfloat16, kTcRows>, A, s)
                            : launch_join(attn_join_kernel<__half, kTcRows>, A, s);
  }
  switch (dtype) {
    case SV_F32: return run_attn<float>(A, weights, s);
    case SV_BF16: return run_attn<__nv_bfloat16>(A, weights, s);
    default: return run_attn<__half>(A, weights, s);
  }
}

}  // namespace sv
