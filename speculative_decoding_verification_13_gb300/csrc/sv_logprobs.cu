// Log probabilities of given tokens, entropy and the most likely alternatives
// of logit rows, and the gradient of the first two.
//
// With z_y = x_y / T, m = max_y x_y and S = sum_y exp((x_y - m) / T):
//   logsum = ln S                      log p_y = (x_y - m) / T - logsum
//   H = logsum - (1/S) sum_y exp((x_y - m) / T) (x_y - m) / T
// and for a loss with gradients g_l of log p_t and g_h of H:
//   dL/dx_y = (1/T) (g_l (1[y = t] - p_y) - g_h p_y (log p_y + H)).
//
// Forward: one pass over a row by one CTA, or by a cluster of up to 8 where
// there are few rows (HBM-bound).  Every thread keeps a running maximum m, sum s
// and weighted sum t = sum e^y y, rescaled when its maximum grows; the row
// comes through a ring of 32 KB copies, and the maximum of a thread's eight
// 16-byte vectors of a round decides whether to rescale.  What bounds the pass
// beside HBM is the issue of instructions, so two elements share an instruction
// wherever the type allows: y = x c - m c (in
// log2 units) is one packed fma, the rounding of m c being taken out of the sums
// at the end.  That form has no room for -inf (0 times -inf) and none for
// products that overflow: a group whose t is not a number is done again with
// (x - m) taken first and exponents bounded, and so is a row of very large
// logits; a row of the type's lowest value is then a uniform row.
// 4096 rows of 151936 in bf16: 233 us with twenty alternatives (5.3 TB/s),
// 205 us without; element by element 266 us.
//
// Alternatives without keeping candidates during the pass: each thread
// remembers the maximum of each eighth of its elements (a cell).  The 4
// (8 where n > 24) largest thread maxima of every warp are elements of the row,
// so the n-th largest of them bounds the row's n-th largest from below; only cells that
// reach it are read again (little more than n of 2048 on random logits), and the
// elements that reach it are ranked by (logit, index).  Parts where more cells
// or elements than there is room for reach the bound (long ties) are scanned
// once more by the warps, each keeping its 32 best in order.
#include <cuda_bf16.h>

#include "sv_internal.cuh"
#include "sv_tcgen05.cuh"

namespace sv {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 8;    // vectors of a thread per round
constexpr int kLpTile = kLpThreads * kLpUnroll * 16;   // bytes of a round: 32 KB
constexpr int kLpStages = 2;    // rounds in flight per CTA; three CTAs fit an SM
constexpr int kLpSegs = 8;      // cells per thread, at most
constexpr int kLpBest = 8;      // maxima of a warp that the bound is taken from
constexpr int kCellCap = 512;   // cells that may reach the bound
constexpr int kLpCluster = 8;   // CTAs per row, at most
constexpr int kCandCap = 256;   // elements that may reach the bound
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFloor2 = -1000.0f;  // exponents below 2^-1000 are zero either way

struct LpArgs {
  const void* x;
  int64_t rows, stride;
  int32_t V, n_top;
  int32_t cluster;            // CTAs per row
  const int32_t* tokens;      // may be null
  const float* temperature;   // may be null
  float *logprob, *entropy, *mx, *logsum;
  int32_t* top_tok;
  float* top_lp;
  int32_t* status;            // [rows]
  WsHeader* hdr;
  int32_t test_expire;        // 1 + the block whose wait runs out, 0 in normal use
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

// Running maximum and sums of one thread.  `exact`: sums refer to m itself and
// (x - m) comes first; otherwise they refer to mc, the float nearest to m c.
struct Running {
  float m = -INFINITY, mc = 0.f, s = 0.f, t = 0.f;
  bool exact = false;
  // the maximum grows to at least g (NaN stays)
  __device__ __forceinline__ void raise(float g, float c2) {
    if (!(g <= m)) {
      const float mn = fmax_nan(m, g), mcn = mn * c2;
      if (!exact && !(fabsf(mcn) < 16384.f)) to_exact(c2);
      if (m > -INFINITY) {
        const float d = fmaxf(exact ? (m - mn) * c2 : mc - mcn, kFloor2);
        const float f = ex2_approx(d);
        t = f * fmaf(s, d, t);
        s *= f;
      }
      m = mn;
      mc = exact ? 0.f : mcn;
    }
  }
  __device__ __forceinline__ void to_exact(float c2) {
    if (!exact && m > -INFINITY) {
      const float d = -fmaf(m, c2, -mc);   // mc - m c, below 2^-10
      const float f = exp2f(d);
      t = f * fmaf(s, d, t);
      s *= f;
    }
    exact = true;
    mc = 0.f;
  }
  __device__ __forceinline__ void add(float x, float c2) {
    const float sh = m > -INFINITY ? m : 0.f;
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

// What a CTA of a cluster finds of its part of a row.
struct LpPart {
  float m;
  double s, t;
  int expired;
};

template <bool TOP>
struct LpShared {
  uint64_t full[kLpStages], empty[kLpStages];
  uint64_t never;   // nothing arrives on it: the test of an expired wait
  double s[kLpWarps], t[kLpWarps];
  float m[kLpWarps];
  alignas(16) uint32_t best[TOP ? kLpWarps * kLpBest : 4];
  int abort, ncell, ncand;
  LpPart part[kLpCluster];                                  // rank 0: the cluster's sums
  uint64_t top[TOP ? kLpCluster * SV_LOGPROBS_TOP_MAX : 1]; // and best keys
  uint64_t cand[TOP ? kCandCap : 1];
  uint16_t cmax[TOP ? kLpSegs : 1][kLpThreads];   // cells' maxima: upper 16 bits of their images
  uint16_t cell[TOP ? kCellCap : 1];
};

// A CTA's part of one row.
template <class T>
struct RowPart {
  int64_t r;
  const T* row;
  const uint4* vec;
  RowCut cut;
  float c2;
  int first, niter;   // its rounds
  int tok, code;
  bool skip;          // a row without a token, or with a bad one: nothing of it is read
};
template <class T>
__device__ __forceinline__ RowPart<T> row_part(const LpArgs& A, int64_t r, int rank) {
  RowPart<T> P;
  P.r = r;
  P.row = static_cast<const T*>(A.x) + r * A.stride;
  P.tok = A.tokens ? A.tokens[r] : 0;
  P.c2 = scale_log2(A.temperature, r);
  P.code = 0;
  if (!(P.c2 == P.c2)) P.code = SV_ERR_DATA_TEMPERATURE;
  if (P.tok < -1 || P.tok >= A.V) P.code = SV_ERR_DATA_TOKEN;
  P.skip = P.code || P.tok == -1;
  P.cut = cut_row(P.row, A.V);
  P.vec = reinterpret_cast<const uint4*>(P.row + P.cut.head);
  const int rounds = (P.cut.nvec + kLpTile / 16 - 1) / (kLpTile / 16);
  P.first = int(int64_t(rounds) * rank / A.cluster);
  P.niter = int(int64_t(rounds) * (rank + 1) / A.cluster) - P.first;
  return P;
}

// A warp gives a slot of the ring back.  Its reads go by way of registers and the
// next copy into the slot does not, so that an arrival alone does not keep them
// in order: without the fence, and with the arrival straight behind the loads, a
// few rows in 4096 had some of their sums from the round after.
__device__ __forceinline__ void give_back(uint64_t* empty) {
  fence_async_proxy();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(empty));
}

// Barrier of the eight warps that read the row.  Lanes may come to it apart (the
// form for whole warps would then count a part of a warp as all of it).
__device__ __forceinline__ void lp_sync() {
  __syncwarp();
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kLpThreads) : "memory");
}

// The n_top best elements of a CTA's part of a row, in order, as composite keys
// at the front of s_cand; returns their number.
template <class T>
__device__ int best_of_part(const LpArgs& A, LpShared<true>& S, const RowCut& cut,
                            const uint4* vec, int first, int niter, int len, int edge, float xe,
                            int ie, uint32_t bound16) {
  using E = Elem<T>;
  constexpr int VE = E::VE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the bound as a value, at least the lowest finite float
  const float bound =
      fmaxf(composite_value(uint64_t(bound16) << 48), -3.402823466e38f);
  auto offer = [&](float x, int i) {
    if (x >= bound) {
      const int at = atomicAdd(&S.ncand, 1);
      if (at < kCandCap) S.cand[at] = composite_key(x, uint32_t(i));
    }
  };
  if (tid < edge) offer(xe, ie);
  for (int q = 0; q * len < niter; ++q)
    if (S.cmax[q][tid] >= bound16) {
      const int at = atomicAdd(&S.ncell, 1);
      if (at < kCellCap) S.cell[at] = uint16_t(q * kLpThreads + tid);
    }
  lp_sync();
  // all vectors of those cells at once, over all threads
  const int cells = S.ncell;
  if (cells <= kCellCap) {
    const int per = len * kLpUnroll;   // vectors per cell, at most
    for (int i = tid; i < cells * per; i += kLpThreads) {
      const int cell = S.cell[i / per], j = cell / kLpThreads * per + i % per;
      if (j >= niter * kLpUnroll) continue;
      const int vi = (first * kLpUnroll + j) * kLpThreads + cell % kLpThreads;
      if (vi >= cut.nvec) continue;
      const uint4 v = vec[vi];
      if (!(E::vmax(v) >= bound)) continue;
      float x[VE];
      E::unpack(v, x);
#pragma unroll
      for (int e = 0; e < VE; ++e) offer(x[e], cut.head + vi * VE + e);
    }
  }
  lp_sync();
  int n = S.ncand;
  if (n > kCandCap || cells > kCellCap) {
    // long ties at the bound: every warp keeps the 32 best of its share in order
    lp_sync();
    uint64_t list = 0;
    auto visit = [&](uint64_t key) {
      const uint64_t last = (uint64_t(__shfl_sync(0xffffffffu, uint32_t(list >> 32), 31)) << 32) |
                            __shfl_sync(0xffffffffu, uint32_t(list), 31);
      if (key <= last) key = 0;
      if (__any_sync(0xffffffffu, key != 0))
        list = warp_merge_desc(list, warp_sort_desc(key));
    };
    const int v1 = min(cut.nvec, (first + niter) * kLpThreads * kLpUnroll);
    for (int i0 = first * kLpThreads * kLpUnroll + warp * 32; i0 < v1; i0 += kLpThreads) {
      const int i = i0 + lane;
      const uint4 v = i < v1
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
    S.cand[tid] = list;
    n = kLpThreads;
    lp_sync();
  }
  // rank by counting: keys are distinct (0 stands for none)
  uint64_t mine[kCandCap / kLpThreads];
  int at[kCandCap / kLpThreads];
#pragma unroll
  for (int j = 0; j < kCandCap / kLpThreads; ++j) {
    const int c = tid + j * kLpThreads;
    mine[j] = c < n ? S.cand[c] : 0;
    at[j] = A.n_top;
    if (mine[j]) {
      at[j] = 0;
      for (int k = 0; k < n; ++k) at[j] += S.cand[k] > mine[j];
    }
  }
  if (tid == 0) S.ncell = 0;
  lp_sync();
#pragma unroll
  for (int j = 0; j < kCandCap / kLpThreads; ++j)
    if (at[j] < A.n_top) {
      S.cand[at[j]] = mine[j];
      atomicAdd(&S.ncell, 1);
    }
  lp_sync();
  return S.ncell;
}

// The address of the cluster's CTA `rank` that holds what p holds here.
template <class P>
__device__ __forceinline__ P* cluster_map(P* p, uint32_t rank) {
  P* q;
  asm("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(p), "r"(rank));
  return q;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// The eight reading warps' work on one row (their CTA's part of it).
template <class T, bool TOP>
__device__ void consume_row(const LpArgs& A, LpShared<TOP>& S, const unsigned char* lp_ring,
                            const RowPart<T>& P, int rank) {
  using E = Elem<T>;
  constexpr int VE = E::VE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = A.cluster;
  const float nan = __int_as_float(0x7fc00000);
  const int64_t r = P.r;
  const T* row = P.row;
  const RowCut cut = P.cut;
  const uint4* vec = P.vec;
  const float c2 = P.c2;
  const int first = P.first, niter = P.niter, tok = P.tok;
  float xt = 0.f;
  if (tid == 0 && rank == 0) xt = E::load(row + tok);
  Running st;
  float lm = -INFINITY;   // the thread's maximum
  const int len = (niter + kLpSegs - 1) / kLpSegs;   // rounds per cell
  const int end = first + niter;
  const uint64_t cc = pk2(c2, c2);
  const bool late = A.test_expire == int(blockIdx.x) + 1 && warp == 0 &&
                    !mbar_wait_for(smem_addr(&S.never), 0, kTestWaitNs);
  auto exact_vector = [&](const uint4& w) {
    float x[VE];
    E::unpack(w, x);
#pragma unroll 1
    for (int e = 0; e < VE; e += 4) {
      const bool high = e != 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) st.add(high ? x[(i + 4) % VE] : x[i], c2);
    }
  };
  for (int q = 0, it = first; it < end; ++q) {
    float cm = -INFINITY;
    const int it1 = min(end, it + len);
    for (; it < it1; ++it) {
      const int k = it - first, stage = k % kLpStages;
      bool there = true;
      if (late ||
          !mbar_wait_for(smem_addr(&S.full[stage]), (k / kLpStages) & 1, kWaitNs, &S.abort)) {
        *reinterpret_cast<volatile int*>(&S.abort) = 1;   // the row fails below
        there = false;
      }
      there = __all_sync(0xffffffffu, there);
      const uint4* tile = reinterpret_cast<const uint4*>(lp_ring + stage * kLpTile) + tid;
      const int left = cut.nvec - it * (kLpTile / 16);   // vectors from this round on
      if (there && left >= kLpTile / 16) {
        uint4 v[kLpUnroll];
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) v[u] = tile[u * kLpThreads];
        float g = E::vmax(v[0]);
#pragma unroll
        for (int u = 1; u < kLpUnroll; ++u) g = fmax_nan(g, E::vmax(v[u]));
        give_back(&S.empty[stage]);
        if (TOP) cm = fmaxf(cm, g);
        st.raise(g, c2);
        if (!st.exact) {
          const uint64_t sh = pk2(-st.mc, -st.mc);
          uint64_t s2 = pk2(st.s, 0.f), t2 = pk2(st.t, 0.f);
#pragma unroll
          for (int u = 0; u < kLpUnroll; ++u) {
            float x[VE];
            E::unpack(v[u], x);
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
              const uint64_t y = fma2(pk2(x[e], x[e + 1]), cc, sh);
              float y0, y1;
              upk2(y, y0, y1);
              const uint64_t w = pk2(ex2_approx(y0), ex2_approx(y1));
              s2 = add2(s2, w);
              t2 = fma2(w, y, t2);
            }
          }
          float s0, s1, t0, t1;
          upk2(s2, s0, s1);
          upk2(t2, t0, t1);
          const float t = t0 + t1;
          if (t == t) {
            st.s = s0 + s1;
            st.t = t;
            continue;
          }
          st.to_exact(c2);   // an element of probability 0, or a product out of range
        }
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) exact_vector(v[u]);
      } else {
        // the row's last round, vector by vector
        st.to_exact(c2);
#pragma unroll 1
        for (int u = 0; there && u * kLpThreads + tid < left; ++u) {
          const uint4 v = tile[u * kLpThreads];
          const float g = E::vmax(v);
          if (TOP) cm = fmaxf(cm, g);
          st.raise(g, c2);
          exact_vector(v);
        }
        // a slot whose copy has not landed is not free, and the copy warp gives up
        if (there) give_back(&S.empty[stage]);
      }
    }
    if (TOP) {
      S.cmax[q][tid] = uint16_t(composite_key(cm, 0) >> 48);
      lm = fmaxf(lm, cm);
    }
  }
  st.to_exact(c2);
  // head and tail: one element per thread, of the first CTA
  const int edge = rank == 0 ? cut.head + cut.tail : 0;
  float xe = -INFINITY;
  int ie = 0;
  if (tid < edge) {
    ie = tid < cut.head ? tid : A.V - edge + tid;
    xe = E::load(row + ie);
    st.raise(xe, c2);
    st.add(xe, c2);
  }

  // ------------------------------------------------ the row's m, S and sum
  float m = st.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) S.m[warp] = m;
  uint32_t bound16 = 0;
  if (TOP) {
    // the warp's largest thread maxima, as the upper 16 bits of their ordered images
    uint32_t key = uint32_t(composite_key(lm, 0) >> 48);
    for (int k = 0; k < kLpBest; ++k) {
      if (k >= 4 && A.n_top <= 24) break;   // 32 of them do
      const uint32_t best = __reduce_max_sync(0xffffffffu, key);
      const uint32_t who = __ballot_sync(0xffffffffu, key == best);
      if (lane == __ffs(who) - 1) key = 0;
      if (lane == 0) S.best[k * kLpWarps + warp] = best;
    }
    if (tid == 0) S.ncell = S.ncand = 0;
  }
  lp_sync();
  if (TOP) {
    // the bound: the n-th largest of those (every warp finds it for itself), the
    // least of the values that fewer than n are above
    static_assert(kLpWarps * kLpBest == 64, "two a lane");
    const uint32_t a = S.best[lane], b = A.n_top <= 24 ? 0u : S.best[lane + 32];
    int ra = 0, rb = 0;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&S.best[k]);
      ra += (o.x > a) + (o.y > a) + (o.z > a) + (o.w > a);
      rb += (o.x > b) + (o.y > b) + (o.z > b) + (o.w > b);
    }
    if (A.n_top > 24) {
#pragma unroll
      for (int k = 32; k < 64; k += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&S.best[k]);
        ra += (o.x > a) + (o.y > a) + (o.z > a) + (o.w > a);
        rb += (o.x > b) + (o.y > b) + (o.z > b) + (o.w > b);
      }
    }
    uint32_t low = ra < A.n_top ? a : 0xffffffffu;
    if (A.n_top > 24 && rb < A.n_top) low = min(low, b);
    bound16 = __reduce_min_sync(0xffffffffu, low);
  }
  m = S.m[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) m = fmax_nan(m, S.m[w]);
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
      S.s[warp] = s;
      S.t[warp] = t;
    }
  }
  lp_sync();
  double sum = 0.0, W = 0.0;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    sum += S.s[w];
    W += S.t[w];
  }
  const float temp = temperature_of(A.temperature, r);

  // ------------------------------------------------------- the alternatives
  int n = 0;   // candidates in S.cand
  if constexpr (TOP) {
    n = best_of_part<T>(A, S, cut, vec, first, niter, len, edge, xe, ie, bound16);
  }
  if (C > 1) {
    // sums and best keys of the cluster's CTAs meet in the first one's memory
    if (tid == 0) {
      LpPart* to = cluster_map(&S.part[rank], 0);
      to->m = m;
      to->s = sum;
      to->t = W;
      to->expired = *reinterpret_cast<volatile int*>(&S.abort);
    }
    if constexpr (TOP) {
      uint64_t* to = cluster_map(&S.top[rank * SV_LOGPROBS_TOP_MAX], 0);
      if (tid < SV_LOGPROBS_TOP_MAX) to[tid] = tid < n ? S.cand[tid] : 0;
    }
    cluster_sync();
    if (rank != 0) return;
    m = S.part[0].m;
    for (int k = 1; k < C; ++k) m = fmax_nan(m, S.part[k].m);
    sum = W = 0.0;
    for (int k = 0; k < C; ++k) {
      const LpPart p = S.part[k];
      if (p.expired) *reinterpret_cast<volatile int*>(&S.abort) = 1;
      if (!(p.m > -INFINITY)) continue;   // a part without a finite logit
      const double d = (double(p.m) - double(m)) * double(c2);
      const double f = exp2(d);
      sum += f * p.s;
      W += f > 0.0 ? f * (p.t + p.s * d) : 0.0;
    }
    if constexpr (TOP) {
      lp_sync();
      n = C * SV_LOGPROBS_TOP_MAX;
      if (tid < n) S.cand[tid] = S.top[tid];
      lp_sync();
    }
  }
  const bool expired = *reinterpret_cast<volatile int*>(&S.abort) != 0;
  const bool bad = expired || !(m > -INFINITY && m < INFINITY);
  const float logsum = bad ? nan : logf(float(sum));
  if (tid == 0) {
    A.status[r] = expired ? SV_ERR_TIMEOUT : bad ? SV_ERR_DATA_LOGIT : 0;
    if (A.logprob)
      A.logprob[r] = bad || !A.tokens ? nan : token_logprob(xt, m, temp, logsum);
    if (A.entropy) A.entropy[r] = bad ? nan : logsum - kLn2 * float(W / sum);
    if (A.mx) A.mx[r] = bad ? nan : m;
    if (A.logsum) A.logsum[r] = logsum;
  }
  if constexpr (TOP) {
    if (tid < A.n_top) {
      A.top_tok[r * A.n_top + tid] = -1;
      A.top_lp[r * A.n_top + tid] = bad ? nan : -INFINITY;   // what is missing stays so
    }
    lp_sync();
    if (bad) return;
    for (int c = tid; c < n; c += kLpThreads) {
      const uint64_t key = S.cand[c];
      if (!key) continue;
      // in order already where one CTA had the row
      int rank_of = c;
      if (C > 1) {
        rank_of = 0;
        for (int k = 0; k < n; ++k) rank_of += S.cand[k] > key;
      }
      if (rank_of < A.n_top) {
        A.top_tok[r * A.n_top + rank_of] = composite_index(key);
        A.top_lp[r * A.n_top + rank_of] = token_logprob(composite_value(key), m, temp, logsum);
      }
    }
  }
}

template <class T, bool TOP>
__global__ void __launch_bounds__(kLpThreads + 32, 3) logprobs_kernel(const LpArgs A) {
  __shared__ LpShared<TOP> S;
  extern __shared__ __align__(128) unsigned char lp_ring[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = A.cluster, rank = int(blockIdx.x) % C;
  if (tid == 0) {
    for (int i = 0; i < kLpStages; ++i) {
      mbar_init(smem_addr(&S.full[i]), 1);
      mbar_init(smem_addr(&S.empty[i]), kLpWarps);
    }
    mbar_init(smem_addr(&S.never), 1);
    fence_mbar_init();
    S.abort = 0;
    if (blockIdx.x == 0) {
      A.hdr->err_code = kStatusList;
      A.hdr->err_row = A.rows;
      A.hdr->err_req = 0;  // entries are rows
      A.hdr->n_active = 0;
    }
  }
  __syncthreads();
  if (C > 1) cluster_sync();   // every CTA of the cluster is there before its memory is written
  const RowPart<T> P = row_part<T>(A, blockIdx.x / C, rank);
  if (warp == kLpWarps) {
    // the row's rounds, 32 KB a copy, kLpStages ahead
    if (lane != 0 || P.skip) return;
    const uint64_t policy = l2_evict_first_policy();
    int k = 0;
    for (; k < P.niter; ++k) {
      const int s = k % kLpStages;
      if (!mbar_wait_for(smem_addr(&S.empty[s]), ((k / kLpStages) & 1) ^ 1, kWaitNs, &S.abort))
        break;
      const int v0 = (P.first + k) * (kLpTile / 16);
      const uint32_t bytes = uint32_t(min(kLpTile / 16, P.cut.nvec - v0)) * 16;
      mbar_arrive_expect_tx(smem_addr(&S.full[s]), bytes);
      bulk_load_hint(smem_addr(lp_ring) + s * kLpTile, P.vec + v0, bytes, smem_addr(&S.full[s]),
                     policy);
    }
    if (k < P.niter) *reinterpret_cast<volatile int*>(&S.abort) = 1;   // gave up
    // the last copies land before the CTA may end, whoever gave up and when
    for (int j = max(0, k - kLpStages); j < k; ++j)
      mbar_wait_for(smem_addr(&S.full[j % kLpStages]), (j / kLpStages) & 1);
    return;
  }
  if (!P.skip) {
    consume_row<T, TOP>(A, S, lp_ring, P, rank);
    return;
  }
  if (rank != 0) return;
  const float nan = __int_as_float(0x7fc00000);
  if (tid == 0) {
    A.status[P.r] = P.code;
    if (A.logprob) A.logprob[P.r] = nan;
    if (A.entropy) A.entropy[P.r] = nan;
    if (A.mx) A.mx[P.r] = nan;
    if (A.logsum) A.logsum[P.r] = nan;
  }
  if (TOP && tid < A.n_top) {
    A.top_tok[P.r * A.n_top + tid] = -1;
    A.top_lp[P.r * A.n_top + tid] = nan;
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

template <class T, bool TOP>
cudaError_t launch_rows(const cudaLaunchConfig_t& cfg, const LpArgs& A) {
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(logprobs_kernel<T, TOP>, cfg.dynamicSmemBytes, configured))
    return e;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, TOP>, A);
}

}  // namespace

size_t logprobs_workspace_bytes(int64_t rows) {
  return align256(sizeof(WsHeader)) + align256(sizeof(int32_t) * size_t(rows > 0 ? rows : 1));
}

cudaError_t launch_logprobs(const sv_logits& x, const int32_t* tokens, const float* temperature,
                            int n_top, float* logprob, float* entropy, float* mx, float* logsum,
                            int32_t* top_tok, float* top_lp, void* workspace, int sms,
                            int test_expire, cudaStream_t s) {
  LpArgs A;
  A.test_expire = test_expire;
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
  // CTAs per row: a power of two, at least a round each, while the grid stays
  // within one CTA per SM (8 rows of 32000 in fp32: one CTA a row 14 us)
  const int rounds = x.vocab / (kLpThreads * kLpUnroll * (x.dtype == SV_BF16 ? 8 : 4));
  A.cluster = 1;
  while (A.cluster < kLpCluster && A.cluster * 2 <= rounds && x.rows * A.cluster * 2 <= sms)
    A.cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(x.rows * A.cluster));
  cfg.blockDim = dim3(kLpThreads + 32);
  cfg.dynamicSmemBytes = size_t(kLpStages) * kLpTile;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(A.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = A.cluster > 1 ? 1 : 0;
  if (x.dtype == SV_BF16)
    return n_top > 0 ? launch_rows<__nv_bfloat16, true>(cfg, A)
                     : launch_rows<__nv_bfloat16, false>(cfg, A);
  return n_top > 0 ? launch_rows<float, true>(cfg, A) : launch_rows<float, false>(cfg, A);
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
