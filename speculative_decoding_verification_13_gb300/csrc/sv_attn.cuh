// Shared parts of the attention kernels over the paged KV cache: arguments,
// the addresses of keys and values, and the cut of the work into CTAs.
//
// Work.  Request b has units (KV head h, row tile mt): up to MR of its
// (k_b + 1) * G query rows that share a KV head, row r = j * G + g being query
// token j of head h * G + g.  A unit walks the key tiles of TN positions that
// its request can see.  All tiles of all units, in the order request, head,
// row tile, position, form one line that is cut evenly over the CTAs, so that
// every CTA has the same number of tiles whatever the lengths are.  A unit
// inside one CTA's piece is finished there; one that spans CTAs leaves an
// unnormalised partial (output, maximum, sum) per CTA, joined by a second
// kernel in order of position.  A CTA holds at most two partials: of the unit
// it begins in (slot 0, begun by an earlier CTA) and of the unit it ends in
// (slot 1, begun by itself).
//
// hg KV heads (a divisor of their number and of the CTAs') can have a line of
// their own each: hg neighbouring CTAs then walk the same positions of
// different heads at the same time, and the pieces of an entry that lie side by
// side in memory are read together.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_internal.cuh"

namespace sv {

// Positions of a request, at most: a tile's end, and a window's start for a token
// up to 32 positions before the first, stay within 32 bits.
constexpr int32_t kMaxPositions = INT32_MAX - 255;

struct AttnSplit {  // a unit begun by this CTA and continued by later ones
  int32_t valid, last;            // last: the CTA that ends it
  int32_t t_off, h, row0, rows;   // its rows row0 .. row0 + rows - 1 of the request
};

struct AttnArgs {
  const void* q;
  int64_t q_ts, q_hs;             // strides of token and head (elements)
  void* out;
  int64_t o_ts, o_hs;
  float* lse;                     // [Rt, Hq]
  const char* cache;              // the layer's K of page 0
  int64_t page_bytes, v_off, entry_bytes, num_pages;
  const char* spec;               // the layer's K of entry 0 of request 0, or null
  int64_t spec_req, spec_tok;     // byte strides
  int32_t slots;
  const int32_t *kv_len, *k_per_req, *table;
  int32_t S, max_pages, B, Hq, Hkv, G, D, window;
  int64_t Rt;
  float scale2;                   // scale * log2(e)
  float* part_o;                  // [CTAs, 2, MR, D]
  float2* part_ml;                // [CTAs, 2, MR]  maximum (log2 domain), sum
  AttnSplit* split;               // [CTAs]
  int32_t* status;                // [B] then one entry per CTA (first request with a bad page),
                                  // of trees then another (first request with a bad parent)
  WsHeader* hdr;
  // accumulated weights
  const int32_t* accept_len;      // may be null
  const float* score;
  float* out_score;
  int64_t score_stride, out_stride;
  int32_t score_cols;
  int32_t ctas;                   // grid of the main kernel
  int32_t hg;                     // heads with a line of their own, 1 or more
  // the tensor-core kernel
  uint32_t s_mul;                 // p / S = p * s_mul >> s_shift for 0 <= p < 2^31
  int32_t s_shift;
  int32_t box_rows;               // entries per box of the copy engine, 0: no boxes
  int32_t page_rows, layer_row;   // entries per page, entries before the layer's first
  int32_t q_vec, out_vec;         // 16-byte aligned heads
  int32_t test_expire;            // 1 + the block whose wait runs out, 0 in normal use
  // a tree of drafts
  const int32_t* parent;          // [Rt] each node's parent in its request, or null: a chain
  int32_t max_k;                  // SV_MAX_K, of a tree SV_TREE_MAX_K
};

#ifdef __CUDACC__

template <class T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <class T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

constexpr float kAttnLn2 = 0.6931471805599453f;
constexpr float kAttnLog2e = 1.4426950408889634f;

// One request as the kernels see it.
struct AttnReq {
  int n, k;        // cached positions, drafts
  int at0;         // position of query token 0: token j sits at at0 + j
  int hi;          // keys are [0, hi)
  int tile0, ntiles, mtiles;
  int take;        // query tokens counted (weights), k + 1 otherwise
  int code;        // a data error of the request, or 0
};

// WEIGHTS: the tiles are shared by all heads and rows (one unit per request),
// keys end at the last counted token, and tiles before the window are kept
// when the scores are written elsewhere.
template <int TN, int MR, bool WEIGHTS>
__device__ __forceinline__ AttnReq attn_request(const AttnArgs& A, int b) {
  AttnReq r;
  r.k = A.k_per_req[b];
  r.n = A.kv_len[b];
  r.code = 0;
  const int k = min(max(r.k, 0), A.max_k);
  if (r.k != k) r.code = SV_ERR_DATA_K;
  else if (r.n < 0 || int64_t(r.n) + k + 1 > kMaxPositions ||
           int64_t(r.n) > int64_t(A.max_pages) * A.S)
    r.code = SV_ERR_DATA_LENGTH;
  else if (A.spec && k + 1 > A.slots) r.code = SV_ERR_DATA_K;
  r.take = k + 1;
  if (WEIGHTS && A.accept_len) {
    const int L = A.accept_len[b];
    if (L > k && !r.code) r.code = SV_ERR_DATA_ACCEPT;
    r.take = L < 0 ? 0 : min(L, k) + 1;
  }
  r.at0 = A.spec ? r.n : r.n - 1 - k;
  r.hi = A.spec ? r.n + r.take : r.n;
  if (WEIGHTS && !r.code && r.hi > A.score_cols) r.code = SV_ERR_DATA_LENGTH;
  r.k = k;
  r.mtiles = WEIGHTS ? 1 : ((k + 1) * A.G + MR - 1) / MR;
  if (r.code) {  // one tile a unit, which fails its rows
    r.tile0 = 0;
    r.ntiles = WEIGHTS ? 0 : 1;
    return r;
  }
  int lo = 0;
  if (A.window > 0 && !(WEIGHTS && A.out_score != A.score)) lo = max(0, r.at0 - A.window + 1);
  r.tile0 = lo / TN;
  r.ntiles = max((r.hi + TN - 1) / TN - r.tile0, WEIGHTS ? 0 : 1);
  if (WEIGHTS && r.take == 0) r.ntiles = 0;
  return r;
}

// A node of a request's tree of drafts.  Node 0 is the last emitted token, at
// position n; a node lies one position behind its parent and sees the cache, its
// ancestors and itself, as far as the window reaches.
struct AttnNode {
  uint64_t path;   // the nodes it sees
  int at;          // its position
};
// parents: of this request's nodes; one that does not point back ends the walk
__device__ __forceinline__ AttnNode attn_node(const AttnArgs& A, const int32_t* parents, int n,
                                              int j) {
  AttnNode x{0, n};
  for (int depth = 0; depth <= SV_TREE_MAX_K; ++depth) {
    if (A.window <= 0 || depth < A.window) x.path |= 1ull << j;
    if (j == 0) break;
    const int up = parents[j];
    if (up < 0 || up >= j) break;
    j = up;
    ++x.at;
  }
  return x;
}

// Where a CTA starts, found by every CTA itself from the lengths.
struct AttnPlan {
  int64_t total;     // tiles of the whole call
  int64_t start, end;  // this CTA's
  int64_t base;      // tiles before request b
  int b, t_off;      // the request `start` lies in, query tokens before it
  int ctas;          // pieces that have tiles
  int code, code_b;  // a data error of the whole batch, and its request
};

// A request's share of the line; PAD: what each of its units adds to its tiles.
template <int TN, int MR, bool WEIGHTS, int PAD = 0>
__device__ __forceinline__ int64_t attn_tiles(const AttnArgs& A, const AttnReq& r) {
  return WEIGHTS ? int64_t(r.ntiles) : int64_t(A.Hkv / A.hg) * r.mtiles * (r.ntiles + PAD);
}

// All threads of the block call this.  CTA 0 records the requests' errors.
template <int TN, int MR, bool WEIGHTS, int THREADS, int PAD = 0>
__device__ AttnPlan attn_plan(const AttnArgs& A) {
  __shared__ int64_t s_tiles[THREADS / 32 + 1];
  __shared__ int s_rows[THREADS / 32 + 1];
  __shared__ int s_badk;
  __shared__ int64_t s_base;
  __shared__ int s_b, s_toff;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_badk = INT32_MAX;
    s_b = 0;
    s_toff = 0;
    s_base = 0;
  }
  __syncthreads();
  const int per = (A.B + THREADS - 1) / THREADS;
  const int b0 = min(A.B, tid * per), b1 = min(A.B, b0 + per);
  int64_t tiles = 0;
  int rows = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const AttnReq r = attn_request<TN, MR, WEIGHTS>(A, b);
    if (A.k_per_req[b] != r.k) atomicMin(&s_badk, b);
    if (blockIdx.x == 0) A.status[b] = r.code;
    tiles += attn_tiles<TN, MR, WEIGHTS, PAD>(A, r);
    rows += r.k + 1;
  }
  int64_t it = tiles;
  int ir = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, it, o);
    const int y = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) {
      it += x;
      ir += y;
    }
  }
  if (lane == 31) {
    s_tiles[warp] = it;
    s_rows[warp] = ir;
  }
  __syncthreads();
  int64_t wt = 0, total = 0;
  int wr = 0, total_rows = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) {
      wt += s_tiles[w];
      wr += s_rows[w];
    }
    total += s_tiles[w];
    total_rows += s_rows[w];
  }
  AttnPlan P;
  P.total = total;
  const int pieces = A.ctas / A.hg;
  P.ctas = int(total < pieces ? total : int64_t(pieces));
  const int c = blockIdx.x / A.hg;
  // total c / ctas, with short divisions where they do
  P.start = P.end = total;
  if (c < P.ctas) {
    const int64_t each = total <= INT32_MAX ? int32_t(total) / P.ctas : total / P.ctas;
    const int rest = int(total - each * P.ctas);
    P.start = each * c + rest * c / P.ctas;
    P.end = each * (c + 1) + rest * (c + 1) / P.ctas;
  }
  int64_t base = wt + it - tiles;
  int toff = wr + ir - rows;
  if (P.start < P.end && P.start >= base && P.start < base + tiles) {
    if (per == 1) {
      s_b = b0;
      s_toff = toff;
      s_base = base;
    }
#pragma unroll 1
    for (int b = b0; per > 1 && b < b1; ++b) {
      const AttnReq r = attn_request<TN, MR, WEIGHTS>(A, b);
      const int64_t t = attn_tiles<TN, MR, WEIGHTS, PAD>(A, r);
      if (P.start < base + t) {
        s_b = b;
        s_toff = toff;
        s_base = base;
        break;
      }
      base += t;
      toff += r.k + 1;
    }
  }
  __syncthreads();
  P.b = s_b;
  P.t_off = s_toff;
  P.base = s_base;
  P.code = 0;
  P.code_b = 0;
  if (s_badk != INT32_MAX) {
    P.code = SV_ERR_DATA_K;
    P.code_b = s_badk;
  } else if (total_rows != A.Rt) {
    P.code = SV_ERR_DATA_ROWS;
  }
  if (P.code && blockIdx.x == 0 && tid == 0) A.status[P.code_b] = P.code;
  if (blockIdx.x == 0 && tid == 0) {
    A.hdr->err_code = kStatusList;
    A.hdr->err_row = A.B;
    A.hdr->err_req = A.parent ? 2 : 1;   // entries are requests
    // followed by the CTAs' first bad-page requests, of trees also the first torn ones
    A.hdr->n_active = A.parent ? 2 * A.ctas : A.ctas;
  }
  return P;
}

// The CTA of this one's heads that owns tile x of the line.
__device__ __forceinline__ int attn_owner(const AttnArgs& A, const AttnPlan& P, int64_t x) {
  const int64_t y = (x + 1) * P.ctas - 1;
  const int piece = y <= INT32_MAX ? int32_t(y) / int32_t(P.total) : int(y / P.total);
  return piece * A.hg + int(blockIdx.x) % A.hg;
}

// Address of key p of request b (head 0, K), null where its page is missing.
__device__ __forceinline__ const char* attn_key(const AttnArgs& A, int b, int n, int p,
                                                int64_t* v_off) {
  if (p >= n) {
    *v_off = A.entry_bytes;
    return A.spec + int64_t(b) * A.spec_req + int64_t(p - n) * A.spec_tok;
  }
  *v_off = A.v_off;
  const int page = A.table[int64_t(b) * A.max_pages + p / A.S];
  if (page < 0 || page >= A.num_pages) return nullptr;
  return A.cache + page * A.page_bytes + int64_t(p % A.S) * A.entry_bytes;
}

template <class T>
__device__ __noinline__ void fail_all(const AttnArgs& A) {
  // a batch whose rows cannot be told apart: every output is NaN
  const float nan = __int_as_float(0x7fc00000);
  const int64_t n = A.Rt * A.Hq;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t t = i / A.Hq, hq = i % A.Hq;
    A.lse[i] = nan;
    T* o = static_cast<T*>(A.out) + t * A.o_ts + hq * A.o_hs;
    for (int d = 0; d < A.D; ++d) o[d] = from_float<T>(nan);
  }
}

#endif  // __CUDACC__

// The tensor-core kernels' share of a call (MR = 128, one CTA per SM).
cudaError_t launch_attn_tc(const AttnArgs& A, int dtype, cudaStream_t s);
cudaError_t launch_attn_tree_tc(const AttnArgs& A, int dtype, cudaStream_t s);
cudaError_t launch_tree_rows_tc(const AttnArgs& A, int dtype, cudaStream_t s);  // MR = 256
cudaError_t launch_attn_weights_tc(const AttnArgs& A, int dtype, cudaStream_t s);

}  // namespace sv
