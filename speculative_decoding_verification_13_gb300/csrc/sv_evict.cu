// Eviction from the paged KV cache by accumulated attention weight.
//
// A request of n cached positions and a budget m < n keeps its first `sinks`
// positions, its last `recent` ones and, of the others, the m - sinks - recent
// of the largest score (the lowest position on ties; a NaN score ranks below
// every number).  The kept positions keep their order: position kept[i] moves
// to position i in every layer, K and V, and the scores move along.
//
// Two launches.  Select: one CTA per request; the threshold score by a radix
// select over the order-preserving image of the floats (four 8-bit digits,
// histograms in shared memory), then one ordered pass that writes kept[].
// Move: HBM-bound, every kept entry is read once and written once.  A group of
// lanes owns a slice of the entry's bytes and takes the positions of its range
// in increasing order, kMoveBatch loads before their stores.  In place,
// position i is the source only of positions <= i, so a slice that is walked
// by one group in increasing order, each batch read before it is written,
// never reads a moved entry; slices share no bytes.  Out of place the range is
// cut further, since nothing read is written.
//
// Measured, bf16, 36 layers of 2 x 1024 elements, pages of 16, 4 requests of 3001
// to 9003 positions cut to 2000, into other pages: 394 us, of which the move 6.0
// TB/s.  One of 1041 positions cut to 512, 4 layers: 16 us, most of it the select's
// chain of four histograms.  In place 4 of 3601 to 9003 positions take 766 us (3.1
// TB/s) and that one 165: a group of lanes walks all positions of its slice, a chain
// of dependent rounds of eight, and the one request has 32 warps in all.  (Slices
// cut down to 128 bytes in place leave the number of threads and these times as
// they are, and cost entries of 1040 bytes 737 -> 770 us.)
// Positions a thread and round of the select: 1, 2, 4 and 8 take it 9.9, 8.7, 10.5
// and 13.4 us at 1041 positions, 20, 18, 19 and 21 at 9003, the call 50, 47 and 43
// us (1, 2, 4) at 30965: two win 1 to 2 us over four at the shorter lengths and lose
// 4 at the longest.  Adding up a warp's equal first digits by a match before the
// histogram cost 6 us there.
#include "sv_internal.cuh"

namespace sv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelEach = 2;     // positions of a thread per round
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;

struct EvictArgs {
  const char* src;
  char* dst;
  int64_t src_pages, dst_pages;
  int32_t page_size;
  int32_t planes;           // layers * 2 (K and V)
  int64_t entry_bytes;
  const int32_t *src_table, *dst_table;
  int32_t src_cols, dst_cols;
  const float* score;
  float* out_score;
  int64_t score_stride, out_stride;
  int32_t score_cols, out_cols;
  const int32_t* kv_len;
  int32_t* out_len;
  int32_t B, budget, sinks, recent;
  int32_t in_place;         // entries stay in their pages: unmoved ones are skipped
  int32_t* kept;            // [B, budget]
  int2* range;              // [B] positions to move: first, end
  int32_t* status;          // [B]
  WsHeader* hdr;
  int32_t slice_bytes;      // bytes of an entry per lane group, a power of two, 16 .. 512
  int32_t slices;           // per entry
  int32_t splits;           // of a request's range (1 in place)
};

// Order-preserving image of a score; NaN is 0, below -inf.
__device__ __forceinline__ uint32_t score_key(float v) {
  return v == v ? uint32_t(composite_key(v, 0) >> 32) : 0u;
}

__device__ __forceinline__ int warp_incl(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Exclusive block scan of two counts at once; totals in *ta, *tb.
__device__ __forceinline__ void block_scan2(int& a, int& b, int* ta, int* tb) {
  __shared__ int s_a[kSelThreads / 32], s_b[kSelThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ia = warp_incl(a), ib = warp_incl(b);
  if (lane == 31) {
    s_a[warp] = ia;
    s_b[warp] = ib;
  }
  __syncthreads();
  if (warp == 0) {
    s_a[lane] = warp_incl(s_a[lane]);
    s_b[lane] = warp_incl(s_b[lane]);
  }
  __syncthreads();
  a = ia - a + (warp ? s_a[warp - 1] : 0);
  b = ib - b + (warp ? s_b[warp - 1] : 0);
  *ta = s_a[kSelThreads / 32 - 1];
  *tb = s_b[kSelThreads / 32 - 1];
  __syncthreads();
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs A) {
  __shared__ int s_hist[256];
  __shared__ int s_bad, s_first;
  __shared__ uint32_t s_prefix;
  __shared__ int s_rank;
  const int tid = threadIdx.x, b = blockIdx.x;
  if (b == 0 && tid == 0) {
    A.hdr->err_code = kStatusList;
    A.hdr->err_row = A.B;
    A.hdr->err_req = 1;  // entries are requests
    A.hdr->n_active = 0;
  }
  const int n = A.kv_len[b];
  const int S = A.page_size;
  const int m = n < A.budget ? n : A.budget;
  int32_t* kept = A.kept + int64_t(b) * A.budget;
  if (tid == 0) {
    s_bad = 0;
    s_first = m;
  }
  __syncthreads();
  int code = 0;
  if (n < 0 || n > A.score_cols || m > A.out_cols || int64_t(n) > int64_t(A.src_cols) * S ||
      int64_t(m) > int64_t(A.dst_cols) * S) {
    code = SV_ERR_DATA_LENGTH;
  } else {
    // every page a kept position may come from or go to
    const int ps = (n + S - 1) / S, pd = (m + S - 1) / S;
    bool bad = false;
    for (int c = tid; c < ps; c += kSelThreads) {
      const int p = A.src_table[int64_t(b) * A.src_cols + c];
      bad |= p < 0 || p >= A.src_pages;
    }
    for (int c = tid; c < pd; c += kSelThreads) {
      const int p = A.dst_table[int64_t(b) * A.dst_cols + c];
      bad |= p < 0 || p >= A.dst_pages;
    }
    if (bad) s_bad = 1;
    __syncthreads();
    if (s_bad) code = SV_ERR_DATA_PAGE;
  }
  const bool same_len = A.out_len == A.kv_len;
  if (code) {
    for (int i = tid; i < A.budget; i += kSelThreads) kept[i] = -1;
    if (tid == 0) {
      A.status[b] = code;
      A.range[b] = make_int2(0, 0);
      if (!same_len) A.out_len[b] = -1;
    }
    return;
  }
  const float* score = A.score + int64_t(b) * A.score_stride;
  float* osc = A.out_score + int64_t(b) * A.out_stride;

  // ------------------------------------------------------------- the threshold
  const int lo = n > A.budget ? A.sinks : 0, hi = n > A.budget ? n - A.recent : 0;
  int need = n > A.budget ? A.budget - A.sinks - A.recent : 0;  // < hi - lo
  uint32_t thr = 0;    // keys above thr are kept, and `ties` of those equal to it
  int ties = 0;
  if (need > 0) {
    uint32_t prefix = 0;
    int rank = need;   // of the sought key among those that share the prefix, from 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i0 = lo + tid; i0 < hi; i0 += kSelEach * kSelThreads) {
        float v[kSelEach];   // loads that do not wait for one another
#pragma unroll
        for (int j = 0; j < kSelEach; ++j) v[j] = score[min(i0 + j * kSelThreads, hi - 1)];
#pragma unroll
        for (int j = 0; j < kSelEach; ++j) {
          const uint32_t k = score_key(v[j]);
          if (i0 + j * kSelThreads < hi && (k & mask) == prefix)
            atomicAdd(&s_hist[(k >> shift) & 255u], 1);
        }
      }
      __syncthreads();
      if (tid < 32) {
        // the digit in which the count from the top reaches the rank: 8 digits a lane
        int c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          c[j] = s_hist[255 - (tid * 8 + j)];
          sum += c[j];
        }
        int before = warp_incl(sum) - sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (before < rank && before + c[j] >= rank) {
            s_prefix = prefix | (uint32_t(255 - (tid * 8 + j)) << shift);
            s_rank = rank - before;
          }
          before += c[j];
        }
      }
      __syncthreads();
      prefix = s_prefix;
      rank = s_rank;
    }
    thr = prefix;
    ties = rank;
  }

  // ------------------------------------------- kept positions and their scores
  // kSelEach positions in a row a thread
  int done = 0, tied = 0;
  for (int base = 0; base < n; base += kSelEach * kSelThreads) {
    const int p0 = base + tid * kSelEach;
    float v[kSelEach];
    uint32_t above = 0, tie = 0;   // a bit a position
#pragma unroll
    for (int j = 0; j < kSelEach; ++j) v[j] = score[min(p0 + j, n - 1)];
#pragma unroll
    for (int j = 0; j < kSelEach; ++j) {
      const int p = p0 + j;
      const uint32_t k = score_key(v[j]);
      const bool inner = n > A.budget && p >= lo && p < hi;
      if (p < n && (!inner || (need > 0 && k > thr))) above |= 1u << j;
      if (p < n && inner && need > 0 && k == thr) tie |= 1u << j;
    }
    int at = __popc(above), tb = __popc(tie), ta_tot, tb_tot;
    block_scan2(at, tb, &ta_tot, &tb_tot);  // scores of this round are read by now
    const int room = max(0, ties - tied);   // ties still to keep
    int i = done + at + min(tb, room);
#pragma unroll
    for (int j = 0; j < kSelEach; ++j) {
      const bool is_tie = (tie >> j) & 1;
      if (((above >> j) & 1) || (is_tie && tb < room)) {
        kept[i] = p0 + j;
        osc[i] = v[j];
        if (i != p0 + j) atomicMin(&s_first, i);
        ++i;
      }
      tb += is_tie;
    }
    done += ta_tot + min(tb_tot, room);
    tied += min(tb_tot, room);
    __syncthreads();
  }
  for (int i = m + tid; i < A.budget; i += kSelThreads) kept[i] = -1;
  const int zero_end = min(n, A.out_cols);
  for (int i = m + tid; i < zero_end; i += kSelThreads) osc[i] = 0.f;
  __syncthreads();
  if (tid == 0) {
    A.status[b] = 0;
    A.range[b] = make_int2(A.in_place ? s_first : 0, m);
    A.out_len[b] = m;
  }
}

// grid: x = slices' groups of one request's planes, y = request, z = range split
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs A) {
  pdl_wait();
  const int b = blockIdx.y;
  const int2 rg = A.range[b];
  if (rg.x >= rg.y) return;
  const int lanes = A.slice_bytes / 16;           // lanes per slice
  const int per_block = kMoveThreads / lanes;     // slices per block
  const int64_t slice = int64_t(blockIdx.x) * per_block + threadIdx.x / lanes;
  if (slice >= int64_t(A.planes) * A.slices) return;
  const int plane = int(slice / A.slices);
  const int64_t byte =
      int64_t(slice % A.slices) * A.slice_bytes + int64_t(threadIdx.x % lanes) * 16;
  if (byte >= A.entry_bytes) return;
  const int len = rg.y - rg.x;
  const int chunk = (len + A.splits - 1) / A.splits;
  const int i0 = rg.x + int(blockIdx.z) * chunk, i1 = min(rg.y, i0 + chunk);
  const int32_t* kept = A.kept + int64_t(b) * A.budget;
  const int32_t* st = A.src_table + int64_t(b) * A.src_cols;
  const int32_t* dt = A.dst_table + int64_t(b) * A.dst_cols;
  const int S = A.page_size;
  for (int i = i0; i < i1; i += kMoveBatch) {
    uint4 v[kMoveBatch];
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j)
      if (i + j < i1) {
        const int p = kept[i + j];
        const int64_t at = (int64_t(st[p / S]) * A.planes + plane) * S + p % S;
        v[j] = __ldcs(reinterpret_cast<const uint4*>(A.src + at * A.entry_bytes + byte));
      }
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j)
      if (i + j < i1) {
        const int64_t at = (int64_t(dt[(i + j) / S]) * A.planes + plane) * S + (i + j) % S;
        *reinterpret_cast<uint4*>(A.dst + at * A.entry_bytes + byte) = v[j];
      }
  }
}

}  // namespace

size_t evict_workspace_bytes(int32_t B, int32_t budget) {
  const size_t b = size_t(B > 0 ? B : 1);
  return align256(sizeof(WsHeader)) + align256(4 * b) + align256(sizeof(int2) * b) +
         align256(4 * b * size_t(budget > 0 ? budget : 1));
}

cudaError_t launch_evict(const sv_kv_cache& src, const int32_t* src_table, int src_cols,
                         const sv_kv_cache& dst, const int32_t* dst_table, int dst_cols,
                         const float* score, int64_t score_stride, int score_cols,
                         float* out_score, int64_t out_stride, int out_cols,
                         const int32_t* kv_len, int32_t* out_len, int B, int budget, int sinks,
                         int recent, int32_t* out_kept, bool in_place, void* workspace, int sms,
                         cudaStream_t s) {
  EvictArgs A;
  A.src = static_cast<const char*>(src.data);
  A.dst = static_cast<char*>(dst.data);
  A.src_pages = src.num_pages;
  A.dst_pages = dst.num_pages;
  A.page_size = src.page_size;
  A.planes = src.n_layers * 2;
  A.entry_bytes = int64_t(src.entry_elems) * src.elem_bytes;
  A.src_table = src_table;
  A.dst_table = dst_table;
  A.src_cols = src_cols;
  A.dst_cols = dst_cols;
  A.score = score;
  A.out_score = out_score;
  A.score_stride = score_stride;
  A.out_stride = out_stride;
  A.score_cols = score_cols;
  A.out_cols = out_cols;
  A.kv_len = kv_len;
  A.out_len = out_len;
  A.B = B;
  A.budget = budget;
  A.sinks = sinks;
  A.recent = recent;
  A.in_place = in_place;
  char* w = static_cast<char*>(workspace);
  A.hdr = reinterpret_cast<WsHeader*>(w);
  size_t o = align256(sizeof(WsHeader));
  A.status = reinterpret_cast<int32_t*>(w + o);
  o += align256(4 * size_t(B));
  A.range = reinterpret_cast<int2*>(w + o);
  o += align256(sizeof(int2) * size_t(B));
  A.kept = out_kept ? out_kept : reinterpret_cast<int32_t*>(w + o);
  // slices of 512 bytes, a warp's, or of what covers a shorter entry
  const int64_t target = int64_t(sms) * (kMoveThreads / 32) * 4;  // warps
  int slice = 512;
  while (slice > 16 && slice / 2 >= A.entry_bytes) slice /= 2;
  A.slice_bytes = slice;
  A.slices = int((A.entry_bytes + slice - 1) / slice);
  const int64_t warps = int64_t(B) * A.planes * A.slices * (slice / 16) / 32 + 1;
  int64_t splits = in_place ? 1 : (4 * target + warps - 1) / warps;
  const int64_t most = (budget + kMoveBatch - 1) / kMoveBatch;
  A.splits = int(splits < most ? splits : most);
  const int per_block = kMoveThreads / (slice / 16);
  evict_select_kernel<<<B, kSelThreads, 0, s>>>(A);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(A.planes) * A.slices + per_block - 1) / per_block),
                     unsigned(B), unsigned(A.splits));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, A);
}

}  // namespace sv
