// Pages and slots of the paged cache, kept on the GPU: block tables that follow
// the requests' lengths, the slots of a step's new tokens, and the writing of
// their keys and values.
//
// All of it is bound by latency and by HBM: nothing is computed but prefix sums
// over the requests, which every CTA forms by itself instead of waiting for a
// kernel that does.  The kernels are launched as dependents of what runs before
// them and wait for it at their beginning.  Tables and slots of 8 requests 9.8 us of
// the GPU, of 1024 with 2048 columns 17.5; 32768 rows of 8 heads of 128 in bf16, 269 MB
// read and written, 42.9 us (6.3 TB/s).
#include "sv_internal.cuh"

namespace sv {
namespace {

constexpr int kTbThreads = 256;
constexpr int kTbWarps = kTbThreads / 32;

// Exclusive scan of one value a thread over the CTA; *total gets the sum.
__device__ int64_t block_scan(int64_t v, int64_t* total) {
  __shared__ int64_t s_w[kTbWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the call before may still be read
  if (lane == 31) s_w[warp] = x;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kTbWarps; ++w) {
    if (w < warp) base += s_w[w];
    all += s_w[w];
  }
  *total = all;
  return base + x - v;
}

// ------------------------------------------------------------ block tables
// Two kernels, since a page given up by one request may be taken by another in
// the same call, in place: the first copies what stays, takes the released pages
// off the tables into a list and notes what every request releases and wants; the
// second hands pages out from the end of the free list followed by that list.
struct ReserveProblem {
  const int32_t* table;
  int32_t* out_table;
  const int32_t *held, *length;
  int32_t* out_held;
  const int32_t* free_pages;
  int32_t* out_free;
  const int32_t* free_count;
  int32_t* out_count;
  int32_t B, cols, S;
  int64_t capacity;    // entries of the free list
  bool copy_table, copy_free;
  int32_t vec;         // table rows and lists move 16 bytes at a time
  WsHeader* hdr;
  int32_t* status;     // [B], then one entry for the whole call
  int2* plan;          // [B] pages held, pages needed; of a request that fails -1, and
                       // how many entries of `released` it has that are no pages to hand out
  int32_t* count;      // free pages before the call, or -1: the call fails
  int32_t* released;   // [capacity]
};

__device__ __forceinline__ int2 reserve_request(const ReserveProblem& Q, int b, int* code) {
  const int held = Q.held[b], n = Q.length[b];
  const int need = n > 0 ? (n - 1) / Q.S + 1 : 0;
  *code = held < 0 || held > Q.cols || n < 0 || need > Q.cols ? SV_ERR_DATA_LENGTH : 0;
  return *code ? make_int2(0, 0) : make_int2(held, need);
}

constexpr int kReserveCtasPerSm = 2;

// The requests of CTA c: neighbouring ones.
__device__ __forceinline__ int chunk_start(int B, int c) {
  return int(int64_t(B) * c / gridDim.x);
}

__global__ void __launch_bounds__(kTbThreads) reserve_release_kernel(const ReserveProblem Q) {
  __shared__ int2 s_plan[kTbThreads];
  __shared__ int64_t s_first[kTbThreads];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = chunk_start(Q.B, blockIdx.x), r1 = chunk_start(Q.B, blockIdx.x + 1);
  const int n = *Q.free_count;
  // released pages of the requests before this CTA's, and of all
  int64_t mine = 0, all = 0, before, total;
#pragma unroll 4
  for (int b = tid; b < Q.B; b += kTbThreads) {
    int code;
    const int2 p = reserve_request(Q, b, &code);
    const int rel = max(p.x - p.y, 0);
    all += rel;
    if (b < r0) mine += rel;
  }
  block_scan(mine, &before);
  block_scan(all, &total);
  const bool fail = n < 0 || n + total > Q.capacity;
  if (blockIdx.x == 0 && tid == 0) {
    Q.hdr->err_code = kStatusList;
    Q.hdr->err_row = Q.B;
    Q.hdr->err_req = 1;      // entries are requests
    Q.hdr->n_active = 1;
    Q.status[Q.B] = fail ? -SV_ERR_DATA_POOL : INT32_MAX;
    *Q.count = fail ? -1 : n;
  }
  for (int c0 = r0; c0 < r1; c0 += kTbThreads) {
    const int b = c0 + tid;
    int2 p = make_int2(0, 0);
    if (b < r1) {
      int code;
      p = reserve_request(Q, b, &code);
      Q.status[b] = code;
      Q.plan[b] = code ? make_int2(-1, 0) : p;
    }
    int64_t here;
    const int64_t first = before + block_scan(max(p.x - p.y, 0), &here);
    before += here;
    s_plan[tid] = p;
    s_first[tid] = first;
    __syncthreads();
    const int rows = min(kTbThreads, r1 - c0);
    // columns given up of row i: [lo, hi)
    auto given_up = [&](int i, int* lo, int* hi) {
      *lo = s_plan[i].y;
      *hi = fail ? *lo : s_plan[i].x;
    };
    if (Q.copy_table) {
      // all rows in one run of the threads: short rows and long ones alike
      const int64_t first_row = int64_t(c0) * Q.cols;
      int lo, hi;
      if (Q.vec) {
        const int per = Q.cols / 4;
        const int4* from = reinterpret_cast<const int4*>(Q.table + first_row);
        int4* to = reinterpret_cast<int4*>(Q.out_table + first_row);
#pragma unroll 4
        for (int64_t x = tid; x < int64_t(rows) * per; x += kTbThreads) {
          const int i = int(x / per), c = int(x - int64_t(i) * per) * 4;
          int4 v = from[x];
          given_up(i, &lo, &hi);
          if (c + 3 >= lo && c < hi) {
            if (c >= lo) v.x = -1;
            if (c + 1 >= lo && c + 1 < hi) v.y = -1;
            if (c + 2 >= lo && c + 2 < hi) v.z = -1;
            if (c + 3 < hi) v.w = -1;
          }
          to[x] = v;
        }
      } else {
#pragma unroll 4
        for (int64_t x = tid; x < int64_t(rows) * Q.cols; x += kTbThreads) {
          const int i = int(x / Q.cols), c = int(x - int64_t(i) * Q.cols);
          given_up(i, &lo, &hi);
          Q.out_table[first_row + x] = c >= lo && c < hi ? -1 : Q.table[first_row + x];
        }
      }
    }
    __syncthreads();
    for (int i = warp; i < rows; i += kTbWarps) {
      const int64_t row = int64_t(c0 + i) * Q.cols;
      int lo, hi;
      given_up(i, &lo, &hi);
      bool torn = false;   // an entry is no page
      for (int c = lo + lane; c < hi; c += 32) {
        const int page = Q.table[row + c];
        Q.released[s_first[i] + c - lo] = page;
        torn |= page < 0;
      }
      torn = __any_sync(0xffffffffu, torn);
      if (!torn && Q.copy_table) continue;
      for (int c = lo + lane; c < hi; c += 32) Q.out_table[row + c] = torn ? Q.table[row + c] : -1;
      if (torn && lane == 0) {
        Q.status[c0 + i] = SV_ERR_DATA_PAGE;
        Q.plan[c0 + i] = make_int2(-1, hi - lo);
      }
    }
    __syncthreads();
  }
  if (Q.copy_free) {
    const int64_t at = int64_t(blockIdx.x) * kTbThreads + tid;
    const int64_t step = int64_t(gridDim.x) * kTbThreads;
    const int64_t vecs = Q.vec ? Q.capacity / 4 : 0;
    const int4* from = reinterpret_cast<const int4*>(Q.free_pages);
    for (int64_t i = at; i < vecs; i += step) reinterpret_cast<int4*>(Q.out_free)[i] = from[i];
    for (int64_t i = vecs * 4 + at; i < Q.capacity; i += step) Q.out_free[i] = Q.free_pages[i];
  }
}

// Where the i-th page that is handed on lies in `released`, of a call with requests
// whose entries there are left out.
__device__ __noinline__ int64_t released_at(const ReserveProblem& Q, int64_t i) {
  int64_t upto = 0;   // entries of the requests so far
  for (int b = 0; b < Q.B && upto <= i; ++b) {
    const int2 p = Q.plan[b];
    const int n = p.x < 0 ? p.y : max(p.x - p.y, 0);
    if (p.x < 0) i += n;
    upto += n;
  }
  return i;
}

__global__ void __launch_bounds__(kTbThreads) reserve_grant_kernel(const ReserveProblem Q) {
  __shared__ int2 s_plan[kTbThreads];
  __shared__ int64_t s_first[kTbThreads];
  __shared__ unsigned long long s_taken;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = chunk_start(Q.B, blockIdx.x), r1 = chunk_start(Q.B, blockIdx.x + 1);
  const int64_t n = *Q.count;
  if (n < 0) {   // nothing changes
    for (int b = r0 + tid; b < r1; b += kTbThreads)
      if (Q.out_held != Q.held) Q.out_held[b] = Q.held[b];
    if (blockIdx.x == 0 && tid == 0 && Q.out_count != Q.free_count) *Q.out_count = *Q.free_count;
    return;
  }
  if (tid == 0) s_taken = 0;
  // Wants in the requests' order: a thread has neighbouring requests.  What is
  // handed out is the longest prefix that the free pages cover.
  const int per = (Q.B + kTbThreads - 1) / kTbThreads;
  const int t0 = min(Q.B, tid * per), t1 = min(Q.B, t0 + per);
  int64_t want = 0, rel = 0, mine = 0, wants, released, before;
  for (int b = t0; b < t1; ++b) {
    const int2 p = Q.plan[b];
    if (p.x < 0) {
      rel += int64_t(p.y) << 32;
      continue;
    }
    const int w = max(p.y - p.x, 0);
    want += w;
    rel += max(p.x - p.y, 0);
    if (b < r0) mine += w;
  }
  const int64_t upto = block_scan(want, &wants);
  block_scan(rel, &released);   // (both counts are at most the list's entries)
  block_scan(mine, &before);
  const bool torn = released >> 32;   // some entries of `released` are left out
  released &= 0xffffffff;
  auto given = [&](int64_t i) { return Q.released[torn ? released_at(Q, i) : i]; };
  const int64_t avail = n + released;
  int64_t taken = wants;
  if (wants > avail) {
    int64_t x = upto;
    for (int b = t0; b < t1; ++b) {
      const int2 p = Q.plan[b];
      if (p.x >= 0) x += max(p.y - p.x, 0);
      if (x <= avail) atomicMax(&s_taken, (unsigned long long)x);
    }
    __syncthreads();
    taken = int64_t(s_taken);
  }
  const int64_t left = avail - taken;
  for (int c0 = r0; c0 < r1; c0 += kTbThreads) {
    const int b = c0 + tid;
    int2 p = make_int2(0, 0);
    if (b < r1) p = Q.plan[b];
    const bool bad = p.x < 0;
    if (bad) p = make_int2(0, 0);
    int64_t here;
    const int w = max(p.y - p.x, 0);
    const int64_t first = before + block_scan(w, &here);
    before += here;
    const bool served = w == 0 || first + w <= avail;
    if (b < r1) {
      if (!bad) Q.out_held[b] = served ? p.y : min(p.x, p.y);
      else if (Q.out_held != Q.held) Q.out_held[b] = Q.held[b];
      if (!served) Q.status[b] = SV_ERR_DATA_POOL;
    }
    s_plan[tid] = served ? p : make_int2(0, 0);
    s_first[tid] = first;
    __syncthreads();
    for (int i = warp; i < min(kTbThreads, r1 - c0); i += kTbWarps) {
      const int64_t row = int64_t(c0 + i) * Q.cols;
      const int2 q = s_plan[i];
      for (int c = q.x + lane; c < q.y; c += 32) {
        const int64_t at = avail - 1 - (s_first[i] + c - q.x);
        Q.out_table[row + c] = at >= n ? given(at - n) : Q.free_pages[at];
        if (at < n) Q.out_free[at] = -1;   // read above, by this thread alone
      }
    }
    __syncthreads();
  }
  // what was released and not handed out again
  for (int64_t i = n + int64_t(blockIdx.x) * kTbThreads + tid; i < left;
       i += int64_t(gridDim.x) * kTbThreads)
    Q.out_free[i] = given(i - n);
  if (blockIdx.x == 0 && tid == 0) *Q.out_count = int(left);
}

// -------------------------------------------------------------------- slots
// A CTA has kSlotRows neighbouring rows.  It finds which requests have some of
// them from the sums of the counts, marks each request's first row there, and a
// scan of the marks tells every row its request.
constexpr int kSlotRows = 1024;
constexpr int kSlotPer = kSlotRows / kTbThreads;

struct SlotsProblem {
  const int32_t *table, *start, *count;
  int32_t B, cols, S;
  int64_t rows;
  int64_t* slots;
  int32_t *request, *position, *offsets;
  WsHeader* hdr;
  int32_t* status;   // [B], one entry for the whole call, then one per CTA
};

__global__ void __launch_bounds__(kTbThreads) slots_kernel(const SlotsProblem Q) {
  __shared__ int s_req[kSlotRows], s_off[kSlotRows];
  __shared__ int s_last[kTbWarps];
  __shared__ int s_bad;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r0 = int64_t(blockIdx.x) * kSlotRows, r1 = min(Q.rows, r0 + kSlotRows);
  if (tid == 0) s_bad = INT32_MAX;
  for (int i = tid; i < kSlotRows; i += kTbThreads) s_req[i] = -1;
  const int per = (Q.B + kTbThreads - 1) / kTbThreads;
  const int t0 = min(Q.B, tid * per), t1 = min(Q.B, t0 + per);
  int64_t sum = 0, total;
  for (int b = t0; b < t1; ++b) sum += max(Q.count[b], 0);
  int64_t at = block_scan(sum, &total);
  const bool fail = total > Q.rows;
  const bool first = blockIdx.x == 0;
  // positions that a request has columns for, and that an int32 holds
  const int64_t most = min(int64_t(Q.cols) * Q.S, int64_t(INT32_MAX));
  if (first && tid == 0) {
    Q.hdr->err_code = kStatusList;
    Q.hdr->err_row = Q.B;
    Q.hdr->err_req = 1;          // entries are requests
    Q.hdr->n_active = 1 + gridDim.x;
    Q.status[Q.B] = fail ? -SV_ERR_DATA_ROWS : INT32_MAX;
    Q.offsets[Q.B] = int(min(total, int64_t(INT32_MAX)));
  }
  if (first || (at < r1 && at + sum > r0 && !fail)) {
    for (int b = t0; b < t1; ++b) {
      const int c = Q.count[b], n = max(c, 0);
      if (first) {
        const int s = Q.start[b];
        Q.offsets[b] = int(min(at, int64_t(INT32_MAX)));
        Q.status[b] = c < 0 || s < 0 || int64_t(s) + c > most ? SV_ERR_DATA_LENGTH : 0;
      }
      if (!fail && n > 0 && at < r1 && at + n > r0) {
        const int mark = int(max(at - r0, int64_t(0)));
        s_req[mark] = b;
        s_off[mark] = int(at);
      }
      at += n;
    }
  }
  __syncthreads();
  // the last mark at or before each row: within a thread, a warp, the CTA
  int mark[kSlotPer], last = -1;
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) {
    const int r = tid * kSlotPer + i;
    if (s_req[r] >= 0) last = r;
    mark[i] = last;
  }
  int upto = last;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto = max(upto, y);
  }
  if (lane == 31) s_last[warp] = upto;
  int prev = __shfl_up_sync(0xffffffffu, upto, 1);
  if (lane == 0) prev = -1;
  __syncthreads();
  for (int w = 0; w < warp; ++w) prev = max(prev, s_last[w]);
#pragma unroll
  for (int i = 0; i < kSlotPer; ++i) {
    const int64_t r = r0 + tid * kSlotPer + i;
    if (r >= r1) break;
    int64_t slot = -1;
    int req = -1, pos = -1;
    const int m = max(mark[i], prev);
    if (r < total && m >= 0) {
      req = s_req[m];
      const int s = Q.start[req];
      pos = int(s + (r - s_off[m]));
      if (s >= 0 && int64_t(s) + Q.count[req] <= most) {
        const int page = Q.table[int64_t(req) * Q.cols + pos / Q.S];
        if (page >= 0) slot = int64_t(page) * Q.S + pos % Q.S;
        else atomicMin(&s_bad, req);
      }
    }
    Q.slots[r] = slot;
    Q.request[r] = req;
    Q.position[r] = pos;
  }
  __syncthreads();
  if (tid == 0) Q.status[Q.B + 1 + blockIdx.x] = s_bad;
}

// -------------------------------------------------------------------- write
// A warp moves one entry (K or V of a row) at a time.
struct WriteProblem {
  char* cache;               // the layer's K of page 0
  int64_t page_bytes, v_off, entry_bytes, num_slots;
  const char *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;   // byte strides of row and head
  const int64_t* slots;
  int64_t rows;
  int32_t S, heads, head_bytes;
  WsHeader* hdr;
  int32_t* status;           // one entry per CTA: the first row that has no place
};

// V: bytes moved at a time; a head is a multiple of them and starts on one.
template <class V>
__global__ void __launch_bounds__(kTbThreads) write_kernel(const WriteProblem Q) {
  __shared__ int s_bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_bad = INT32_MAX;
  __syncthreads();
  pdl_wait();
  const int per_head = Q.head_bytes / int(sizeof(V));
  const int n = per_head * Q.heads;
  for (int64_t it = int64_t(blockIdx.x) * kTbWarps + warp; it < 2 * Q.rows;
       it += int64_t(gridDim.x) * kTbWarps) {
    const int64_t r = it >> 1;
    const bool value = it & 1;
    const int64_t slot = __ldg(Q.slots + r);
    if (slot < 0 || slot >= Q.num_slots) {
      // -1 is a row without a place; other such numbers are mistakes
      if (slot != -1 && lane == 0) atomicMin(&s_bad, int(r));
      continue;
    }
    const int64_t page = slot / Q.S;
    V* to = reinterpret_cast<V*>(Q.cache + page * Q.page_bytes + (value ? Q.v_off : 0) +
                                 (slot - page * Q.S) * Q.entry_bytes);
    const char* from = (value ? Q.v : Q.k) + r * (value ? Q.v_ts : Q.k_ts);
    const int64_t hs = value ? Q.v_hs : Q.k_hs;
    for (int i0 = lane; i0 < n; i0 += 128) {
      V x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 32 * u;
        if (i >= n) break;
        const int h = i / per_head;
        x[u] = *reinterpret_cast<const V*>(from + h * hs + (i - h * per_head) * int64_t(sizeof(V)));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (i0 + 32 * u >= n) break;
        to[i0 + 32 * u] = x[u];
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Q.status[blockIdx.x] = s_bad;
    if (blockIdx.x == 0) {
      Q.hdr->err_code = kStatusList;
      Q.hdr->err_row = 0;
      Q.hdr->err_req = 0;      // rows
      Q.hdr->n_active = gridDim.x;
    }
  }
}

constexpr int kWriteCtasPerSm = 8;

template <class Kern, class Problem_>
cudaError_t launch_pdl(Kern kernel, int grid, cudaStream_t s, const Problem_& Q) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kTbThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Q);
}

struct ReserveLayout {
  size_t status, plan, count, released, total;
};
ReserveLayout reserve_layout(int B, int64_t capacity) {
  ReserveLayout L;
  size_t o = align256(sizeof(WsHeader));
  L.status = o;   // right behind the header, as spec_verify_get_error reads it
  o += align256(sizeof(int32_t) * (size_t(B) + 1));
  L.plan = o;
  o += align256(sizeof(int2) * size_t(B));
  L.count = o;
  o += 256;
  L.released = o;
  o += align256(sizeof(int32_t) * size_t(capacity));
  L.total = o;
  return L;
}

}  // namespace

size_t reserve_workspace_bytes(int32_t B, int64_t capacity) {
  return reserve_layout(B, capacity).total;
}

cudaError_t launch_reserve(const int32_t* table, int32_t* out_table, int B, int cols,
                           const int32_t* held, int32_t* out_held, const int32_t* length,
                           const int32_t* free_pages, int32_t* out_free, int64_t capacity,
                           const int32_t* free_count, int32_t* out_count, int page_size,
                           void* workspace, int sms, cudaStream_t s) {
  ReserveProblem Q;
  Q.table = table;
  Q.out_table = out_table;
  Q.held = held;
  Q.length = length;
  Q.out_held = out_held;
  Q.free_pages = free_pages;
  Q.out_free = out_free;
  Q.free_count = free_count;
  Q.out_count = out_count;
  Q.B = B;
  Q.cols = cols;
  Q.S = page_size;
  Q.capacity = capacity;
  Q.copy_table = out_table != table;
  Q.copy_free = out_free != free_pages;
  auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  Q.vec = cols % 4 == 0 && aligned(table) && aligned(out_table) && aligned(free_pages) &&
          aligned(out_free);
  char* w = static_cast<char*>(workspace);
  const ReserveLayout L = reserve_layout(B, capacity);
  Q.hdr = reinterpret_cast<WsHeader*>(w);
  Q.status = reinterpret_cast<int32_t*>(w + L.status);
  Q.plan = reinterpret_cast<int2*>(w + L.plan);
  Q.count = reinterpret_cast<int32_t*>(w + L.count);
  Q.released = reinterpret_cast<int32_t*>(w + L.released);
  // two requests a CTA while the CTAs fit (1024 rows of 2048 columns: 12.9 us with the
  // second kernel; one CTA an SM 14.0, four 14.4)
  const int want = B > 0 ? (B + 1) / 2 : 1, cap = kReserveCtasPerSm * sms;
  const int grid = want < cap ? want : cap;
  if (cudaError_t e = launch_pdl(reserve_release_kernel, grid, s, Q)) return e;
  return launch_pdl(reserve_grant_kernel, grid, s, Q);
}

size_t slots_workspace_bytes(int32_t B, int64_t rows) {
  const int64_t ctas = (rows + kSlotRows - 1) / kSlotRows;
  return align256(sizeof(WsHeader)) +
         align256(sizeof(int32_t) * (size_t(B) + 1 + size_t(ctas > 0 ? ctas : 1)));
}

cudaError_t launch_slots(const int32_t* table, int B, int cols, const int32_t* start,
                         const int32_t* count, int64_t rows, int page_size, int64_t* slots,
                         int32_t* request, int32_t* position, int32_t* offsets, void* workspace,
                         cudaStream_t s) {
  SlotsProblem Q;
  Q.table = table;
  Q.start = start;
  Q.count = count;
  Q.B = B;
  Q.cols = cols;
  Q.S = page_size;
  Q.rows = rows;
  Q.slots = slots;
  Q.request = request;
  Q.position = position;
  Q.offsets = offsets;
  Q.hdr = static_cast<WsHeader*>(workspace);
  Q.status = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(sizeof(WsHeader)));
  const int64_t ctas = (rows + kSlotRows - 1) / kSlotRows;
  return launch_pdl(slots_kernel, int(ctas > 0 ? ctas : 1), s, Q);
}

size_t write_workspace_bytes(int sms) {
  return align256(sizeof(WsHeader)) + align256(sizeof(int32_t) * size_t(sms) * kWriteCtasPerSm);
}

cudaError_t launch_write(const sv_kv_cache& c, int layer, int heads, const void* k, int64_t k_ts,
                         int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs,
                         const int64_t* slots, int64_t rows, void* workspace, int sms,
                         cudaStream_t s) {
  WriteProblem Q;
  const int es = c.elem_bytes;
  Q.entry_bytes = int64_t(c.entry_elems) * es;
  Q.v_off = Q.entry_bytes * c.page_size;
  Q.page_bytes = Q.v_off * 2 * c.n_layers;
  Q.cache = static_cast<char*>(c.data) + Q.v_off * 2 * layer;
  Q.num_slots = c.num_pages * c.page_size;
  Q.S = c.page_size;
  Q.k = static_cast<const char*>(k);
  Q.v = static_cast<const char*>(v);
  Q.k_ts = k_ts * es;
  Q.k_hs = k_hs * es;
  Q.v_ts = v_ts * es;
  Q.v_hs = v_hs * es;
  Q.slots = slots;
  Q.rows = rows;
  Q.heads = heads;
  Q.head_bytes = int(Q.entry_bytes / heads);
  Q.hdr = static_cast<WsHeader*>(workspace);
  Q.status = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(sizeof(WsHeader)));
  if (Q.k_hs == Q.head_bytes && Q.v_hs == Q.head_bytes) {   // an entry is one piece
    Q.heads = 1;
    Q.head_bytes = int(Q.entry_bytes);
  }
  // everything that a vector's address is made of
  const uint64_t bits = reinterpret_cast<uintptr_t>(Q.cache) | reinterpret_cast<uintptr_t>(k) |
                        reinterpret_cast<uintptr_t>(v) | uint64_t(Q.entry_bytes) |
                        uint64_t(Q.head_bytes) | (rows > 1 ? uint64_t(Q.k_ts | Q.v_ts) : 0) |
                        (Q.heads > 1 ? uint64_t(Q.k_hs | Q.v_hs) : 0);
  const int64_t want = (2 * rows + kTbWarps - 1) / kTbWarps, cap = int64_t(sms) * kWriteCtasPerSm;
  const int grid = int(want < cap ? want : cap);
  if (bits % 16 == 0) return launch_pdl(write_kernel<uint4>, grid, s, Q);
  if (es == 4 || bits % 4 == 0) return launch_pdl(write_kernel<uint32_t>, grid, s, Q);
  return launch_pdl(write_kernel<uint16_t>, grid, s, Q);
}

}  // namespace sv
