// Host side of the C ABI: argument validation, workspace layout, and the
// launches on the caller's stream: setup -> row pass over the rows not
// filtered by a kept-set threshold -> row pass over those -> filter / decide
// -> draw pass for verification; sampler setup -> the same two row passes ->
// sampler rows -> draw pass for the draft-side sampler.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>
#include <vector>

#include "sv_attn.cuh"
#include "sv_internal.cuh"
#include "sv_prompt.cuh"

namespace sv {
cudaError_t rowpass_configure();
cudaError_t filter_occupancy(int* occ);
cudaError_t draw_configure();
cudaError_t draw_occupancy(int V, int* occ, int* occ_locate);
}  // namespace sv

using namespace sv;

namespace {

constexpr int kMaxDevices = 64;

struct DeviceState {
  int sms = 0;
  int occ_filter = 1;  // resident filter / decide CTAs per SM
  int occ_draw = 1;    // resident draw CTAs per SM for vocabulary draw_v
  int occ_locate = 1;  // resident locate CTAs per SM for vocabulary draw_v
  int draw_v = -1;
  bool ready = false;
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

// Per-device set-up: SM count, the kernels' shared-memory limits and the
// post-pass kernels' occupancy (the draw pass's depends on the vocabulary).
int prepare_device(int vocab, DeviceState* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SV_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_dev[dev].ready) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      return SV_ERR_CUDA;
    int of = 1;
    if (rowpass_configure() != cudaSuccess || draw_configure() != cudaSuccess ||
        filter_occupancy(&of) != cudaSuccess)
      return SV_ERR_CUDA;
    g_dev[dev].sms = n;
    g_dev[dev].occ_filter = of;
    g_dev[dev].ready = true;
  }
  if (g_dev[dev].draw_v != vocab) {
    int od = 1, ol = 1;
    if (draw_occupancy(vocab, &od, &ol) != cudaSuccess) return SV_ERR_CUDA;
    g_dev[dev].occ_draw = od;
    g_dev[dev].occ_locate = ol;
    g_dev[dev].draw_v = vocab;
  }
  *out = g_dev[dev];
  return SV_OK;
}

std::atomic<int32_t> g_expire_wait{0};

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

size_t elem_size(int dtype) { return dtype == SV_BF16 || dtype == SV_F16 ? 2 : 4; }

int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kMaxDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kMaxDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// The checks and arguments that spec_attention and spec_attention_weights share.
int attn_args(const sv_kv_cache* cache, int32_t dtype, int32_t layer, int32_t kv_heads,
              const void* q, int64_t q_ts, int64_t q_hs, int32_t q_heads, int64_t rows,
              const void* spec, int32_t slots, const int32_t* k_per_req, const int32_t* kv_len,
              const int32_t* table, int32_t max_pages, float scale, int32_t window, int32_t batch,
              AttnArgs* out) {
  if (!cache || batch < 0 || rows < 0 || max_pages < 0 || window < 0) return SV_ERR_ARG;
  const sv_kv_cache& c = *cache;
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_UNSUPPORTED;
  if (c.num_pages < 0 || c.n_layers < 1 || c.page_size < 1 || c.entry_elems < 1 ||
      size_t(c.elem_bytes) != elem_size(dtype) || layer < 0 || layer >= c.n_layers ||
      kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || c.entry_elems % kv_heads != 0)
    return SV_ERR_ARG;
  if (!(scale > -INFINITY && scale < INFINITY)) return SV_ERR_ARG;
  if (rows < batch || rows >= INT_MAX || (rows > 0 && batch == 0)) return SV_ERR_ARG;
  const int D = c.entry_elems / kv_heads;
  if (D > SV_HEAD_DIM_MAX || (size_t(D) * c.elem_bytes) % 16 != 0) return SV_ERR_UNSUPPORTED;
  if (batch > 0) {
    if (!q || !k_per_req || !kv_len || (max_pages > 0 && !table) ||
        (c.num_pages > 0 && !c.data) || (spec && slots < 1))
      return SV_ERR_ARG;
    if (misaligned(c.data, 16) || misaligned(spec, 16)) return SV_ERR_UNSUPPORTED;
  }
  AttnArgs A{};
  A.q = q;
  A.q_ts = q_ts;
  A.q_hs = q_hs;
  A.entry_bytes = int64_t(c.entry_elems) * c.elem_bytes;
  A.v_off = A.entry_bytes * c.page_size;
  A.page_bytes = A.v_off * 2 * c.n_layers;
  A.cache = static_cast<const char*>(c.data) + A.v_off * 2 * layer;
  A.layer_row = 2 * layer * c.page_size;
  A.num_pages = c.num_pages;
  A.spec_tok = A.entry_bytes * 2 * c.n_layers;
  A.spec_req = A.spec_tok * slots;
  A.spec = spec ? static_cast<const char*>(spec) + A.entry_bytes * 2 * layer : nullptr;
  A.slots = slots;
  A.kv_len = kv_len;
  A.k_per_req = k_per_req;
  A.table = table;
  A.S = c.page_size;
  A.max_pages = max_pages;
  A.B = batch;
  A.Hq = q_heads;
  A.Hkv = kv_heads;
  A.G = q_heads / kv_heads;
  A.D = D;
  A.window = window < kMaxPositions ? window : 0;  // a wider one hides nothing
  A.Rt = rows;
  A.scale2 = scale * 1.4426950408889634f;
  A.max_k = SV_MAX_K;
  A.test_expire = g_expire_wait.load(std::memory_order_relaxed);
  *out = A;
  return SV_OK;
}

}  // namespace

extern "C" {

size_t spec_verify_workspace_size(int32_t batch, int64_t target_rows, int64_t draft_rows) {
  if (batch < 0 || target_rows < 0 || draft_rows < 0 || target_rows + draft_rows >= INT_MAX)
    return 0;
  return ws_layout(batch, target_rows, draft_rows).total;
}

int spec_verify(const sv_logits* target_logits, const sv_logits* draft_logits,
                const int32_t* draft_tokens, const int32_t* k_per_req, const float* temperature,
                const int32_t* top_k, const float* top_p, const float* uniforms,
                int32_t* out_accept_len, int32_t* out_tokens, void* stream, int32_t batch,
                void* workspace, size_t workspace_bytes, const sv_options* options) {
  if (!target_logits || !draft_logits || batch < 0) return SV_ERR_ARG;
  const sv_logits& t = *target_logits;
  const sv_logits& d = *draft_logits;
  if (t.dtype != SV_F32 && t.dtype != SV_BF16) return SV_ERR_UNSUPPORTED;
  if (d.dtype != t.dtype) return SV_ERR_UNSUPPORTED;
  if (d.vocab != t.vocab || t.vocab < 1) return SV_ERR_ARG;
  if (t.vocab > SV_VOCAB_MAX) return SV_ERR_UNSUPPORTED;
  if (t.rows < 0 || d.rows < 0 || t.rows + d.rows >= INT_MAX) return SV_ERR_ARG;
  // sum_b (k_b + 1) = B + sum_b k_b, whatever the k_b are
  if (t.rows != int64_t(batch) + d.rows) return SV_ERR_ARG;
  const size_t es = elem_size(t.dtype);
  if (t.row_stride < t.vocab) return SV_ERR_ARG;
  if (d.data && d.rows > 0 && d.row_stride < d.vocab) return SV_ERR_ARG;
  if (batch > 0 && (!t.data || !k_per_req || !temperature || !uniforms || !out_accept_len ||
                    !out_tokens))
    return SV_ERR_ARG;
  if (d.rows > 0 && !draft_tokens) return SV_ERR_ARG;
  if (misaligned(t.data, 16) || (size_t(t.row_stride) * es) % 16 != 0) return SV_ERR_UNSUPPORTED;
  if (d.data && (misaligned(d.data, 16) || (size_t(d.row_stride) * es) % 16 != 0))
    return SV_ERR_UNSUPPORTED;
  const WsLayout L = ws_layout(batch, t.rows, d.rows);
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < L.total)
    return SV_ERR_WORKSPACE;
  if (batch == 0) return SV_OK;

  DeviceState ds;
  if (int rc = prepare_device(t.vocab, &ds)) return rc;
  const int sms = ds.sms;

  Problem P{};
  P.target = t.data;
  P.draft = d.data;
  P.t_stride = t.row_stride;
  P.d_stride = d.data ? d.row_stride : 0;
  P.Rt = t.rows;
  P.Rd = d.rows;
  P.V = t.vocab;
  P.B = batch;
  P.draft_tokens = draft_tokens;
  P.k_per_req = k_per_req;
  P.temperature = temperature;
  P.top_k = top_k;
  P.top_p = top_p;
  P.uniforms = uniforms;
  P.out_accept_len = out_accept_len;
  P.out_tokens = out_tokens;
  P.out_pq = options ? options->out_pq : nullptr;
  P.out_q = nullptr;
  P.n_seg = 1;
  P.test_expire = options ? options->test_expire_wait : 0;
  P.inline_draw = t.vocab <= kInlineDrawV;
  P.ws = ws_bind(workspace, L);

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_setup(P, s) != cudaSuccess) return SV_ERR_CUDA;
  const int64_t rows = t.rows + d.rows;
  const int64_t ctas = int64_t(sms) * kRowpassCtasPerSm;
  const int grid = int(rows < ctas ? rows : ctas);
  if (options && options->event_rowpass_begin &&
      cudaEventRecord(static_cast<cudaEvent_t>(options->event_rowpass_begin), s) != cudaSuccess)
    return SV_ERR_CUDA;
  // every row but those filtered by a kept-set threshold (top-p alone, large
  // top-k), then those: the second launch's CTAs become resident in the
  // first one's tail, so that it costs little when it has no rows; without
  // top_k and top_p arrays no row can need it, and it is not launched
  const bool threshold_rows = top_k != nullptr || top_p != nullptr;
  if (grid > 0 && (launch_rowpass(P, t.dtype == SV_BF16, false, grid, s) != cudaSuccess ||
                   (threshold_rows &&
                    launch_rowpass(P, t.dtype == SV_BF16, true, grid, s) != cudaSuccess)))
    return SV_ERR_CUDA;
  if (options && options->event_rowpass_end &&
      cudaEventRecord(static_cast<cudaEvent_t>(options->event_rowpass_end), s) != cudaSuccess)
    return SV_ERR_CUDA;
  const bool bf16 = t.dtype == SV_BF16;
  const int64_t fjobs = rows;  // at most one job per row
  const int64_t fmax = int64_t(sms) * ds.occ_filter;
  if (launch_filter_decide(P, bf16, int(fjobs < fmax ? fjobs : fmax), s) != cudaSuccess)
    return SV_ERR_CUDA;
  // short rows: every draw was taken by its decide job
  if (P.inline_draw) return SV_OK;
  // draw pass: a queued draw is cut into segments so that the units (draws x
  // segments) outnumber the resident CTAs about kDrawUnitsPerCta-fold and the
  // last round is short (at most one queued draw per request); then the
  // locate kernel, one CTA per queued draw
  const int64_t dmax = int64_t(sms) * ds.occ_draw;
  P.n_seg = int(std::max<int64_t>(
      1, std::min<int64_t>(kMaxSeg, (kDrawUnitsPerCta * dmax + batch - 1) / std::max(batch, 1))));
  const int64_t djobs = int64_t(batch) * P.n_seg;
  const int64_t lmax = int64_t(sms) * ds.occ_locate;
  if (launch_draw(P, bf16, int(djobs < dmax ? djobs : dmax), s) != cudaSuccess ||
      launch_locate(P, bf16, int(batch < lmax ? batch : lmax), s) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}

size_t spec_draft_sample_workspace_size(int32_t batch, int64_t rows) {
  if (batch < 0 || rows < 0 || rows >= INT_MAX) return 0;
  return sample_ws_layout(batch, rows).total;
}

int spec_draft_sample(const sv_logits* draft_logits, const int32_t* k_per_req,
                      const float* temperature, const int32_t* top_k, const float* top_p,
                      const float* uniforms, int32_t* out_tokens, float* out_q, void* stream,
                      int32_t batch, void* workspace, size_t workspace_bytes,
                      const sv_options* options) {
  if (!draft_logits || batch < 0) return SV_ERR_ARG;
  const sv_logits& x = *draft_logits;
  if (x.dtype != SV_F32 && x.dtype != SV_BF16) return SV_ERR_UNSUPPORTED;
  if (x.vocab < 1) return SV_ERR_ARG;
  if (x.vocab > SV_VOCAB_MAX) return SV_ERR_UNSUPPORTED;
  if (x.rows < 0 || x.rows >= INT_MAX || x.row_stride < x.vocab) return SV_ERR_ARG;
  if (batch > 0 && (!k_per_req || !temperature)) return SV_ERR_ARG;
  if (x.rows > 0 && (!x.data || !uniforms || !out_tokens)) return SV_ERR_ARG;
  const size_t es = elem_size(x.dtype);
  if (x.data && (misaligned(x.data, 16) || (size_t(x.row_stride) * es) % 16 != 0))
    return SV_ERR_UNSUPPORTED;
  const WsLayout L = sample_ws_layout(batch, x.rows);
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < L.total)
    return SV_ERR_WORKSPACE;
  if (batch == 0) return x.rows == 0 ? SV_OK : SV_ERR_ARG;

  DeviceState ds;
  if (int rc = prepare_device(x.vocab, &ds)) return rc;
  const int sms = ds.sms;

  Problem P{};
  P.target = x.data;
  P.draft = nullptr;
  P.t_stride = x.row_stride;
  P.d_stride = 0;
  P.Rt = x.rows;  // the drafter rows play the part of target rows in the row pass
  P.Rd = 0;
  P.V = x.vocab;
  P.B = batch;
  P.n_seg = 1;
  P.draft_tokens = nullptr;
  P.k_per_req = k_per_req;
  P.temperature = temperature;
  P.top_k = top_k;
  P.top_p = top_p;
  P.uniforms = uniforms;
  P.out_accept_len = nullptr;
  P.out_tokens = out_tokens;
  P.out_pq = nullptr;
  P.out_q = out_q;
  P.test_expire = 0;
  P.ws = ws_bind(workspace, L);

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_sample_setup(P, s) != cudaSuccess) return SV_ERR_CUDA;
  const int64_t rows = x.rows;
  if (rows == 0) return SV_OK;
  const bool bf16 = x.dtype == SV_BF16;
  const int64_t ctas = int64_t(sms) * kRowpassCtasPerSm;
  if (options && options->event_rowpass_begin &&
      cudaEventRecord(static_cast<cudaEvent_t>(options->event_rowpass_begin), s) != cudaSuccess)
    return SV_ERR_CUDA;
  const bool threshold_rows = top_k != nullptr || top_p != nullptr;
  if (launch_rowpass(P, bf16, false, int(rows < ctas ? rows : ctas), s) != cudaSuccess ||
      (threshold_rows &&
       launch_rowpass(P, bf16, true, int(rows < ctas ? rows : ctas), s) != cudaSuccess))
    return SV_ERR_CUDA;
  if (options && options->event_rowpass_end &&
      cudaEventRecord(static_cast<cudaEvent_t>(options->event_rowpass_end), s) != cudaSuccess)
    return SV_ERR_CUDA;
  const int64_t fmax = int64_t(sms) * ds.occ_filter;
  if (launch_sample_post(P, bf16, int(rows < fmax ? rows : fmax), s) != cudaSuccess)
    return SV_ERR_CUDA;
  // every sampled unfiltered row may queue a draw
  const int64_t dmax = int64_t(sms) * ds.occ_draw;
  P.n_seg = int(std::max<int64_t>(
      1, std::min<int64_t>(kMaxSeg, (kDrawUnitsPerCta * dmax + rows - 1) / rows)));
  const int64_t djobs = rows * P.n_seg;
  const int64_t lmax = int64_t(sms) * ds.occ_locate;
  if (launch_draw(P, bf16, int(djobs < dmax ? djobs : dmax), s) != cudaSuccess ||
      launch_locate(P, bf16, int(rows < lmax ? rows : lmax), s) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}

size_t spec_kv_commit_workspace_size(int32_t batch) {
  return batch < 0 ? 0 : kv_workspace_bytes(batch, SV_MAX_K);
}

size_t spec_kv_commit_path_workspace_size(int32_t batch) {
  return batch < 0 ? 0 : kv_workspace_bytes(batch, SV_TREE_MAX_K);
}

static int kv_commit(const sv_kv_cache* cache, const void* spec, int32_t spec_slots,
                     const int32_t* accept_len, const int32_t* k_per_req, const int32_t* path,
                     int64_t rows, int max_k, int32_t* kv_len, const int32_t* block_table,
                     int32_t max_pages, void* stream, int32_t batch, void* workspace,
                     size_t workspace_bytes) {
  if (!cache || batch < 0 || spec_slots < 1 || max_pages < 0) return SV_ERR_ARG;
  const sv_kv_cache& c = *cache;
  if (c.num_pages < 0 || c.n_layers < 1 || c.page_size < 1 || c.entry_elems < 1 ||
      (c.elem_bytes != 2 && c.elem_bytes != 4))
    return SV_ERR_ARG;
  const int64_t entry_bytes = int64_t(c.entry_elems) * c.elem_bytes;
  if (entry_bytes % 16 != 0) return SV_ERR_UNSUPPORTED;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < kv_workspace_bytes(batch, max_k))
    return SV_ERR_WORKSPACE;
  if (batch == 0) return SV_OK;
  if (!c.data || !spec || !accept_len || !k_per_req || !kv_len || (max_pages > 0 && !block_table))
    return SV_ERR_ARG;
  if (misaligned(c.data, 16) || misaligned(spec, 16)) return SV_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SV_ERR_CUDA;
  if (launch_kv_commit(c.data, spec, c.num_pages, c.n_layers, c.page_size, entry_bytes,
                       spec_slots, accept_len, k_per_req, kv_len, block_table, max_pages, batch,
                       path, rows, max_k, workspace, sms,
                       static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return SV_ERR_CUDA;
  return SV_OK;
}

int spec_kv_commit(const sv_kv_cache* cache, const void* spec, int32_t spec_slots,
                   const int32_t* accept_len, const int32_t* k_per_req, int32_t* kv_len,
                   const int32_t* block_table, int32_t max_pages, void* stream, int32_t batch,
                   void* workspace, size_t workspace_bytes) {
  return kv_commit(cache, spec, spec_slots, accept_len, k_per_req, nullptr, 0, SV_MAX_K, kv_len,
                   block_table, max_pages, stream, batch, workspace, workspace_bytes);
}

// Batches of trees whose rows a 32-bit sum holds whatever their lengths say.
static bool tree_batch(int32_t batch) { return batch <= INT_MAX / (SV_TREE_MAX_K + 1); }

int spec_kv_commit_path(const sv_kv_cache* cache, const void* spec, int32_t spec_slots,
                        const int32_t* accept_len, const int32_t* k_per_req, const int32_t* path,
                        int64_t rows, int32_t* kv_len, const int32_t* block_table,
                        int32_t max_pages, void* stream, int32_t batch, void* workspace,
                        size_t workspace_bytes) {
  if (rows < batch || rows >= INT_MAX || (batch > 0 && !path)) return SV_ERR_ARG;
  if (!tree_batch(batch)) return SV_ERR_UNSUPPORTED;
  return kv_commit(cache, spec, spec_slots, accept_len, k_per_req, path, rows, SV_TREE_MAX_K,
                   kv_len, block_table, max_pages, stream, batch, workspace, workspace_bytes);
}

size_t spec_lmhead_stats_workspace_size(int32_t rows, int32_t vocab) {
  if (rows < 0 || vocab < 1) return 0;
  return lmhead_workspace_bytes(rows, vocab);
}

int spec_lmhead_stats(const void* hidden, const void* unembed, int32_t rows, int32_t vocab,
                      int32_t d, const float* temperature, const int32_t* tokens,
                      float* out_max, double* out_sum, int32_t* out_argmax, float* out_token,
                      void* stream, void* workspace, size_t workspace_bytes) {
  if (rows < 0 || vocab < 1 || d < 1) return SV_ERR_ARG;
  if (d % 8 != 0) return SV_ERR_UNSUPPORTED;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < lmhead_workspace_bytes(rows, vocab))
    return SV_ERR_WORKSPACE;
  if (rows == 0) return SV_OK;
  if (!hidden || !unembed || !temperature || !out_max || !out_sum || !out_argmax || !out_token)
    return SV_ERR_ARG;
  if (misaligned(hidden, 16) || misaligned(unembed, 16)) return SV_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SV_ERR_CUDA;
  return launch_lmhead_stats(hidden, unembed, rows, vocab, d, temperature, tokens, out_max,
                             out_sum, out_argmax, out_token, workspace, sms,
                             static_cast<cudaStream_t>(stream));
}

int spec_adapt_k(const int32_t* accept_len, const int32_t* k_used, double* succ, double* fail,
                 double decay, double c, int32_t k_min, int32_t k_max, int32_t* k_next,
                 float* alpha, void* stream, int32_t batch) {
  if (batch < 0 || k_min < 0 || k_max < k_min || k_max > SV_MAX_K || !(decay >= 0.0) ||
      !(decay <= 1.0) || !(c >= 0.0))
    return SV_ERR_ARG;
  if (batch == 0) return SV_OK;
  if (!accept_len || !k_used || !succ || !fail || !k_next) return SV_ERR_ARG;
  return launch_adapt_k(accept_len, k_used, succ, fail, decay, c, k_min, k_max, k_next, alpha,
                        batch, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_verify_greedy_workspace_size(void) { return align256(sizeof(WsHeader)); }

int spec_verify_greedy_from_argmax(const int32_t* target_argmax, const int32_t* draft_tokens,
                                   const int32_t* k_per_req, int32_t* out_accept_len,
                                   int32_t* out_tokens, void* stream, int32_t batch,
                                   int64_t target_rows, int32_t vocab, void* workspace,
                                   size_t workspace_bytes) {
  if (batch < 0 || target_rows < 0 || vocab < 1 || target_rows >= INT_MAX) return SV_ERR_ARG;
  if (target_rows < int64_t(batch)) return SV_ERR_ARG;
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < sizeof(WsHeader))
    return SV_ERR_WORKSPACE;
  if (batch == 0) return SV_OK;
  if (!target_argmax || !k_per_req || !out_accept_len || !out_tokens) return SV_ERR_ARG;
  if (target_rows > int64_t(batch) && !draft_tokens) return SV_ERR_ARG;
  return launch_greedy_from_argmax(target_argmax, draft_tokens, k_per_req, out_accept_len,
                                   out_tokens, batch, target_rows, vocab, workspace,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_verify_tree_greedy_workspace_size(int32_t batch) {
  return batch < 0 ? 0 : tree_greedy_workspace_bytes(batch);
}

int spec_verify_tree_greedy(const int32_t* target_argmax, const int32_t* draft_tokens,
                            const int32_t* parent, const int32_t* k_per_req,
                            int32_t* out_accept_len, int32_t* out_tokens, int32_t* out_path,
                            void* stream, int32_t batch, int64_t target_rows, int32_t vocab,
                            void* workspace, size_t workspace_bytes) {
  if (batch < 0 || target_rows < batch || vocab < 1 || target_rows >= INT_MAX) return SV_ERR_ARG;
  if (!tree_batch(batch)) return SV_ERR_UNSUPPORTED;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < tree_greedy_workspace_bytes(batch))
    return SV_ERR_WORKSPACE;
  if (batch == 0) return SV_OK;
  if (!target_argmax || !parent || !k_per_req || !out_accept_len || !out_tokens || !out_path ||
      (target_rows > batch && !draft_tokens))
    return SV_ERR_ARG;
  return launch_tree_greedy(target_argmax, draft_tokens, parent, k_per_req, out_accept_len,
                            out_tokens, out_path, batch, target_rows, vocab, workspace,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

void spec_test_expire_wait(int32_t n) { g_expire_wait.store(n, std::memory_order_relaxed); }

size_t spec_attention_workspace_size(int32_t batch, int32_t head_dim) {
  const int sms = sm_count();
  if (batch < 0 || head_dim < 1 || head_dim > SV_HEAD_DIM_MAX || sms == 0) return 0;
  return attn_workspace_bytes(batch, head_dim, sms, false);
}

// What spec_attention and spec_tree_attention do with the arguments they have checked.
static int attention_call(AttnArgs& A, int32_t dtype, void* out, float* lse, void* stream,
                          void* workspace, size_t workspace_bytes) {
  const bool tree = A.parent != nullptr;
  if (A.B == 0) return SV_OK;
  if (!out || !lse) return SV_ERR_ARG;
  if (!workspace || misaligned(workspace, 256)) return SV_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms == 0) return SV_ERR_CUDA;
  if (workspace_bytes < attn_workspace_bytes(A.B, A.D, sms, false, tree)) return SV_ERR_WORKSPACE;
  A.out = out;
  A.o_hs = A.D;
  A.o_ts = int64_t(A.D) * A.Hq;
  A.lse = lse;
  return launch_attn(A, dtype, false, workspace, sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

int spec_attention(const sv_kv_cache* cache, int32_t dtype, int32_t layer, int32_t kv_heads,
                   const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads,
                   int64_t rows, const void* spec, int32_t spec_slots, const int32_t* k_per_req,
                   const int32_t* kv_len, const int32_t* block_table, int32_t max_pages,
                   float scale, int32_t window, void* out, float* lse, void* stream,
                   int32_t batch, void* workspace, size_t workspace_bytes) {
  AttnArgs A;
  if (int rc = attn_args(cache, dtype, layer, kv_heads, q, q_token_stride, q_head_stride, q_heads,
                         rows, spec, spec_slots, k_per_req, kv_len, block_table, max_pages, scale,
                         window, batch, &A))
    return rc;
  return attention_call(A, dtype, out, lse, stream, workspace, workspace_bytes);
}

size_t spec_tree_attention_workspace_size(int32_t batch, int32_t head_dim) {
  const int sms = sm_count();
  if (batch < 0 || head_dim < 1 || head_dim > SV_HEAD_DIM_MAX || sms == 0) return 0;
  return attn_workspace_bytes(batch, head_dim, sms, false, true);
}

int spec_tree_attention(const sv_kv_cache* cache, int32_t dtype, int32_t layer, int32_t kv_heads,
                        const void* q, int64_t q_token_stride, int64_t q_head_stride,
                        int32_t q_heads, int64_t rows, const void* spec, int32_t spec_slots,
                        const int32_t* k_per_req, const int32_t* parent, const int32_t* kv_len,
                        const int32_t* block_table, int32_t max_pages, float scale, int32_t window,
                        void* out, float* lse, void* stream, int32_t batch, void* workspace,
                        size_t workspace_bytes) {
  AttnArgs A;
  if (int rc = attn_args(cache, dtype, layer, kv_heads, q, q_token_stride, q_head_stride, q_heads,
                         rows, spec, spec_slots, k_per_req, kv_len, block_table, max_pages, scale,
                         window, batch, &A))
    return rc;
  if (batch > 0 && (!spec || !parent)) return SV_ERR_ARG;
  if (!tree_batch(batch)) return SV_ERR_UNSUPPORTED;
  A.parent = parent;
  A.max_k = SV_TREE_MAX_K;
  return attention_call(A, dtype, out, lse, stream, workspace, workspace_bytes);
}

size_t spec_prompt_attention_workspace_size(int32_t batch) {
  const int sms = sm_count();
  return batch < 0 || sms == 0 ? 0 : prompt_workspace_bytes(batch, sms);
}

int spec_prompt_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          const void* k, int64_t k_row_stride, int64_t k_head_stride,
                          const void* v, int64_t v_row_stride, int64_t v_head_stride,
                          int32_t dtype, int64_t rows, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, const int32_t* offsets, float scale, int32_t window,
                          void* out, float* lse, void* stream, int32_t batch, void* workspace,
                          size_t workspace_bytes) {
  if (batch < 0 || rows < 0 || rows >= INT_MAX - 255 || window < 0 || head_dim < 1 ||
      kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0)
    return SV_ERR_ARG;
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_UNSUPPORTED;
  if (!(scale > -INFINITY && scale < INFINITY)) return SV_ERR_ARG;
  // (tiles of rows and heads are a grid's extents, and a sequence has a unit a KV head)
  if (head_dim > SV_HEAD_DIM_MAX || kv_heads > 65535 ||
      rows * (q_heads / kv_heads) / 64 + batch >= INT_MAX || int64_t(batch) * kv_heads >= INT_MAX)
    return SV_ERR_UNSUPPORTED;
  if (rows == 0 || batch == 0) return SV_OK;
  if (!q || !k || !v || !offsets || !out || !lse) return SV_ERR_ARG;
  const size_t es = elem_size(dtype);
  if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(out, es))
    return SV_ERR_UNSUPPORTED;
  if (!workspace || misaligned(workspace, 256)) return SV_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms == 0) return SV_ERR_CUDA;
  if (workspace_bytes < prompt_workspace_bytes(batch, sms)) return SV_ERR_WORKSPACE;
  PromptArgs A{};
  A.q = q;
  A.q_ts = q_row_stride;
  A.q_hs = q_head_stride;
  A.k = k;
  A.k_ts = k_row_stride;
  A.k_hs = k_head_stride;
  A.v = v;
  A.v_ts = v_row_stride;
  A.v_hs = v_head_stride;
  A.out = out;
  A.lse = lse;
  A.offsets = offsets;
  A.B = batch;
  A.Hq = q_heads;
  A.Hkv = kv_heads;
  A.G = q_heads / kv_heads;
  A.D = head_dim;
  A.window = window < rows ? window : 0;   // a wider one hides nothing
  A.rows = rows;
  A.scale2 = scale * 1.4426950408889634f;
  A.test_expire = g_expire_wait.load(std::memory_order_relaxed);
  return launch_prompt(A, dtype, workspace, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_kv_reserve_workspace_size(int32_t batch, int64_t capacity) {
  return batch < 0 || capacity < 0 || capacity >= INT_MAX ? 0
                                                          : reserve_workspace_bytes(batch, capacity);
}

int spec_kv_reserve(const int32_t* table, int32_t* out_table, int32_t max_pages,
                    const int32_t* held, int32_t* out_held, const int32_t* length,
                    const int32_t* free_pages, int32_t* out_free, int64_t capacity,
                    const int32_t* free_count, int32_t* out_count, int32_t page_size,
                    void* stream, int32_t batch, void* workspace, size_t workspace_bytes) {
  if (batch < 0 || max_pages < 0 || page_size < 1 || capacity < 0 || capacity >= INT_MAX)
    return SV_ERR_ARG;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < reserve_workspace_bytes(batch, capacity))
    return SV_ERR_WORKSPACE;
  // without requests there is a list to copy, or nothing to do
  if (batch == 0 && free_pages == out_free && free_count == out_count) return SV_OK;
  if ((batch > 0 && ((max_pages > 0 && (!table || !out_table)) || !held || !out_held || !length)) ||
      (capacity > 0 && (!free_pages || !out_free)) || !free_count || !out_count)
    return SV_ERR_ARG;
  const int sms = sm_count();
  if (sms == 0) return SV_ERR_CUDA;
  return launch_reserve(table, out_table, batch, max_pages, held, out_held, length, free_pages,
                        out_free, capacity, free_count, out_count, page_size, workspace, sms,
                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_kv_slots_workspace_size(int32_t batch, int64_t rows) {
  return batch < 0 || rows < 0 || rows >= INT_MAX ? 0 : slots_workspace_bytes(batch, rows);
}

int spec_kv_slots(const int32_t* block_table, int32_t max_pages, const int32_t* start,
                  const int32_t* count, int64_t rows, int32_t page_size, int64_t* out_slots,
                  int32_t* out_request, int32_t* out_position, int32_t* out_offsets, void* stream,
                  int32_t batch, void* workspace, size_t workspace_bytes) {
  if (batch < 0 || max_pages < 0 || page_size < 1 || rows < 0 || rows >= INT_MAX)
    return SV_ERR_ARG;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < slots_workspace_bytes(batch, rows))
    return SV_ERR_WORKSPACE;
  if (!out_offsets || (rows > 0 && (!out_slots || !out_request || !out_position)) ||
      (batch > 0 && (!start || !count || (max_pages > 0 && !block_table))))
    return SV_ERR_ARG;
  if (misaligned(out_slots, 8)) return SV_ERR_UNSUPPORTED;
  return launch_slots(block_table, batch, max_pages, start, count, rows, page_size, out_slots,
                      out_request, out_position, out_offsets, workspace,
                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_kv_write_workspace_size(int64_t rows) {
  const int sms = sm_count();
  return rows < 0 || sms == 0 ? 0 : write_workspace_bytes(sms);
}

int spec_kv_write(const sv_kv_cache* cache, int32_t layer, int32_t kv_heads, const void* k,
                  int64_t k_row_stride, int64_t k_head_stride, const void* v,
                  int64_t v_row_stride, int64_t v_head_stride, const int64_t* slots, int64_t rows,
                  void* stream, void* workspace, size_t workspace_bytes) {
  if (!cache || rows < 0 || rows >= INT_MAX) return SV_ERR_ARG;
  const sv_kv_cache& c = *cache;
  if (c.num_pages < 0 || c.n_layers < 1 || c.page_size < 1 || c.entry_elems < 1 ||
      (c.elem_bytes != 2 && c.elem_bytes != 4) || layer < 0 || layer >= c.n_layers ||
      kv_heads < 1 || c.entry_elems % kv_heads != 0)
    return SV_ERR_ARG;
  if (rows == 0) return SV_OK;
  if (!k || !v || !slots || (c.num_pages > 0 && !c.data)) return SV_ERR_ARG;
  const size_t es = size_t(c.elem_bytes);
  if (misaligned(c.data, es) || misaligned(k, es) || misaligned(v, es) || misaligned(slots, 8))
    return SV_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms == 0) return SV_ERR_CUDA;
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < write_workspace_bytes(sms))
    return SV_ERR_WORKSPACE;
  return launch_write(c, layer, kv_heads, k, k_row_stride, k_head_stride, v, v_row_stride,
                      v_head_stride, slots, rows, workspace, sms,
                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_attention_weights_workspace_size(int32_t batch) {
  const int sms = sm_count();
  return batch < 0 || sms == 0 ? 0 : attn_workspace_bytes(batch, 16, sms, true);
}

int spec_attention_weights(const sv_kv_cache* cache, int32_t dtype, int32_t layer,
                           int32_t kv_heads, const void* q, int64_t q_token_stride,
                           int64_t q_head_stride, int32_t q_heads, int64_t rows, const void* spec,
                           int32_t spec_slots, const int32_t* k_per_req, const int32_t* kv_len,
                           const int32_t* block_table, int32_t max_pages, float scale,
                           int32_t window, const float* lse, const int32_t* accept_len,
                           const float* score, int64_t score_stride, float* out_score,
                           int64_t out_stride, int32_t score_cols, void* stream, int32_t batch,
                           void* workspace, size_t workspace_bytes) {
  AttnArgs A;
  if (int rc = attn_args(cache, dtype, layer, kv_heads, q, q_token_stride, q_head_stride, q_heads,
                         rows, spec, spec_slots, k_per_req, kv_len, block_table, max_pages, scale,
                         window, batch, &A))
    return rc;
  if (score_cols < 0 || (batch > 1 && (score_stride < score_cols || out_stride < score_cols)))
    return SV_ERR_ARG;
  // one buffer has one row stride
  if (score == out_score && batch > 1 && score_stride != out_stride) return SV_ERR_ARG;
  if (batch == 0) return SV_OK;
  if (!lse || (score_cols > 0 && (!score || !out_score))) return SV_ERR_ARG;
  if (!workspace || misaligned(workspace, 256)) return SV_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms == 0) return SV_ERR_CUDA;
  if (workspace_bytes < attn_workspace_bytes(batch, A.D, sms, true)) return SV_ERR_WORKSPACE;
  A.lse = const_cast<float*>(lse);
  A.accept_len = accept_len;
  A.score = score;
  A.out_score = out_score;
  A.score_stride = score_stride;
  A.out_stride = out_stride;
  A.score_cols = score_cols;
  return launch_attn(A, dtype, true, workspace, sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_kv_evict_workspace_size(int32_t batch, int32_t budget) {
  return batch < 0 || budget < 1 ? 0 : evict_workspace_bytes(batch, budget);
}

int spec_kv_evict(const sv_kv_cache* cache, const int32_t* block_table, int32_t max_pages,
                  const sv_kv_cache* dst, const int32_t* dst_table, int32_t dst_max_pages,
                  const float* score, int64_t score_stride, int32_t score_cols, float* out_score,
                  int64_t out_stride, int32_t out_cols, const int32_t* kv_len, int32_t* out_len,
                  int32_t budget, int32_t sinks, int32_t recent, int32_t* out_kept, void* stream,
                  int32_t batch, void* workspace, size_t workspace_bytes) {
  if (!cache || batch < 0 || max_pages < 0 || budget < 1 || sinks < 0 || recent < 0 ||
      int64_t(sinks) + recent > budget || score_cols < 0 || out_cols < 0)
    return SV_ERR_ARG;
  if (batch > 1 && (score_stride < score_cols || out_stride < out_cols)) return SV_ERR_ARG;
  if (score == out_score && batch > 1 && score_stride != out_stride) return SV_ERR_ARG;
  const sv_kv_cache& c = *cache;
  if (c.num_pages < 0 || c.n_layers < 1 || c.page_size < 1 || c.entry_elems < 1 ||
      (c.elem_bytes != 2 && c.elem_bytes != 4))
    return SV_ERR_ARG;
  if ((int64_t(c.entry_elems) * c.elem_bytes) % 16 != 0 || batch > 65535)
    return SV_ERR_UNSUPPORTED;
  if (dst) {
    if (dst->n_layers != c.n_layers || dst->page_size != c.page_size ||
        dst->entry_elems != c.entry_elems || dst->elem_bytes != c.elem_bytes ||
        dst->num_pages < 0 || dst_max_pages < 0)
      return SV_ERR_ARG;
  }
  // the request's own pages, named as such or as the destination
  const bool in_place = !dst || (dst->data == c.data && dst->num_pages == c.num_pages &&
                                 dst_table == block_table && dst_max_pages == max_pages);
  const sv_kv_cache& d = in_place ? c : *dst;
  const int32_t* dt = in_place ? block_table : dst_table;
  const int32_t dcols = in_place ? max_pages : dst_max_pages;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < evict_workspace_bytes(batch, budget))
    return SV_ERR_WORKSPACE;
  if (batch == 0) return SV_OK;
  if (!kv_len || !out_len || (max_pages > 0 && !block_table) || (dcols > 0 && !dt) ||
      (c.num_pages > 0 && !c.data) || (d.num_pages > 0 && !d.data) || (score_cols > 0 && !score) ||
      (out_cols > 0 && !out_score))
    return SV_ERR_ARG;
  if (misaligned(c.data, 16) || misaligned(d.data, 16)) return SV_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms == 0) return SV_ERR_CUDA;
  return launch_evict(c, block_table, max_pages, d, dt, dcols, score, score_stride, score_cols,
                      out_score, out_stride, out_cols, kv_len, out_len, batch, budget, sinks,
                      recent, out_kept, in_place, workspace, sms,
                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

size_t spec_logprobs_workspace_size(int64_t rows) {
  return rows < 0 || rows >= INT_MAX ? 0 : logprobs_workspace_bytes(rows);
}

// Logits that may start at any element.
static int logprobs_check(const sv_logits* logits) {
  if (!logits) return SV_ERR_ARG;
  const sv_logits& x = *logits;
  if (x.dtype != SV_F32 && x.dtype != SV_BF16) return SV_ERR_UNSUPPORTED;
  if (x.vocab < 1 || x.rows < 0 || x.rows >= INT_MAX || (x.rows > 1 && x.row_stride < x.vocab))
    return SV_ERR_ARG;
  if (x.vocab > SV_VOCAB_MAX) return SV_ERR_UNSUPPORTED;
  if (x.rows > 0 && !x.data) return SV_ERR_ARG;
  if (misaligned(x.data, elem_size(x.dtype))) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

int spec_logprobs(const sv_logits* logits, const int32_t* tokens, const float* temperature,
                  int32_t n_top, float* out_logprob, float* out_entropy, float* out_max,
                  float* out_logsum, int32_t* out_top_tokens, float* out_top_logprobs,
                  void* stream, void* workspace, size_t workspace_bytes) {
  if (int rc = logprobs_check(logits)) return rc;
  if (n_top < 0) return SV_ERR_ARG;
  if (n_top > SV_LOGPROBS_TOP_MAX) return SV_ERR_UNSUPPORTED;
  if (n_top > 0 && logits->rows > 0 && (!out_top_tokens || !out_top_logprobs)) return SV_ERR_ARG;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < logprobs_workspace_bytes(logits->rows))
    return SV_ERR_WORKSPACE;
  if (logits->rows == 0) return SV_OK;
  const int sms = sm_count();
  if (sms == 0) return SV_ERR_CUDA;
  return launch_logprobs(*logits, tokens, temperature, n_top, out_logprob, out_entropy, out_max,
                         out_logsum, out_top_tokens, out_top_logprobs, workspace, sms,
                         g_expire_wait.load(std::memory_order_relaxed),
                         static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

int spec_logprobs_grad(const sv_logits* logits, const int32_t* tokens, const float* temperature,
                       const float* max, const float* logsum, const float* entropy,
                       const float* g_logprob, const float* g_entropy, void* out,
                       int64_t out_stride, void* stream) {
  if (int rc = logprobs_check(logits)) return rc;
  if (logits->rows > 1 && out_stride < logits->vocab) return SV_ERR_ARG;
  if (logits->rows == 0) return SV_OK;
  if (!tokens || !max || !logsum || (g_entropy && !entropy) || !out) return SV_ERR_ARG;
  if (misaligned(out, elem_size(logits->dtype))) return SV_ERR_UNSUPPORTED;
  // one buffer has one row stride
  if (out == logits->data && logits->rows > 1 && out_stride != logits->row_stride)
    return SV_ERR_ARG;
  if (logprobs_grad_blocks(*logits) > INT_MAX) return SV_ERR_UNSUPPORTED;
  return launch_logprobs_grad(*logits, tokens, temperature, max, logsum, entropy, g_logprob,
                              g_entropy, out, out_stride,
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

int spec_verify_get_error(const void* workspace, void* stream, int32_t* code, int32_t* request,
                          int64_t* row) {
  if (!workspace || !code) return SV_ERR_ARG;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SV_ERR_CUDA;
  WsHeader h;
  if (cudaMemcpy(&h, workspace, sizeof h, cudaMemcpyDeviceToHost) != cudaSuccess)
    return SV_ERR_CUDA;
  if (h.err_code == kStatusList) {
    // one status per row or request: the lowest that failed
    if (h.err_row < 0 || h.err_row > INT_MAX || h.n_active < 0) return SV_ERR_INTERNAL;
    const size_t n = size_t(h.err_row), extra = size_t(h.n_active);
    std::vector<int32_t> st;
    try {
      st.resize(n + extra);
    } catch (...) {
      return SV_ERR_INTERNAL;
    }
    if (!st.empty() &&
        cudaMemcpy(st.data(), static_cast<const char*>(workspace) + align256(sizeof(WsHeader)),
                   st.size() * sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
      return SV_ERR_CUDA;
    size_t at = 0;
    while (at < n && st[at] == 0) ++at;
    int32_t c = at < n ? st[at] : 0;
    if (at == n) at = INT32_MAX;   // none: as the entries that follow say it
    const size_t trees = h.err_req == 2 ? n + extra / 2 : n + extra;
    for (size_t i = n; i < n + extra; ++i)
      if (st[i] < 0) {  // a CTA's failure, no request's
        *code = -st[i];
        if (request) *request = -1;
        if (row) *row = -1;
        return SV_OK;
      } else if (size_t(st[i]) < at) {
        at = size_t(st[i]);
        c = i < trees ? SV_ERR_DATA_PAGE : SV_ERR_DATA_TREE;
      }
    *code = c;
    if (request) *request = c && h.err_req ? int32_t(at) : -1;
    if (row) *row = c && !h.err_req ? int64_t(at) : -1;
    return SV_OK;
  }
  *code = h.err_code;
  if (request) *request = h.err_req;
  if (row) *row = h.err_row;
  return SV_OK;
}

int spec_verify_dump_rows(const void* workspace, size_t workspace_bytes, int32_t batch,
                          int64_t target_rows, int64_t draft_rows, void* stream, double* stats,
                          int32_t* kept_count, int32_t* kept_idx, double* kept_p) {
  if (!workspace || batch < 0 || target_rows < 0 || draft_rows < 0) return SV_ERR_ARG;
  const WsLayout L = ws_layout(batch, target_rows, draft_rows);
  if (workspace_bytes < L.total) return SV_ERR_WORKSPACE;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SV_ERR_CUDA;
  const char* base = static_cast<const char*>(workspace);
  const size_t R = size_t(target_rows + draft_rows);
  if (R == 0) return SV_OK;
  if (stats || kept_count) {
    std::vector<RowStat> st(R);
    if (cudaMemcpy(st.data(), base + L.off_stats, R * sizeof(RowStat), cudaMemcpyDeviceToHost) !=
        cudaSuccess)
      return SV_ERR_CUDA;
    // the kept-set thresholds of kBig rows (slot 0 of each row's survivors)
    std::vector<uint64_t> th(R, 0ull);
    for (size_t r = 0; r < R; ++r)
      if (st[r].mode == kBig &&
          cudaMemcpy(&th[r], base + L.off_raw + r * kRawCap * sizeof(uint64_t), sizeof(uint64_t),
                     cudaMemcpyDeviceToHost) != cudaSuccess)
        return SV_ERR_CUDA;
    for (size_t r = 0; r < R; ++r) {
      if (stats) {
        stats[5 * r + 0] = st[r].m;
        stats[5 * r + 1] = st[r].s;
        stats[5 * r + 2] = st[r].pg;
        stats[5 * r + 3] = st[r].arg;
        // the last kept token of a threshold-filtered row: ~ the key's low word
        stats[5 * r + 4] = st[r].mode == kBig ? double(int32_t(~uint32_t(th[r]))) : -1.0;
      }
      if (kept_count) kept_count[r] = (st[r].mode == kTopk || st[r].mode == kBig) ? st[r].kept : 0;
    }
  }
  if (kept_idx && cudaMemcpy(kept_idx, base + L.off_cidx, R * kTopkMax * sizeof(int32_t),
                             cudaMemcpyDeviceToHost) != cudaSuccess)
    return SV_ERR_CUDA;
  if (kept_p) {
    std::vector<float> kp(R * kTopkMax);
    if (cudaMemcpy(kp.data(), base + L.off_cp, R * kTopkMax * sizeof(float),
                   cudaMemcpyDeviceToHost) != cudaSuccess)
      return SV_ERR_CUDA;
    for (size_t i = 0; i < kp.size(); ++i) kept_p[i] = kp[i];
  }
  return SV_OK;
}

const char* spec_verify_strerror(int code) {
  switch (code) {
    case SV_OK: return "ok";
    case SV_ERR_ARG: return "invalid argument";
    case SV_ERR_UNSUPPORTED: return "unsupported dtype, vocabulary size, alignment or stride";
    case SV_ERR_CUDA: return "CUDA runtime error";
    case SV_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case SV_ERR_DATA_K: return "k_per_req outside [0, SV_MAX_K]";
    case SV_ERR_DATA_TEMPERATURE: return "temperature negative, NaN or infinite";
    case SV_ERR_DATA_TOP_P: return "top_p outside (0, 1]";
    case SV_ERR_DATA_TOP_K: return "top_k negative";
    case SV_ERR_DATA_TOKEN: return "draft token outside [0, V)";
    case SV_ERR_DATA_ROWS: return "row counts do not match k_per_req";
    case SV_ERR_DATA_LOGIT: return "NaN or +inf logit, or a sampled row without a finite logit";
    case SV_ERR_DATA_NO_DRAFT: return "temperature > 0 without draft logits";
    case SV_ERR_TIMEOUT: return "internal bounded wait expired";
    case SV_ERR_INTERNAL: return "internal capacity invariant failed";
    case SV_ERR_DATA_ACCEPT: return "KV commit: accept length above k";
    case SV_ERR_DATA_PAGE: return "a page missing from the block table, or negative kv_len";
    case SV_ERR_DATA_LENGTH: return "kv_len negative, or past the block table or the scores";
    case SV_ERR_DATA_TREE: return "a tree's parent that is no earlier node, or a path without one";
    case SV_ERR_DATA_POOL: return "too few free pages, or a free list that cannot hold them";
    default: return "unknown status";
  }
}

int spec_verify_version(void) { return 100; }

}  // extern "C"
