// Greedy verification of a tree of drafts from the target rows' argmax.
//
// Node 0 of a request is its last emitted token, nodes 1 .. k are drafts, each
// hanging from an earlier node.  From node 0 on, the walk goes to the child whose
// token is the target's argmax at the node (the lowest such child) until there is
// none; the tokens on the way and the argmax at its last node are emitted.  It is
// the rule of a chain ("DFlash" §4 step 5; "Speculative decoding and multi-token
// prediction", "Draft and verify", step Three) on the branch that the target takes.
//
// A warp has a request: a lane holds nodes `lane` and `lane + 32`, so a step of the
// walk is two ballots and one shuffle.  Every CTA adds up the rows of the requests
// before its own by itself (and checks the batch on the way), which takes one
// launch instead of two.  Latency is what counts: 8 requests 2.5 us of the GPU,
// 4096 with up to 63 drafts, 2.6 MB in and out, 6.8 us.
#include "sv_internal.cuh"

namespace sv {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeWarps = kTreeThreads / 32;

struct TreeProblem {
  const int32_t *argmax, *draft_tokens, *parent, *k_per_req;
  int32_t *accept_len, *tokens, *path;
  int32_t B, V;
  int64_t Rt;
  WsHeader* hdr;
  int32_t* status;   // [B]
};

__global__ void __launch_bounds__(kTreeThreads) tree_greedy_kernel(const TreeProblem Q) {
  __shared__ int s_before[kTreeWarps], s_total[kTreeWarps], s_k[kTreeWarps];
  __shared__ int s_badk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b0 = blockIdx.x * kTreeWarps, b = b0 + warp;
  if (tid == 0) s_badk = INT32_MAX;
  __syncthreads();
  // rows of the requests before this CTA's, and of all
  int before = 0, total = 0;
#pragma unroll 4
  for (int i = tid; i < Q.B; i += kTreeThreads) {
    const int k = Q.k_per_req[i];
    if (k < 0 || k > SV_TREE_MAX_K) {
      atomicMin(&s_badk, i);
      continue;
    }
    total += k + 1;
    if (i < b0) before += k + 1;
    if (i >= b0 && i < b0 + kTreeWarps) s_k[i - b0] = k;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) {
    s_before[warp] = before;
    s_total[warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kTreeWarps; ++w) {
    before += s_before[w];
    total += s_total[w];
  }
  if (blockIdx.x == 0 && tid == 0) {
    Q.hdr->err_code = kStatusList;
    Q.hdr->err_row = Q.B;
    Q.hdr->err_req = 1;   // entries are requests
    Q.hdr->n_active = 0;
  }
  const int code = s_badk != INT32_MAX ? SV_ERR_DATA_K : total != Q.Rt ? SV_ERR_DATA_ROWS : 0;
  if (code) {   // requests cannot be told apart
    const int code_b = code == SV_ERR_DATA_K ? s_badk : 0;
    if (b < Q.B && lane == 0) {
      Q.status[b] = b == code_b ? code : 0;
      Q.accept_len[b] = -1;
    }
    for (int64_t i = int64_t(blockIdx.x) * kTreeThreads + tid; i < Q.Rt;
         i += int64_t(gridDim.x) * kTreeThreads)
      Q.tokens[i] = Q.path[i] = -1;
    return;
  }
  if (b >= Q.B) return;
  int64_t t0 = before;
  for (int w = 0; w < warp; ++w) t0 += s_k[w] + 1;
  const int n = s_k[warp] + 1;
  // the lane's nodes
  int best[2], parent[2], token[2];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    best[i] = token[i] = -1;
    parent[i] = -2;
    if (j >= n) continue;
    best[i] = Q.argmax[t0 + j];
    bad |= best[i] < 0 || best[i] >= Q.V;
    if (j == 0) continue;
    parent[i] = Q.parent[t0 + j];
    token[i] = Q.draft_tokens[t0 - b + j - 1];
    bad |= token[i] < 0 || token[i] >= Q.V;
  }
  bool torn = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    torn |= j > 0 && j < n && (parent[i] < 0 || parent[i] >= j);
  }
  bad = __any_sync(0xffffffffu, bad);
  torn = __any_sync(0xffffffffu, torn);
  // what the lane's places of the path hold
  int path[2] = {-1, -1}, emit[2] = {-1, -1}, L = -1;
  if (!bad && !torn) {
    int cur = 0;
    for (;;) {
      ++L;
      const int want = __shfl_sync(0xffffffffu, cur < 32 ? best[0] : best[1], cur & 31);
      if ((L & 31) == lane) {
        path[L >> 5] = cur;
        emit[L >> 5] = want;
      }
      const uint32_t lo = __ballot_sync(0xffffffffu, parent[0] == cur && token[0] == want);
      const uint32_t hi = __ballot_sync(0xffffffffu, parent[1] == cur && token[1] == want);
      if (!(lo | hi)) break;
      cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);   // a child comes behind its parent: it ends
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    if (j >= n) continue;
    Q.path[t0 + j] = path[i];
    Q.tokens[t0 + j] = emit[i];
  }
  if (lane == 0) {
    Q.accept_len[b] = L;
    Q.status[b] = torn ? SV_ERR_DATA_TREE : bad ? SV_ERR_DATA_TOKEN : 0;
  }
}

}  // namespace

size_t tree_greedy_workspace_bytes(int32_t B) {
  return align256(sizeof(WsHeader)) + align256(sizeof(int32_t) * size_t(B > 0 ? B : 1));
}

cudaError_t launch_tree_greedy(const int32_t* argmax, const int32_t* draft_tokens,
                               const int32_t* parent, const int32_t* k_per_req,
                               int32_t* accept_len, int32_t* tokens, int32_t* path, int B,
                               int64_t Rt, int V, void* workspace, cudaStream_t s) {
  TreeProblem Q;
  Q.argmax = argmax;
  Q.draft_tokens = draft_tokens;
  Q.parent = parent;
  Q.k_per_req = k_per_req;
  Q.accept_len = accept_len;
  Q.tokens = tokens;
  Q.path = path;
  Q.B = B;
  Q.V = V;
  Q.Rt = Rt;
  Q.hdr = static_cast<WsHeader*>(workspace);
  Q.status = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(sizeof(WsHeader)));
  tree_greedy_kernel<<<(B + kTreeWarps - 1) / kTreeWarps, kTreeThreads, 0, s>>>(Q);
  return cudaGetLastError();
}

}  // namespace sv
