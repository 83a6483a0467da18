// Attention with many query rows a KV head on the fifth-generation tensor cores, for
// bf16 and fp16: causal over packed prompts, and over the paged cache where trees of
// drafts bring more rows than one product has.  Heads of up to 256 elements (trees: 64
// to 128) that lie on 16 bytes, taken at D, the next of 64, 128 and 256; what lies
// behind a prompt's head is filled with zeros by the copy engine.
//
// A row tile is 128 / G tokens (nodes of a tree) of one KV head with the G query heads
// that share it, the M of the products: row r is token r / G, head r % G, and the rows
// of a tile are one box of the copy engine.  A unit is NQ row tiles that follow one
// another (two, one for heads of 256, whose output takes half of TMEM) over the
// tiles of TN positions that they see: S = Q K^T (128 x TN x D), P = exp S, O += P V
// (128 x D x TN).  With two row tiles one's softmax runs during the other's
// products, and every tile of K and V serves both.
//
// One CTA per SM, over units u = c, 2 n - 1 - c, 2 n + c, ... (n CTAs, forth and back)
// in the order of the tokens' place in their sequence, the last first: what a unit
// costs falls with its number, so that the CTAs' sums stay close without a queue (24
// sequences of 1 to 4000 tokens, 11978 in all: the most 86 tiles a CTA, the mean 82).  Trees: over its
// piece of the line of tiles, as sv_attn_tc_kernel.cuh has it; what a unit leaves in
// several CTAs is joined by a second kernel.
//   warps 0-3, 4-7  softmax of the first and the second row tile, one row a thread
//                   (the lanes of TMEM): scores from TMEM, running maximum, P rounded
//                   to the type (half a step of it, the one rounding of a weight;
//                   sums stay in 32 bits) back over the scores, where the second
//                   product reads it as its A operand.  O is rescaled only when a
//                   row's maximum has grown by more than 2^8 since the last time.
//   warp 8          finds the units, announces them, and has the copy engine load Q,
//                   K and V into rings of slots, 128-byte swizzled (of a cache, V by
//                   warp 10, tiles that are not whole by 16-byte copies: load_tile).
//   warp 9          issues the products.  The tensor cores run them in the order of
//                   issue, so that S of the next tile may follow the product that
//                   reads P in the same place.  A warp for each row tile instead, with
//                   or without turns, 1350 us -> 1480 to 1680 on the case below: their
//                   products come between one another's.
//   warps 10, 11    (trees: 11; 10 loads V) look through V of the tiles that some row of
//                   the unit sees in part: masked weights are 0, but 0 times an infinite
//                   or NaN value would still reach the row.  If such a tile holds any,
//                   each row collects the signs of those that it sees, they are replaced
//                   by 0, and added to the row's O afterwards.  (A weight that is 0 in the
//                   type, more than 2^126 below its row's largest, 2^31 in fp16, times
//                   an infinite value in any other tile is NaN.)
//
// Every wait is bounded; on expiry the CTA's status records it, its copies and
// products land, TMEM is freed, and the rows of all its units become NaN.
//
// Measured, prompts, 32 + 8 heads of 128 in bf16: 16001 tokens 1.31 ms, 1600 TFLOP/s of
// what the visible pairs take; 4 times 2048 tokens 110 us, 1250; 201 tokens 11 us.  Heads
// of 64 985 TFLOP/s, of 256 1300 (8 to 16 thousand tokens).  Bound by a row tile's round:
// softmax 1200 to 1300 cycles, products 1050, and about 600 from barrier to barrier,
// 2950 where the products of both row tiles take 2050; then by a unit's end (its last
// product, 2500 cycles of output, the next unit's first scores: 6000 in all).  Heads of
// 64: a product with V takes as long for 64 columns as for 128.  Every wait is a small
// loop: unrolled, the kernel's 260 KB of instructions cost 5 to 9 %.
// Trees, 32 requests of 2001 to 8190 positions with 8 to 63 drafts, the same heads: 127 us,
// 4.9 TB/s of their entries; 8 of 30000 with 63 drafts 184 us, 5.3.  Bound by the row
// tiles' rounds: a tile of 128 positions of both takes 3500 cycles, 2050 of them products
// (pages of 128 instead of 16 positions, boxes 8 times as large, change nothing; entries
// that the L2 holds, 5 %).  Loads of K and V by the same instructions, and what is rare
// out of line, 149 -> 138 us: the tensor cores' warp waits for instructions otherwise.
#pragma once

#include <type_traits>

#include "sv_attn_tc.cuh"
#include "sv_prompt.cuh"

namespace sv {
namespace {

constexpr int kPtThreads = 384;
// the last warp and, of prompts, the one before look through V; of trees that one loads it
constexpr int kLoadWarp = 8, kMmaWarp = 9, kValueWarp = 10, kLastWarp = 11;
constexpr int kM = 128;
constexpr int kSegs = 4;          // units announced ahead of the warp that is furthest back
constexpr float kRescaleLog2 = 8.0f;
constexpr uint32_t kTmemCols = 512;
// Registers a thread: of the launch, of the softmax warps, of the others (three
// warpgroups share 3 x 168).
constexpr int kSoftmaxRegs = 192, kOtherRegs = 120;

template <int D>
struct PtShape {
  static constexpr int NQ = D == 256 ? 1 : 2;         // row tiles of a unit
  static constexpr int TN = D == 256 ? 64 : 128;      // positions of a tile
  static constexpr int NB = D == 256 ? 2 : 1;         // S accumulators of a row tile
  static constexpr int kQBytes = kM * D * 2;
  static constexpr int kSlotBytes = TN * D * 2;
  static constexpr int kSlots = D == 64 ? 10 : 5;     // what shared memory holds
  static constexpr int kKSlots = kSlots / 2;          // of K; the rest are of V
  static constexpr uint32_t kOCol = 256;              // S accumulators, then O
  static constexpr size_t kSmem = 1024 + size_t(NQ) * kQBytes + size_t(kSlots) * kSlotBytes;
};

// One unit, or a CTA's part of it.  The load warp finds them, a few ahead, and
// announces them to the others; n 0 is the end.
struct PtSeg {
  int row0;       // first row of the sequence (request)
  int h;          // KV head
  int tok0;       // first token
  int tile0, n;   // tiles of positions
  int cnt[2];     // of them what each row tile sees, from the first on
  int live[2];    // tokens of each row tile
  int all_lo, all_hi;   // positions that every row sees
};
struct PtTreeSeg : PtSeg {
  int b, first;         // request; the part's first tile among the unit's
  bool whole;
  int64_t unit_end;     // tile of the line after the unit's last
  AttnReq R;
};

template <bool TREE>
struct PtShared {
  std::conditional_t<TREE, PtTreeSeg, PtSeg> seg[kSegs];
  uint64_t announced[kSegs], taken[kSegs];   // taken: no warp needs the entry any more
  uint64_t noted[kSegs];            // trees: every page of the part was looked at
  uint64_t full[10], empty[10];
  uint64_t looked[10], clean[10];   // of V slots: looked through; nothing to be kept out
  uint64_t qfull[2], qempty[2], ofree[2];
  // Per S accumulator: with two, a warp may be a tile ahead of another, and a tile's
  // product two tiles behind the scores, whose barriers' parities would be alike.
  uint64_t sfull[2][2], pfull[2][2], pvdone[2][2];
  uint64_t collected[2];            // the row tile has the signs of a dirty tile
  uint64_t drain, never;
  int dirty[10][2];                 // per V slot and looking warp
  int copied[10];                   // trees, per slot: filled by copies of the lanes
  int part_bad[kSegs];              // trees: the part fails
  int first_bad, first_torn;        // first request with a missing page, with a bad parent
  uint32_t tmem;
  int abort, bad, top;
};

// The units of a CTA, found by a whole warp.
template <int NQ>
struct PtWalk {
  int span;            // tokens of a unit
  int64_t u, step0, step1, base;   // unit number, the two strides in turn; units before the level
  // The level: units that begin at token level * span of their sequence.  cnt sequences have
  // one, those with more than `level` units; so it is down to level `same`.
  int level, cnt, same;
  __device__ __forceinline__ int units(const PromptArgs& A, int b) const {
    if (b >= A.B) return 0;
    int first, len;
    prompt_sequence(A, b, &first, &len);
    return (len + span - 1) / span;
  }
  __device__ __forceinline__ void look(const PromptArgs& A) {
    const int lane = threadIdx.x & 31;
    cnt = same = 0;
    for (int b = 0; b < A.B; b += 32) {
      const int n = units(A, b + lane);
      cnt += __popc(__ballot_sync(0xffffffffu, n > level));
      same = max(same, __reduce_max_sync(0xffffffffu, n > level ? 0 : n));
    }
  }
  // top: units of the longest sequence
  __device__ __forceinline__ PtWalk(const PromptArgs& A, int top)
      : span(NQ * (kM / A.G)), u(blockIdx.x), step0(2 * int64_t(gridDim.x) - 1 - 2 * blockIdx.x),
        step1(1 + 2 * int64_t(blockIdx.x)), base(0), level(top - 1), cnt(0), same(0) {
    if (level >= 0) look(A);
  }
  template <int TN>
  __device__ __forceinline__ bool next(const PromptArgs& A, PtSeg& s) {
    s.n = 0;
    while (level >= 0) {
      const int64_t each = int64_t(cnt) * A.Hkv, off = (u - base) / each;
      const int down = int(min(off, int64_t(level - same + 1)));
      if (down == 0) break;
      base += down * each;
      level -= down;
      if (level >= 0 && level < same) look(A);
    }
    if (level < 0) return false;
    const int local = int(u - base), lane = threadIdx.x & 31;
    int rank = local / A.Hkv, b = 0;
    for (int b0 = 0;; b0 += 32) {
      const uint32_t has = __ballot_sync(0xffffffffu, units(A, b0 + lane) > level);
      const int c = __popc(has);
      if (rank < c) {
        b = b0 + int(__fns(has, 0, rank + 1));
        break;
      }
      rank -= c;
    }
    int len;
    prompt_sequence(A, b, &s.row0, &len);
    s.h = local % A.Hkv;
    s.tok0 = level * span;
    s.tile0 = (A.window > 0 ? max(0, s.tok0 - A.window + 1) : 0) / TN;
    s.all_hi = s.tok0 + 1;
    s.all_lo = A.window > 0 ? max(0, min(s.tok0 + span, len) - A.window) : 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int first = s.tok0 + g * (kM / A.G);
      s.live[g] = g < NQ ? max(0, min(kM / A.G, len - first)) : 0;
      s.cnt[g] = s.live[g] ? (first + s.live[g] - 1) / TN + 1 - s.tile0 : 0;
      s.n = max(s.n, s.cnt[g]);
    }
    u += step0;
    const int64_t x = step0;
    step0 = step1;
    step1 = x;
    return true;
  }
};


// What a unit of a tree costs beside its tiles, in tiles (sv_attn_tc_kernel.cuh).
constexpr int kTreePad = 4;

// The parts of a CTA's piece of the line of tiles, units of 256 rows of a KV head.
template <int TN>
struct PtTreeWalk {
  int64_t pos, end, base;
  int b, t_off;
  AttnReq R;
  __device__ __forceinline__ PtTreeWalk(const AttnArgs& A, const AttnPlan& P)
      : pos(P.start), end(P.end), base(P.base), b(P.b), t_off(P.t_off) {
    if (pos < end) R = attn_request<TN, 2 * kM, false>(A, b);
  }
  __device__ __forceinline__ bool next(const AttnArgs& A, PtTreeSeg& s) {
    s.n = 0;
    if (pos >= end) return false;
    int unit;
    for (;;) {
      int64_t nt = attn_tiles<TN, 2 * kM, false, kTreePad>(A, R);
      while (pos >= base + nt) {
        base += nt;
        t_off += R.k + 1;
        R = attn_request<TN, 2 * kM, false>(A, ++b);
        nt = attn_tiles<TN, 2 * kM, false, kTreePad>(A, R);
      }
      const int64_t local = pos - base;
      const int span = R.ntiles + kTreePad, at = int(local % span);
      unit = int(local / span);
      if (at >= kTreePad) {
        s.first = at - kTreePad;
        break;
      }
      pos += kTreePad - at;   // a unit's tiles come behind what it costs itself
      if (pos >= end) return false;
    }
    const int64_t left = end - pos;
    const int toks = kM / A.G;
    s.b = b;
    s.row0 = t_off;
    s.n = int(left < R.ntiles - s.first ? left : R.ntiles - s.first);
    s.h = unit / R.mtiles * A.hg + int(blockIdx.x) % A.hg;
    s.tok0 = unit % R.mtiles * 2 * toks;
    s.tile0 = R.tile0 + s.first;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      s.live[g] = max(0, min(toks, R.k + 1 - s.tok0 - g * toks));
      s.cnt[g] = s.live[g] ? s.n : 0;
    }
    // a tree is no deeper than its nodes are many
    s.all_hi = R.code ? 0 : R.n;
    s.all_lo = A.window > 0 ? max(0, R.n + R.k - A.window + 1) : 0;
    s.whole = s.first == 0 && s.n == R.ntiles;
    s.unit_end = pos - s.first + R.ntiles;
    s.R = R;
    pos += s.n;
    return true;
  }
};

// The unit that the CTA begins with s ends in a later one: the join's record of it.
__device__ __forceinline__ void pt_begin_split(const AttnArgs& A, const AttnPlan& P,
                                               const PtTreeSeg& s) {
  AttnSplit& u = A.split[blockIdx.x];
  u.last = attn_owner(A, P, s.unit_end - 1);
  u.t_off = s.row0;
  u.h = s.h;
  u.row0 = s.tok0 * A.G;
  u.rows = (s.live[0] + s.live[1]) * A.G;
  u.valid = 1;
}

__device__ __forceinline__ void box_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Descriptor of an MN-major 16-bit tile with 128-byte swizzling: rows (of K)
// of 128 bytes, 8-row groups 1024 bytes apart, blocks of 64 elements of MN
// `block` bytes apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t block) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(block >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

template <class Sh, class Seg>
__device__ __forceinline__ bool pt_next_seg(Sh& S, int unit, Seg& s) {
  if (!tc_wait_warp(&S.announced[unit % kSegs], (unit / kSegs) & 1, S)) return false;
  s = S.seg[unit % kSegs];
  __syncwarp();
  return s.n > 0;
}
// The warp needs the unit's entry no more.
template <class Sh>
__device__ __forceinline__ void pt_taken(Sh& S, int unit) {
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&S.taken[unit % kSegs]));
}

// Four lanes exchange 16-byte pieces: w[i], the lane's piece i, becomes the piece of
// this lane's number of the i-th lane of the four.
__device__ __forceinline__ void exchange4(uint32_t (&w)[4][4]) {
  const int piece = threadIdx.x & 3;
#pragma unroll
  for (int step = 1; step < 4; step <<= 1) {
    const bool up = piece & step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & step) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t give = up ? w[i][e] : w[i | step][e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, step);
        if (up) w[i][e] = got;
        else w[i | step][e] = got;
      }
    }
  }
}

// A thread's row of O where it does not lie on 16 bytes; none where out is null.
template <class T>
__device__ __noinline__ void rows_one_by_one(uint32_t o_at, int dim, float inv, T* out) {
#pragma unroll 1
  for (int c = 0; c * 16 < dim; ++c) {
    uint32_t o[16];
    tmem_ld16(o_at + c * 16, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (out && c * 16 + e < dim) out[c * 16 + e] = from_float<T>(__uint_as_float(o[e]) * inv);
  }
}

// All threads, after a wait of the CTA expired and every warp has left its loop:
// what was issued has landed; every row of the CTA's units becomes NaN, and what the
// join makes of them with other CTAs' parts.
template <class T, int D>
__device__ __noinline__ void pt_give_up(const PromptArgs& A, int top) {
  using C = PtShape<D>;
  const float nan = __int_as_float(0x7fc00000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PtWalk<C::NQ> walk(A, top);
  PtSeg s;
  while (walk.template next<C::TN>(A, s)) {
    const int rows = (s.live[0] + s.live[1]) * A.G;
    for (int r = warp; r < rows; r += kPtThreads / 32) {
      const int64_t to = (int64_t(s.row0) + s.tok0 + r / A.G) * A.Hq + s.h * A.G + r % A.G;
      T* out = static_cast<T*>(A.out) + to * A.D;
      for (int d = lane; d < A.D; d += 32) out[d] = from_float<T>(nan);
      if (lane == 0) A.lse[to] = nan;
    }
  }
}
template <class T, int D>
__device__ __noinline__ void pt_give_up(const AttnArgs& A, int) {
  using C = PtShape<D>;
  const float nan = __int_as_float(0x7fc00000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnPlan P = attn_plan<C::TN, 2 * kM, false, kPtThreads, kTreePad>(A);
  PtTreeWalk<C::TN> walk(A, P);
  PtTreeSeg s;
  while (walk.next(A, s)) {
    const int rows = (s.live[0] + s.live[1]) * A.G;
    for (int r = warp; r < rows; r += kPtThreads / 32) {
      const int64_t to = (int64_t(s.row0) + s.tok0 + r / A.G) * A.Hq + s.h * A.G + r % A.G;
      T* out = static_cast<T*>(A.out) + to * A.D;
      for (int d = lane; s.whole && d < A.D; d += 32) out[d] = from_float<T>(nan);
      if (lane != 0) continue;
      if (s.whole) A.lse[to] = nan;
      else A.part_ml[(int64_t(blockIdx.x) * 2 + (s.first == 0)) * 2 * kM + r] =
               make_float2(nan, 0.f);
    }
    if (threadIdx.x == 0 && !s.whole && s.first == 0) pt_begin_split(A, P, s);
  }
}

// Args: PromptArgs or, of trees, AttnArgs, whose cache is k_map and v_map alike.
template <class T, int D, bool PART, class Args>
__global__ void __launch_bounds__(kPtThreads, 1)
    row_tiles_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map,
                        const __grid_constant__ Args A) {
  using C = PtShape<D>;
  constexpr bool TREE = std::is_same_v<Args, AttnArgs>;
  constexpr int kLooks = TREE ? 1 : 2;   // warps that look through V
  using Seg = std::conditional_t<TREE, PtTreeSeg, PtSeg>;
  constexpr int TN = C::TN, NQ = C::NQ, NB = C::NB;
  constexpr int kSlotBytes = C::kSlotBytes;
  extern __shared__ unsigned char pt_smem_raw[];
  __shared__ PtShared<TREE> S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_addr(pt_smem_raw) + 1023u) & ~1023u;
  unsigned char* smem_p = pt_smem_raw + (smem0 - smem_addr(pt_smem_raw));
  const uint32_t ring0 = smem0 + NQ * C::kQBytes;
  const int dim = PART ? A.D : D;
  const int parts = PART ? (A.D + 63) / 64 : D / 64;
  const int toks = kM / A.G;

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_addr(&S.full[i]), TREE ? 32 : 1);   // lanes of the load warp
      mbar_init(smem_addr(&S.empty[i]), 1);
      mbar_init(smem_addr(&S.looked[i]), kLooks);
      mbar_init(smem_addr(&S.clean[i]), kLooks);
      S.dirty[i][0] = S.dirty[i][1] = 0;
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_addr(&S.qfull[g]), 1);
      mbar_init(smem_addr(&S.qempty[g]), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_addr(&S.sfull[g][i]), 1);
        mbar_init(smem_addr(&S.pfull[g][i]), 4);
        mbar_init(smem_addr(&S.pvdone[g][i]), 1);
      }
      mbar_init(smem_addr(&S.ofree[g]), 4);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(smem_addr(&S.announced[i]), 1);
      mbar_init(smem_addr(&S.noted[i]), 1);
      mbar_init(smem_addr(&S.taken[i]), 4 * NQ + 3);   // every warp but the load warp
    }
    for (int g = 0; g < 2; ++g) mbar_init(smem_addr(&S.collected[g]), 4);
    mbar_init(smem_addr(&S.drain), 1);
    mbar_init(smem_addr(&S.never), 1);
    fence_mbar_init();
    S.abort = S.bad = S.top = 0;
    S.first_bad = S.first_torn = INT32_MAX;
    if constexpr (TREE) A.split[blockIdx.x].valid = 0;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&S.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncthreads();
  AttnPlan P{};
  if constexpr (TREE) {
    P = attn_plan<TN, 2 * kM, false, kPtThreads, kTreePad>(A);
  } else {   // the sequences, looked through by every CTA
    int top = 0;
    bool bad = false;
    for (int b = tid; b < A.B; b += kPtThreads) {
      int first, len;
      bad |= !prompt_sequence(A, b, &first, &len);
      top = max(top, (len + NQ * toks - 1) / (NQ * toks));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (top > 0) atomicMax(&S.top, top);
      if (bad) S.bad = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  bool go;
  if constexpr (TREE) {
    go = P.code == 0 && P.start < P.end;
    if (P.code) fail_all<T>(A);
  } else {
    go = S.bad == 0;
    if (!go) prompt_fail<T>(A);
  }

  if (go && warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp || (TREE && warp == kValueWarp)) {
      // ------------------------------------------------------- units and loads
      // (of trees one warp loads K, the other V, by the same instructions)
      const bool leads = warp == kLoadWarp;
      const int kv = leads ? 0 : 1;
      Ring kr(kv ? C::kKSlots : 0, kv ? C::kSlots - C::kKSlots : C::kKSlots, 1);
      Ring vr(C::kKSlots, C::kSlots - C::kKSlots, 1);   // of prompts
      int kfilled = 0, vfilled = 0, quse[2] = {0, 0};
      bool stop = false;
      const uint32_t lead = lane == 0;
      auto walk = [&] {
        if constexpr (TREE) return PtTreeWalk<TN>(A, P);
        else return PtWalk<NQ>(A, S.top);
      }();
      Seg next;
      auto find = [&] {
        if constexpr (TREE) walk.next(A, next);
        else walk.template next<TN>(A, next);
      };
      find();
      for (int unit = 0;; ++unit) {
        Seg s;
        if (leads) {
          s = next;
          stop = !tc_wait_warp(&S.taken[unit % kSegs], ((unit / kSegs) & 1) ^ 1, S);
          if (stop) break;
          if (lead) {
            S.seg[unit % kSegs] = s;
            if constexpr (TREE) S.part_bad[unit % kSegs] = s.n && s.R.code != 0;
            mbar_arrive(smem_addr(&S.announced[unit % kSegs]));
          }
          __syncwarp();
          if (s.n == 0) break;
#pragma unroll
          for (int g = 0; g < NQ; ++g) {
            if (s.cnt[g] == 0 || stop) continue;
            stop = !tc_wait_warp(&S.qempty[g], (quse[g] & 1) ^ 1, S);
            quse[g] += !stop;
            if (lead && !stop) {
              const uint32_t bar = smem_addr(&S.qfull[g]);
              mbar_arrive_expect_tx(bar, uint32_t(parts * toks * A.G * 128));
              for (int p = 0; p < parts; ++p)
                box_load3(smem0 + g * C::kQBytes + p * (kM * 128), &q_map, p * 64, s.h * A.G,
                          s.row0 + s.tok0 + g * toks, bar);
            }
            __syncwarp();
          }
        } else if (!pt_next_seg(S, unit, s)) {
          break;
        }
        if constexpr (TREE) {
          const int hi = s.R.code ? 0 : s.R.hi, cached = min(s.R.n, hi);
          const int32_t* table = A.table + int64_t(s.b) * A.max_pages;
          // keys that no other unit of the call reads leave the L2 first
          const uint64_t policy =
              s.R.mtiles > 1 ? l2_evict_normal_policy() : l2_evict_first_policy();
          auto missing = [&](int page) {
            if (page >= 0 && page < A.num_pages) return false;
            S.part_bad[unit % kSegs] = 1;
            atomicMin(&S.first_bad, s.b);
            return true;
          };
          // pages are read one tile ahead, so that nothing waits for the block table
          TilePages<TN, 1> ahead = tile_pages<D, PART, TN>(A, table, cached, s.tile0 * TN);
          for (int t = 0; t < s.n && !stop; ++t) {
            const TilePages<TN, 1> pages = ahead;
            const int p0 = (s.tile0 + t) * TN;
            if (t + 1 < s.n) ahead = tile_pages<D, PART, TN>(A, table, cached, p0 + TN);
            stop = !tc_wait_warp(&S.empty[kr.at], kr.phase, S);
            if (stop) break;
            load_tile<D, PART, TN, 1>(A, k_map, pages, s.b, s.R.n, cached, hi, p0, s.h, kv,
                                      ring0 + kr.at * kSlotBytes, &S.full[kr.at], &S.copied[kr.at],
                                      policy, 0, missing);
            kr.step();
            ++kfilled;
            if (t == 0 && leads) find();   // while the first tile is on its way
          }
          __syncwarp();
          if (leads) {
            if (lead && !stop) mbar_arrive(smem_addr(&S.noted[unit % kSegs]));
          } else {
            pt_taken(S, unit);
          }
        } else {
          auto load = [&](Ring& r, const CUtensorMap* map, int t) {
            if (!tc_wait_warp(&S.empty[r.at], r.phase, S)) return false;
            if (lead) {
              const uint32_t bar = smem_addr(&S.full[r.at]);
              mbar_arrive_expect_tx(bar, uint32_t(parts * TN * 128));
              for (int p = 0; p < parts; ++p)
                box_load3(ring0 + r.at * kSlotBytes + p * (TN * 128), map, p * 64, s.h,
                          s.row0 + (s.tile0 + t) * TN, bar);
            }
            __syncwarp();
            r.step();
            return true;
          };
          for (int t = 0; t < s.n && !stop; ++t) {
            stop = !load(kr, &k_map, t);
            kfilled += !stop;
            if (!stop) {
              stop = !load(vr, &v_map, t);
              vfilled += !stop;
            }
            if (t == 0) find();   // while the first tile is on its way
          }
        }
        if (stop) break;
      }
      // The copies that were issued land before the block ends, whatever the other warps
      // do: one of them may give up after this one has left.
      ring_land(kr, kfilled, S.full);
      ring_land(vr, vfilled, S.full);
      for (int g = 0; g < NQ; ++g)
        if (quse[g] > 0) mbar_wait_for(smem_addr(&S.qfull[g]), (quse[g] - 1) & 1);
      if constexpr (TREE) asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kMmaWarp) {
      // -------------------------------------------------------------- products
      constexpr uint32_t kBase = (1u << 4) | (Bits<T>::kFmt << 7) | (Bits<T>::kFmt << 10) |
                                 (uint32_t(kM >> 4) << 24);
      constexpr uint32_t kIdescS = kBase | (uint32_t(TN >> 3) << 17);
      const uint32_t wide = uint32_t(dim + 15) / 16;   // 16-element pieces of the head
      const uint32_t idesc_o = kBase | ((wide * 2) << 17) | (1u << 16);
      const uint32_t lead = elect_one();
      Ring kr(0, C::kKSlots, 0), vr(C::kKSlots, C::kSlots - C::kKSlots, 0);
      const uint64_t q_desc = sw128_desc(smem0), k_desc = sw128_desc(ring0);
      const uint64_t v_desc = mn_desc(ring0, TN * 128);
      uint32_t quse[2] = {0, 0}, pcount[2] = {0, 0}, scount[2] = {0, 0}, ouse[2] = {0, 0};
      bool ok = true;
      // orders the lanes' copies before the products' reads
      auto fence_copied = [&](uint32_t slot) {
        if (TREE && *reinterpret_cast<volatile int*>(&S.copied[slot])) fence_async_proxy();
        tc_fence_after();
      };
      auto score = [&](int g, const Seg& s, int t) {   // S of row tile g
        const uint64_t k = k_desc + kr.at * (kSlotBytes >> 4), q = q_desc + g * (C::kQBytes >> 4);
        const uint32_t buf = NB == 2 ? scount[g] & 1 : 0;
        const uint32_t d = tmem + (g * NB + buf) * TN;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          if (PART && c >= int(wide)) break;
          mma_ss(lead, d, q + (((c >> 2) * (kM * 128) + (c & 3) * 32) >> 4),
                 k + (((c >> 2) * (TN * 128) + (c & 3) * 32) >> 4), kIdescS, c != 0);
        }
        mma_commit(lead, &S.sfull[g][buf]);
        if (t + 1 == s.cnt[g]) mma_commit(lead, &S.qempty[g]);
        ++scount[g];
      };
      for (int unit = 0; ok; ++unit) {
        Seg s;
        ok = pt_next_seg(S, unit, s);
        if (!ok) break;
        pt_taken(S, unit);
        ok = tc_wait_warp(&S.full[kr.at], kr.phase, S);
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          if (!ok || s.cnt[g] == 0) continue;
          ok = tc_wait_warp(&S.qfull[g], quse[g]++ & 1, S);
          if (!ok) break;
          fence_copied(kr.at);
          score(g, s, 0);
        }
        if (!ok) break;
        mma_commit(lead, &S.empty[kr.at]);
        kr.step();
        for (int t = 0; ok && t < s.n; ++t) {
          const bool more = t + 1 < s.n;
          if (NB == 2 && more) {
            // two accumulators: the next scores before this tile's P is waited for
            ok = tc_wait_warp(&S.full[kr.at], kr.phase, S);
            if (!ok) break;
            fence_copied(kr.at);
            score(0, s, t + 1);
            mma_commit(lead, &S.empty[kr.at]);
            kr.step();
          }
#pragma unroll
          for (int g = 0; g < NQ; ++g) {
            if (!ok || t >= s.cnt[g]) continue;
            if (t == 0) {   // O still holds the unit before until its rows have been read
              ok = tc_wait_warp(&S.ofree[g], (ouse[g]++ & 1) ^ 1, S);
              if (!ok) break;
            }
            const uint32_t buf = NB == 2 ? pcount[g] & 1 : 0;
            // (tiles of K and V are waited for once, by the first row tile that has them:
            // a wait that succeeds takes about 100 cycles; 16001 tokens 1335 -> 1317 us)
            ok = ((g > 0 && t < s.cnt[0]) ||
                  tc_wait_two(&S.full[vr.at], vr.phase, &S.clean[vr.at], vr.phase, S)) &&
                 tc_wait_warp(&S.pfull[g][buf], (NB == 2 ? pcount[g] >> 1 : pcount[g]) & 1, S);
            if (!ok) break;
            if (g == 0 || t >= s.cnt[0]) fence_copied(vr.at);
            else tc_fence_after();
            const uint64_t v = v_desc + vr.at * (kSlotBytes >> 4);
            const uint32_t p = tmem + (g * NB + buf) * TN;
#pragma unroll
            for (int c = 0; c < TN / 16; ++c)
              mma_ts(lead, tmem + C::kOCol + g * D, p + c * 8, v + c * (2048 >> 4), idesc_o,
                     (c != 0) || t > 0);
            mma_commit(lead, &S.pvdone[g][buf]);
            ++pcount[g];
            if (NB == 1 && t + 1 < s.cnt[g]) {
              if (g == 0 || t + 1 >= s.cnt[0]) {
                ok = tc_wait_warp(&S.full[kr.at], kr.phase, S);
                if (!ok) break;
                fence_copied(kr.at);
              }
              score(g, s, t + 1);
            }
          }
          if (!ok) break;
          mma_commit(lead, &S.empty[vr.at]);
          vr.step();
          if (NB == 1 && more) {
            mma_commit(lead, &S.empty[kr.at]);
            kr.step();
          }
        }
      }
      // products in flight land, whichever warp gave up
      mma_commit(lead, &S.drain);
      mbar_wait_for(smem_addr(&S.drain), 0);
      __syncwarp();
    } else {
      // ------------------------------------------- values of tiles seen in part
      const int w = kLastWarp - warp;
      Ring vr(C::kKSlots, C::kSlots - C::kKSlots, 0);
      uint32_t dirties[2] = {0, 0};
      bool ok = true;
      for (int unit = 0; ok; ++unit) {
        Seg s;
        ok = pt_next_seg(S, unit, s);
        if (!ok) break;
        pt_taken(S, unit);
        for (int t = 0; t < s.n; ++t, vr.step()) {
          const int p0 = (s.tile0 + t) * TN;
          ok = tc_wait_warp(&S.full[vr.at], vr.phase, S);
          if (!ok) break;
          const bool edge = p0 < s.all_lo || p0 + TN > s.all_hi;
          if (!edge) {
            if (lane == 0) {
              mbar_arrive(smem_addr(&S.looked[vr.at]));
              mbar_arrive(smem_addr(&S.clean[vr.at]));
            }
            continue;
          }
          constexpr int kVecs = kSlotBytes / 16 / kLooks;   // a warp's share
          uint4* v = reinterpret_cast<uint4*>(smem_p + NQ * C::kQBytes + vr.at * kSlotBytes) +
                     w * kVecs;
          // parts behind a narrow head were not loaded
          const int mine = PART ? max(0, min(kVecs, parts * TN * 8 - w * kVecs)) : kVecs;
          bool found = false;
#pragma unroll 8
          for (int i = lane; i < mine; i += 32) {
            const uint4 x = v[i];
            found |= any_nonfinite<T>(x.x) | any_nonfinite<T>(x.y) | any_nonfinite<T>(x.z) |
                     any_nonfinite<T>(x.w);
          }
          found = __any_sync(0xffffffffu, found);
          if (lane == 0) {
            S.dirty[vr.at][w] = found;
            mbar_arrive(smem_addr(&S.looked[vr.at]));
          }
          ok = tc_wait_warp(&S.looked[vr.at], vr.phase, S);
          if (!ok) break;
          const volatile int* dirty = S.dirty[vr.at];
          if (dirty[0] | dirty[1]) {
#pragma unroll
            for (int g = 0; g < NQ; ++g)
              if (t < s.cnt[g]) ok = tc_wait_warp(&S.collected[g], dirties[g]++ & 1, S) && ok;
            if (!ok) break;
            for (int i = lane; i < mine; i += 32) {
              uint32_t* x = reinterpret_cast<uint32_t*>(v + i);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t odd = ((x[e] & Bits<T>::kExp) + Bits<T>::kOne) & 0x80008000u;
                x[e] &= ~((odd >> 15) * 0xffffu);
              }
            }
            fence_async_proxy();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(smem_addr(&S.clean[vr.at]));
        }
      }
    }
  } else if (go && warp < 4 * NQ) {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int g = warp >> 2, rr = tid & 127;
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t o_at = lanes + C::kOCol + g * D;
    const int mine = rr / A.G, head = rr % A.G;   // token of the tile, head of the group
    int quad_row[4];                               // rows of out of the four lanes
#pragma unroll
    for (int i = 0; i < 4; ++i) quad_row[i] = ((rr & ~3) + i) / A.G * A.Hq + ((rr & ~3) + i) % A.G;
    uint32_t count = 0;                            // tiles of this row tile so far
    Ring vr(C::kKSlots, C::kSlots - C::kKSlots, 0);
    bool ok = true;
    for (int unit = 0; ok; ++unit) {
      Seg s;
      ok = pt_next_seg(S, unit, s);
      if (unit == 0 && A.test_expire == int(blockIdx.x) + 1 && ok &&
          !mbar_wait_for(smem_addr(&S.never), 0, kTestWaitNs)) {
        *reinterpret_cast<volatile int*>(&S.abort) = 1;
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int tok0 = s.tok0 + g * toks;          // of this row tile
      const int tok = tok0 + mine;
      const int cnt = s.cnt[g];
      const bool live = mine < s.live[g];
      // the row sees positions row_lo .. row_hi - 1, of a tree also path's bits behind
      int row_hi = INT32_MAX, row_lo = 0;
      uint64_t path = 0;
      if constexpr (TREE) {
        // Every part's CTA, and every warp, looks at all the request's parents, so that
        // a torn tree fails in all of them.
        const int32_t* parents = A.parent + s.row0;
        bool torn = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = lane + 32 * i;
          if (j == 0 || j > s.R.k || s.R.code) continue;
          const int up = parents[j];
          torn |= up < 0 || up >= j;
        }
        if (__any_sync(0xffffffffu, torn) && lane == 0) {
          S.part_bad[unit % kSegs] = 1;
          atomicMin(&S.first_torn, s.b);
        }
        const AttnNode node = attn_node(A, parents, s.R.n, min(tok, s.R.k));
        if (live) {
          row_hi = s.all_hi;
          row_lo = A.window > 0 ? max(0, node.at - A.window + 1) : 0;
          path = s.R.code ? 0 : node.path;
        }
      } else if (live) {
        row_hi = tok + 1;
        row_lo = A.window > 0 ? max(0, tok - A.window + 1) : 0;
      }
      // what all rows of this row tile see
      const int own_hi = TREE ? s.all_hi : tok0 + 1;
      const int own_lo = TREE           ? s.all_lo
                         : A.window > 0 ? max(0, tok0 + s.live[g] - A.window)
                                        : 0;
      // the product with P of the row tile's tile number x (of all units) has landed
      auto product_done = [&](uint32_t x) {
        return tc_wait_warp(&S.pvdone[g][NB == 2 ? x & 1 : 0], (NB == 2 ? x >> 1 : x) & 1, S);
      };
      float m = -INFINITY, l = 0.f;   // m: the maximum that the sum and O refer to
      for (int t = 0; t < s.n; ++t, vr.step()) {
        const int p0 = (s.tile0 + t) * TN;
        if (t >= cnt) continue;   // the other row tile's: its slot may be filled again by now
        bool dirty = false;
        uint32_t signs[2 * D / 32];
        if (p0 < s.all_lo || p0 + TN > s.all_hi) {
          ok = tc_wait_warp(&S.looked[vr.at], vr.phase, S);
          if (!ok) break;
          const volatile int* d = S.dirty[vr.at];
          dirty = (d[0] | d[1]) != 0;
          if (dirty) {
            collect_signs<T, D, TN>(
                reinterpret_cast<const uint32_t*>(smem_p + NQ * C::kQBytes + vr.at * kSlotBytes),
                0, TN, row_lo - p0, live ? row_hi - p0 : 0, path, row_hi - p0, signs);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&S.collected[g]));
          }
        }
        const uint32_t buf = NB == 2 ? count & 1 : 0;
        const uint32_t phase = (NB == 2 ? count >> 1 : count) & 1;
        const uint32_t scol = lanes + (g * NB + buf) * TN;
        ok = tc_wait_warp(&S.sfull[g][buf], phase, S);
        if (!ok) break;
        tc_fence_after();
        float x[TN];
#pragma unroll
        for (int c = 0; c < TN / 32; ++c)
          tmem_ld32(scol + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[c * 32]));
        tmem_ld_wait();
        if (TREE && p0 + TN > own_hi) {
#pragma unroll
          for (int c0 = 0; c0 < TN; c0 += 32) {
            // a bit per column: cached positions, then nodes
            const int hi = row_hi - p0 - c0;
            uint32_t see = hi >= 32 ? ~0u : hi > 0 ? (1u << hi) - 1 : 0u;
            if (hi < 32 && hi > -64)
              see |= hi >= 0 ? uint32_t(path) << hi : uint32_t(path >> -hi);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c0 + c] = (see >> c) & 1 ? x[c0 + c] : -INFINITY;
          }
        }
        if (!TREE && p0 + TN > own_hi) {
          const int hi = row_hi - p0;
#pragma unroll
          for (int c = 0; c < TN; ++c) x[c] = c < hi ? x[c] : -INFINITY;
        }
        if (p0 < own_lo) {   // (what a tree's row sees of the nodes is behind its row_lo)
          const int lo = min(row_lo, row_hi) - p0;
#pragma unroll
          for (int c = 0; c < TN; ++c) x[c] = c >= lo ? x[c] : -INFINITY;
        }
        // four chains, two values a step
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = fmaxf(x[2 * c], x[2 * c + 1]);
#pragma unroll
        for (int c = 8; c < TN; c += 2)
          asm("max.f32 %0, %0, %1, %2;" : "+f"(top[c / 2 & 3]) : "f"(x[c]), "f"(x[c + 1]));
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const float grown = fmaxf(m, high * A.scale2);   // scale2 > 0
        const bool rescale = live && grown > m + kRescaleLog2;
        if (__any_sync(0xffffffffu, rescale)) {
          // all rows of the warp move to their present maximum
          const float f = m == -INFINITY ? 0.f : exp2f(m - grown);
          if (t > 0) {
            ok = product_done(count - 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c * 16 < dim; ++c) {
              uint32_t o[16];
              tmem_ld16(o_at + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_at + c * 16, o);
            }
          }
          l *= f;
          m = grown;
        }
        const float sh = (m == -INFINITY ? 0.f : m) - Bits<T>::kLift;
        const uint64_t sc2 = pk2(A.scale2, A.scale2), sh2 = pk2(-sh, -sh);
        uint64_t sum[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
        for (int c0 = 0; c0 < TN; c0 += 32) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float e0, e1;
            upk2(fma2(pk2(x[c0 + c], x[c0 + c + 1]), sc2, sh2), e0, e1);
            e0 = ex2_approx(e0);
            e1 = ex2_approx(e1);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pk2(e0, e1));
            w[c / 2] = Bits<T>::pack(e0, e1);
          }
          tmem_st16(scol + c0 / 2, w);
        }
        float s0, s1;
        upk2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&S.pfull[g][buf]));
        ++count;
        if (dirty) {
          ok = product_done(count - 1);
          if (!ok) break;
          tc_fence_after();
          add_signs<D>(o_at, dim, signs);
          tc_fence_before();
        }
      }
      if (!ok) break;
      if (cnt == 0) {
        pt_taken(S, unit);
        continue;
      }
      // ------------------------------------------------- the row tile's rows
      ok = product_done(count - 1);
      if (!ok) break;
      tc_fence_after();
      float inv = l == 0.f ? 0.f : 1.f / l;
      bool bad = false;
      if constexpr (TREE) {
        ok = tc_wait_warp(&S.noted[unit % kSegs], (unit / kSegs) & 1, S);
        if (!ok) break;
        bad = *reinterpret_cast<volatile int*>(&S.part_bad[unit % kSegs]) != 0;
        if (bad) inv = __int_as_float(0x7fc00000);
        if (!s.whole) {
          // the part as it is, 16 columns at a time, and what it refers to
          const int64_t row = (int64_t(blockIdx.x) * 2 + (s.first == 0)) * 2 * kM + g * kM;
          float* part = A.part_o + (row + (rr & ~3)) * dim + (lane & 3) * 4;
          const int rows = s.live[g] * A.G - (rr & ~3);
#pragma unroll 1
          for (int c = 0; c * 16 < dim; ++c) {
            uint32_t o[16], w[4][4];
            tmem_ld16(o_at + c * 16, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e >> 2][e & 3] = o[e];
            exchange4(w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < rows)
                *reinterpret_cast<uint4*>(part + i * dim + c * 16) =
                    make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
          }
          if (live)
            A.part_ml[row + rr] =
                make_float2(bad ? __int_as_float(0x7fc00000) : m - Bits<T>::kLift, l);
          if (tid == 0 && s.first == 0) pt_begin_split(A, P, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&S.ofree[g]));
          pt_taken(S, unit);
          continue;
        }
      }
      const int64_t to = (int64_t(s.row0) + tok) * A.Hq + s.h * A.G + head;
      T* out = static_cast<T*>(A.out) + to * A.D;
      if (A.out_vec) {
        // Four lanes exchange their rows' pieces of 16 bytes, so that each store writes
        // 64 bytes of eight rows instead of 16 of 32 rows.  A loop of few instructions:
        // once a unit, it is their fetching that takes the time.
        T* unit_out = static_cast<T*>(A.out) + ((int64_t(s.row0) + tok0) * A.Hq + s.h * A.G) * A.D;
        const int piece = lane & 3, live_rows = s.live[g] * A.G - (rr & ~3);
        const uint64_t inv2 = pk2(inv, inv);
#pragma unroll 1
        for (int c = 0; c * 32 < dim; ++c) {
          uint32_t o[32], w[4][4];
          tmem_ld32(o_at + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, b;
            upk2(mul2(pk2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2), a, b);
            w[e >> 2][e & 3] = Bits<T>::pack(a, b);
          }
          exchange4(w);
          const int col = c * 32 + piece * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < live_rows && !(PART && col >= dim))
              *reinterpret_cast<uint4*>(unit_out + int64_t(quad_row[i]) * A.D + col) =
                  make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        }
      } else {
        rows_one_by_one<T>(o_at, dim, inv, live ? out : nullptr);
      }
      if (live) {
        const float ref = m - Bits<T>::kLift;   // what O and the sum refer to
        const float lse = (ref == -INFINITY ? 0.f : ref * kAttnLn2) + logf(l);
        A.lse[to] = bad ? __int_as_float(0x7fc00000) : lse;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&S.ofree[g]));
      pt_taken(S, unit);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (go && S.abort) pt_give_up<T, D>(A, S.top);
  if constexpr (TREE) {
    if (tid == 0) {
      A.status[A.B + blockIdx.x] = S.abort ? -SV_ERR_TIMEOUT : S.first_bad;
      A.status[A.B + A.ctas + blockIdx.x] = S.first_torn;
    }
  } else if (tid == 0) {
    A.status[1 + blockIdx.x] = S.abort ? -SV_ERR_TIMEOUT : INT32_MAX;
    if (blockIdx.x == 0) prompt_header(A, !go, gridDim.x);
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
  }
}

// Rows of heads as boxes of 64 elements by `heads` heads by `rows` rows, 128-byte
// swizzled.
bool heads_map(CUtensorMap* map, const void* data, bool bf16, int D, int H, int64_t rows,
               int64_t ts, int64_t hs, int heads, int box_rows) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(H), cuuint64_t(rows)};
  // a stride that nothing is multiplied with may be anything
  const cuuint64_t strides[2] = {cuuint64_t(H > 1 ? hs : 64) * 2,
                                 cuuint64_t(rows > 1 ? ts : 64) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(heads), cuuint32_t(box_rows)}, step[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace sv
