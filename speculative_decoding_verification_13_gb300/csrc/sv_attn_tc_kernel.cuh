// Attention over the paged KV cache on the fifth-generation tensor cores, for
// bf16 and fp16 and heads of 64 to 256, multiples of 16 (taken at D, the next of
// 64, 128 and 256).  TREE: the drafts are a tree and see their ancestors.
//
// A unit is up to 128 query rows of one KV head, the M of the products:
// S = Q K^T (128 x TN x D) and O += P V (128 x D x TN) per tile of TN = 128
// positions (64 for D = 256, whose O takes half of TMEM).  Few rows leave most
// of M idle, which costs the HBM nothing: with heads of 128 the two products of
// a tile take about 1100 cycles of the tensor cores, its 64 KB of K and V about
// 2800 of an SM's share of the HBM.  It would cost the softmax: so a unit of up
// to 64 rows lies twice in M, one of up to 32 four times, and each copy weighs
// its half or quarter of a tile's columns (all four warps work, with a quarter
// of the chain of each row); the copies' sums and outputs add up at the end.
//
// One CTA per SM, over its piece of the line of tiles (sv_attn.cuh):
//   warp 8     finds the CTA's units, announces them and loads their Q, one ahead
//              where two fit (64 rows of heads of 128, twice in M: an address and
//              an asynchronous copy at a time 26000 cycles, now 8500).
//   warps 4, 5 load, tile by tile, K and V into rings of slots, in the
//              128-byte swizzled layout that the tensor cores read (K along the
//              head: K-major; V along the head: MN-major).  The copy engine
//              moves what a page has of the tile in boxes of 128 bytes by the
//              page's rows, one box a lane.  Tiles that are not whole (the end
//              of the cache, speculative entries) and pages of other than a
//              multiple of 8 positions come by 16-byte asynchronous copies of
//              the lanes, which fill positions outside the request's keys with
//              zeros; the product warp's fence orders them before its reads.
//              Measured on 32 requests with up to 15 drafts: all tiles by
//              16-byte copies with the fence on the writing side, which waits
//              for every copy in flight, 229 us; rows gathered by the copy
//              engine, four an instruction, of which it takes one in about 50
//              cycles, 264 us.
//   warps 6, 7 issue the products, one S and one O.  S has three accumulators, so
//              that S of the next tiles does not wait for the product of this
//              one.  (One warp for both: a tile of 128 positions of heads of 64
//              took 1760 cycles, of which its 12 products 620.)
//   warps 0-3  softmax, one row a thread (the lanes of TMEM): scores from TMEM,
//              running maximum, P rounded to the type (half a step of it, the
//              one rounding of a weight: 0.0023 of the result's norm off 64 bits
//              with 15 drafts in bf16, where weights of 32 bits leave 0.0017;
//              sums stay in 32 bits) back to TMEM over the scores, where the
//              second product reads it as its A operand.
//              O is rescaled only when a row's maximum has grown by more than
//              2^8 since the last time: the stored maximum is then exact enough
//              for P and the sum to stay in range, and most tiles skip it.
// A warp without live rows only keeps the barriers' count.
//
// Tiles that some row of the unit sees in part (the drafts' triangle, a
// window's edge): the masked weights are 0, but 0 times an infinite or NaN
// value would still reach the row.  The softmax warps look through V of such a
// tile; if it holds any, each row collects the signs of those that it sees,
// they are replaced by 0 in the tile, and added to the row's O afterwards.
//
// Every wait is bounded; on expiry the CTA's status records it, its copies and
// products land, TMEM is freed, and the rows of the CTA's parts become NaN.
//
// Measured, bf16, 8 KV heads of 128 with 4 query heads each, pages of 16: 64
// requests of 1 to 16000 positions, one token, 77 us with the join (5.4 TB/s); 32
// of 2001 to 8190 with up to 15 drafts 108 us (5.6 TB/s); one of 900 positions 15
// us, all of it latency.  fp16, 16 heads of 64, 3 requests of 100001 to 131071
// positions and 7 drafts, pages of 64: 219 us (7.0 TB/s).  What the first two lose
// to the HBM's rate is the units' beginnings and ends: short requests have few
// tiles for each.
#pragma once

#include <type_traits>

#include "sv_attn_tc.cuh"

namespace sv {
namespace {

constexpr int kTcThreads = 288;   // 4 softmax warps, then one each of the following
constexpr int kTcMr = 128;
constexpr int kBufs = 3;          // S accumulators, each then the P of its tile
constexpr int kLoadWarp = 4, kScoreWarp = 6, kValueWarp = 7, kQueryWarp = 8;
constexpr int kSegs = 8;          // parts announced ahead of the warp that is furthest back
constexpr float kRescaleLog2 = 8.0f;

// Copies' sums meet in shared memory: maximum and sum of each row of M, what
// its row is divided by, and as many columns of the live rows' O as fit.
constexpr int kStageFloats = kTcMr * 33;
struct Stage {
  float2 ml[kTcMr];
  int64_t out[kTcMr];   // where the row's output begins
  float inv[kTcMr];
  float o[kStageFloats];
};
constexpr size_t kStageBytes = (sizeof(Stage) + 127) / 128 * 128;

// What a unit costs beside its tiles, in tiles: the line that is cut over the
// CTAs counts it.  64 requests of 1 to 16000 positions: without it the CTA with the
// most short ones took twice as long as the others; with 2 tiles 158000 cycles
// against 127000 (88 us), a unit costing about 3.5 of 2200; with 4 82 us, as with 6.
template <int D>
constexpr int kUnitTiles = D == 64 ? 3 : 4;

template <int D>
struct Shape {
  static constexpr int TN = D == 256 ? 64 : 128;
  static constexpr int kSlotBytes = TN * D * 2;
  static constexpr int kQBytes = kTcMr * D * 2;
  static constexpr int kQBufs = D == 256 ? 1 : 2;
  static constexpr int kSlots = D == 64 ? 10 : 5;  // what shared memory holds
  // of K; the rest, three at least (the softmax warps look at V of a tile whose
  // slot was filled before at most three tiles ago), are of V
  static constexpr int kKSlots = kSlots / 2;
  static constexpr uint32_t kOCol = kBufs * TN;     // TMEM columns: the S accumulators, then O
  // where copies of rows are added up: a query buffer, or a place of its own
  static constexpr bool kOwnStage = kQBytes < int(kStageBytes);
  static constexpr size_t kSmem = 1024 + kQBufs * size_t(kQBytes) + size_t(kSlots) * kSlotBytes +
                                  (kOwnStage ? kStageBytes : 0);
};
constexpr uint32_t kTmemCols = 512;

// One unit's part of a CTA's piece.  The query warp finds them, a few ahead, and
// announces them to the others; count 0 is the end.
struct Seg {
  int b, t_off, h, row0, rows, first, count;
  int copies;         // of the rows in the M of the products
  bool whole;
  int64_t unit_end;   // tile of the line after the unit's last
  AttnReq R;
};

struct TcShared {
  Seg seg[kSegs];
  uint64_t announced[kSegs], noted[kSegs];   // noted: every page of the part was looked at
  uint64_t full[11], empty[11];
  uint64_t qfull[2], qempty[2], sfull[kBufs], pfull[kBufs], pvdone[kBufs], ofree;
  uint64_t looked[2], drain[2];  // softmax warps among themselves; products after a failure
  uint64_t never;                // nothing arrives on it: the test of an expired wait
  uint32_t tmem;
  int abort;
  int first_bad;
  struct {
    uint32_t at, phase;
    int filled;
  } loaded[2];       // the rings of K and V as their warps left them
  int bad[kSegs];    // the part needs a missing page
  int copied[11];    // per slot: filled by the lanes' copies, not by the copy engine
  uint32_t signs[2][8];  // per column: +inf, -inf among the part's values
  int dirty[kBufs];  // per S buffer: 1 + the tile whose V holds a non-finite value
  int first_torn;    // first request with a parent that does not point back
};

// One of the S buffers and the phase of its barriers, one tile a step.
struct Buf {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++at == kBufs) {
      at = 0;
      phase ^= 1;
    }
  }
};

template <int TN, int PAD>
struct Walk {
  int64_t pos, end, base;
  int b, t_off;
  AttnReq R;
  __device__ __forceinline__ Walk(const AttnArgs& A, const AttnPlan& P)
      : pos(P.start), end(P.end), base(P.base), b(P.b), t_off(P.t_off) {
    if (pos < end) R = attn_request<TN, kTcMr, false>(A, b);
  }
  __device__ __forceinline__ bool next(const AttnArgs& A, Seg& s) {
    if (pos >= end) return false;
    int64_t nt, local;
    int unit;
    for (;;) {
      nt = attn_tiles<TN, kTcMr, false, PAD>(A, R);
      while (pos >= base + nt) {
        base += nt;
        t_off += R.k + 1;
        R = attn_request<TN, kTcMr, false>(A, ++b);
        nt = attn_tiles<TN, kTcMr, false, PAD>(A, R);
      }
      local = pos - base;
      const int span = R.ntiles + PAD, at = int(local % span);
      unit = int(local / span);
      if (at >= PAD) {
        s.first = at - PAD;
        break;
      }
      pos += PAD - at;   // a unit's tiles come behind what it costs itself
      if (pos >= end) return false;
    }
    s.b = b;
    s.t_off = t_off;
    const int64_t left = end - pos;
    s.count = int(left < R.ntiles - s.first ? left : R.ntiles - s.first);
    s.h = unit / R.mtiles * A.hg + int(blockIdx.x) % A.hg;
    s.row0 = (unit % R.mtiles) * kTcMr;
    s.rows = min(kTcMr, (R.k + 1) * A.G - s.row0);
    s.copies = s.rows <= 32 && TN == 128 ? 4 : s.rows <= 64 ? 2 : 1;
    s.whole = s.first == 0 && s.count == R.ntiles;
    s.unit_end = pos - s.first + R.ntiles;
    s.R = R;
    pos += s.count;
    return true;
  }
};

// Descriptor of an MN-major 16-bit tile with 128-byte swizzling: rows (of K)
// of 128 bytes, 8-row groups 1024 bytes apart, blocks of 64 elements of MN
// `block` bytes apart.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t addr, uint32_t block) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(block >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}


// Bit 0: a value is +inf, bit 1: it is -inf; both: NaN.
template <class T>
__device__ __forceinline__ uint32_t value_signs(uint32_t x) {
  if ((x & Bits<T>::kExp1) != Bits<T>::kExp1) return 0;
  return (x & Bits<T>::kMan1) ? 3u : (x & 0x8000u) ? 2u : 1u;
}

// Hardware barrier of the softmax warps, and the same with one truth value for
// all of them.  None may stay away: they leave their loop only together.
__device__ __forceinline__ void softmax_sync() {
  __syncwarp();
  asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
}
__device__ __forceinline__ bool softmax_any(bool x) {
  int any;
  __syncwarp();
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 2, 128, p;\nselp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"(int(x))
      : "memory");
  return any != 0;
}

// The part that warp comes to next; false at the end, or when the CTA gave up.
__device__ __forceinline__ bool next_seg(TcShared& S, int unit, Seg& s) {
  if (!tc_wait_warp(&S.announced[unit % kSegs], (unit / kSegs) & 1, S)) return false;
  s = S.seg[unit % kSegs];
  return s.count > 0;
}

// The unit that the CTA begins with s ends in a later one: the join's record of it.
__device__ __forceinline__ void begin_split(const AttnArgs& A, const AttnPlan& P, const Seg& s) {
  AttnSplit& u = A.split[blockIdx.x];
  u.last = attn_owner(A, P, s.unit_end - 1);
  u.t_off = s.t_off;
  u.h = s.h;
  u.row0 = s.row0;
  u.rows = s.rows;
  u.valid = 1;
}

// All threads, after a wait of the CTA expired and every warp has left its loop.
// Copies and products that were issued finish, whichever warp gave up and when.
// Then every row of the CTA's parts becomes NaN, whether it was written or not, and
// so does what the join makes of them with other CTAs' parts.  A function of its
// own, which finds the CTA's piece again: in the kernel's body it cost the loops
// their registers (long contexts 230 -> 247 us).
template <class T, int D>
__device__ __noinline__ void give_up(const AttnArgs& A, TcShared& S) {
  using C = Shape<D>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    const int kv = warp - kLoadWarp;
    Ring at(kv ? C::kKSlots : 0, kv ? C::kSlots - C::kKSlots : C::kKSlots, S.loaded[kv].phase);
    at.at = S.loaded[kv].at;
    ring_land(at, S.loaded[kv].filled, S.full);
  } else if (warp == kScoreWarp || warp == kValueWarp) {
    uint64_t* drain = &S.drain[warp - kScoreWarp];
    mma_commit(elect_one(), drain);   // of the lane that issued the products
    mbar_wait_for(smem_addr(drain), 0);
    __syncwarp();
  }
  __syncthreads();
  const float nan = __int_as_float(0x7fc00000);
  const AttnPlan P = attn_plan<C::TN, kTcMr, false, kTcThreads, kUnitTiles<D>>(A);
  Walk<C::TN, kUnitTiles<D>> walk(A, P);
  Seg s;
  while (walk.next(A, s)) {
    const int slot = s.first == 0 ? 1 : 0;
    for (int r = warp; r < s.rows; r += kTcThreads / 32) {
      const int x = s.row0 + r, hq = s.h * A.G + x % A.G;
      const int64_t t = int64_t(s.t_off) + x / A.G;
      if (s.whole) {
        T* out = static_cast<T*>(A.out) + t * A.o_ts + int64_t(hq) * A.o_hs;
        for (int d = lane; d < A.D; d += 32) out[d] = from_float<T>(nan);
        if (lane == 0) A.lse[t * A.Hq + hq] = nan;
      } else if (lane == 0) {
        A.part_ml[(int64_t(blockIdx.x) * 2 + slot) * kTcMr + r] = make_float2(nan, 0.f);
      }
    }
    if (tid == 0 && !s.whole && s.first == 0) begin_split(A, P, s);
  }
}

template <class T, int D, bool PART, bool TREE>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap rows_map,
                   const __grid_constant__ AttnArgs A) {
  using C = Shape<D>;
  constexpr int TN = C::TN;
  extern __shared__ unsigned char tc_smem_raw[];
  __shared__ TcShared S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_addr(tc_smem_raw) + 1023u) & ~1023u;
  unsigned char* smem_p = tc_smem_raw + (smem0 - smem_addr(tc_smem_raw));
  const uint32_t ring0 = smem0 + C::kQBufs * C::kQBytes;
  constexpr int kSlotBytes = C::kSlotBytes;
  const int dim = head_width<D, PART>(A);

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_addr(&S.full[i]), 32);  // the lanes of a load warp
      mbar_init(smem_addr(&S.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&S.qfull[i]), 1);
      mbar_init(smem_addr(&S.qempty[i]), 4);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_addr(&S.sfull[i]), 1);
      mbar_init(smem_addr(&S.pfull[i]), 4);
      mbar_init(smem_addr(&S.pvdone[i]), 1);
      S.dirty[i] = 0;
    }
    mbar_init(smem_addr(&S.ofree), 4);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(smem_addr(&S.announced[i]), 1);
      mbar_init(smem_addr(&S.noted[i]), 2);
    }
    mbar_init(smem_addr(&S.looked[0]), 4);
    mbar_init(smem_addr(&S.looked[1]), 4);
    mbar_init(smem_addr(&S.drain[0]), 1);
    mbar_init(smem_addr(&S.drain[1]), 1);
    mbar_init(smem_addr(&S.never), 1);
    fence_mbar_init();
    S.abort = 0;
    S.first_bad = S.first_torn = INT32_MAX;
    A.split[blockIdx.x].valid = 0;
  }
  if (warp == kValueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&S.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  const AttnPlan P = attn_plan<TN, kTcMr, false, kTcThreads, kUnitTiles<D>>(A);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  if (P.code) fail_all<T>(A);
  const bool go = P.code == 0 && P.start < P.end;

  if (go && warp >= kLoadWarp && warp < kScoreWarp) {
    // ----------------------------------------------------------------- loads
    const int kv = warp - kLoadWarp;              // 0: K, 1: V
    // keys that no other unit of the call reads leave the L2 first
    const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
    Seg s;
    Ring at(kv ? C::kKSlots : 0, kv ? C::kSlots - C::kKSlots : C::kKSlots,
            1);  // empty barriers: the first round passes at once
    bool stop = false;
    int filled = 0;
    for (int unit = 0; !stop && next_seg(S, unit, s); ++unit) {
      const int hi = s.R.code ? 0 : s.R.hi;
      const int cached = min(s.R.n, hi);
      const int p0 = (s.R.tile0 + s.first) * TN;
      const int32_t* table = A.table + int64_t(s.b) * A.max_pages;
      auto missing = [&](int page) {
        if (page >= 0 && page < A.num_pages) return false;
        S.bad[unit % kSegs] = 1;
        atomicMin(&S.first_bad, s.b);
        return true;
      };
      // pages are read one tile ahead, so that nothing waits for the block table
      TilePages<TN, 1> next = tile_pages<D, PART, TN>(A, table, cached, p0);
      int t = 0;
      for (; t < s.count; ++t) {
        const TilePages<TN, 1> pages = next;
        if (t + 1 < s.count) next = tile_pages<D, PART, TN>(A, table, cached, p0 + (t + 1) * TN);
        if (!tc_wait_warp(&S.empty[at.at], at.phase, S)) {
          stop = true;
          break;
        }
        load_tile<D, PART, TN, 1>(A, rows_map, pages, s.b, s.R.n, cached, hi, p0 + t * TN, s.h, kv,
                                  ring0 + at.at * kSlotBytes, &S.full[at.at],
                                  &S.copied[at.at], s.R.mtiles > 1 ? again : once, 0, missing);
        at.step();
      }
      filled += t;
      // Missing pages are noted while a tile's boxes are issued, after the lane's
      // arrival (before it they would hold up the copies: long contexts 229 -> 234
      // us); those who read the note wait for this arrival.
      __syncwarp();
      if (lane == 0 && !stop) mbar_arrive(smem_addr(&S.noted[unit % kSegs]));
    }
    if (lane == 0) {
      S.loaded[kv].at = at.at;
      S.loaded[kv].phase = at.phase;
      S.loaded[kv].filled = filled;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (go && warp == kQueryWarp) {
    // --------------------------------------------- parts, and their queries
    constexpr int kChunks = D / 8, kStep = 32 / kChunks;
    const int ch = lane % kChunks;
    const T* q = static_cast<const T*>(A.q);
    Walk<TN, kUnitTiles<D>> walk(A, P);
    for (int unit = 0;; ++unit) {
      Seg s;
      s.count = 0;
      walk.next(A, s);
      // This entry's part before is done with everywhere: the wait for a query
      // buffer in the last round saw the end of the third part before this one.
      if (lane == 0) {
        S.seg[unit % kSegs] = s;
        S.bad[unit % kSegs] = s.count && s.R.code != 0;
        mbar_arrive(smem_addr(&S.announced[unit % kSegs]));
      }
      if (s.count == 0) break;
      const int qb = unit % C::kQBufs;
      if (!tc_wait_warp(&S.qempty[qb], ((unit / C::kQBufs) & 1) ^ 1, S)) break;
      // Rows of a row-major swizzled tile per 64 elements of the head, copies of
      // them 128 / copies rows apart; rows between them stay as they are (what
      // a row of S or O holds reaches no other row).
      // The lanes find the rows' addresses together, and fetch them from one another;
      // eight loads are under way at once.  No branches (one takes as long as ten
      // other instructions of a lone warp): lanes without a row repeat the last one.
      const int apart = kTcMr / s.copies, last = s.rows - 1;
      auto fill = [&](auto vec) {
        constexpr int kAhead = 8;
        for (int r0 = 0; r0 < s.rows; r0 += 32) {
          const int mine = s.row0 + min(r0 + lane, last);
          const uint64_t own = reinterpret_cast<uint64_t>(
              q + int64_t(s.t_off + mine / A.G) * A.q_ts + int64_t(s.h * A.G + mine % A.G) * A.q_hs);
#pragma unroll 1
          for (int j0 = 0; j0 < min(32, s.rows - r0); j0 += kAhead * kStep) {
            uint4 v[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
              const int from = j0 + x * kStep + lane / kChunks;
              const uint64_t at =
                  (uint64_t(__shfl_sync(0xffffffffu, uint32_t(own >> 32), from)) << 32) |
                  __shfl_sync(0xffffffffu, uint32_t(own), from);
              v[x] = load_chunk<decltype(vec)::value>(reinterpret_cast<const T*>(at) +
                                                      (PART && ch * 8 >= dim ? 0 : ch * 8));
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
              const int r = min(r0 + j0 + x * kStep + lane / kChunks, last);
              unsigned char* to = smem_p + qb * C::kQBytes + (ch >> 3) * (kTcMr * 128) + r * 128;
              // copies lie 32, 64 or 128 rows apart: the same place in the swizzle
              const int place = ((ch & 7) ^ (r & 7)) << 4;
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (c < s.copies) *reinterpret_cast<uint4*>(to + c * apart * 128 + place) = v[x];
            }
          }
        }
      };
      if (A.q_vec) fill(std::true_type());
      else fill(std::false_type());
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&S.qfull[qb]));
    }
  } else if (go && (warp == kScoreWarp || warp == kValueWarp)) {
    // -------------------------------------------------------------- products
    // Two warps, so that one's waits do not hold up the other's products: every
    // order between them goes by barriers.
    constexpr uint32_t kBase = (1u << 4) | (Bits<T>::kFmt << 7) | (Bits<T>::kFmt << 10) |
                               (uint32_t(kTcMr >> 4) << 24);
    constexpr uint32_t kIdescS = kBase | (uint32_t(TN >> 3) << 17);
    const uint32_t idesc_o = kBase | (uint32_t(dim >> 3) << 17) | (1u << 16);
    const uint32_t lead = elect_one();
    const bool scores = warp == kScoreWarp;
    Ring slot(scores ? 0 : C::kKSlots, scores ? C::kKSlots : C::kSlots - C::kKSlots, 0);
    Buf buf;
    // The fence that orders the lanes' copies before the products' reads takes
    // as long as the products in flight: only slots that were filled by them.
    auto slot_copied = [&](uint32_t i) {
      return *reinterpret_cast<volatile int*>(&S.copied[i]) != 0;
    };
    // descriptors of the first Q buffer and slot; others lie a constant away
    const uint64_t q_desc = sw128_desc(smem0), k_desc = sw128_desc(ring0);
    const uint64_t v_desc = sw128_mn_desc(ring0, TN * 128);
    bool ok = true;
    for (int unit = 0; ok; ++unit) {
      ok = tc_wait_warp(&S.announced[unit % kSegs], (unit / kSegs) & 1, S);
      const int count = ok ? S.seg[unit % kSegs].count : 0;
      if (count == 0) break;
      if (scores) {
        const int qb = unit % C::kQBufs;
        ok = tc_wait_warp(&S.qfull[qb], (unit / C::kQBufs) & 1, S);
        const uint64_t q = q_desc + uint32_t(qb * (C::kQBytes >> 4));
        for (int t = 0; ok && t < count; ++t) {
          // keys there, and the buffer's last P read (the first round passes at once)
          ok = tc_wait_two(&S.full[slot.at], slot.phase, &S.pvdone[buf.at], buf.phase ^ 1, S);
          if (!ok) break;
          if (slot_copied(slot.at)) fence_async_proxy();
          tc_fence_after();
          const uint64_t k = k_desc + slot.at * (kSlotBytes >> 4);
          const uint32_t d = tmem + buf.at * TN;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            if (PART && c * 16 >= dim) break;
            mma_ss(lead, d, q + (((c >> 2) * (kTcMr * 128) + (c & 3) * 32) >> 4),
                   k + (((c >> 2) * (TN * 128) + (c & 3) * 32) >> 4), kIdescS, c != 0);
          }
          mma_commit(lead, &S.sfull[buf.at]);
          mma_commit(lead, &S.empty[slot.at]);
          slot.step();
          buf.step();
        }
      } else {
        // O still holds the unit before until its rows have been read
        if (unit > 0) ok = tc_wait_warp(&S.ofree, (unit - 1) & 1, S);
        for (int t = 0; ok && t < count; ++t) {
          ok = tc_wait_two(&S.full[slot.at], slot.phase, &S.pfull[buf.at], buf.phase, S);
          if (!ok) break;
          if (slot_copied(slot.at)) fence_async_proxy();
          tc_fence_after();
          const uint64_t v = v_desc + slot.at * (kSlotBytes >> 4);
          const uint32_t p = tmem + buf.at * TN;
#pragma unroll
          for (int c = 0; c < TN / 16; ++c)
            mma_ts(lead, tmem + C::kOCol, p + c * 8, v + c * (2048 >> 4), idesc_o,
                   (c != 0) || t > 0);
          mma_commit(lead, &S.pvdone[buf.at]);
          mma_commit(lead, &S.empty[slot.at]);
          slot.step();
          buf.step();
        }
      }
    }
  } else if (go && warp < kLoadWarp) {
    // --------------------------------------------------------------- softmax
    const uint32_t lanes = tmem + (uint32_t(warp * 32) << 16);
    Seg s;
    int g = 0;
    uint32_t looked = 0, collected = 0;
    Ring v_slot(C::kKSlots, C::kSlots - C::kKSlots, 0);
    Buf bf, done;                // of this tile, and of the one before (its product with V)
    for (int unit = 0;; ++unit) {
      bool stop = !next_seg(S, unit, s);
      if (unit == 0 && A.test_expire == int(blockIdx.x) + 1 && !stop &&
          !mbar_wait_for(smem_addr(&S.never), 0, kTestWaitNs)) {
        *reinterpret_cast<volatile int*>(&S.abort) = 1;
        stop = true;
      }
      if (softmax_any(stop)) break;
      const int apart = kTcMr / s.copies;
      const int copy = tid / apart, rr = tid % apart;   // warps lie in one copy
      const bool active = warp * 32 % apart < s.rows;
      const bool live = rr < s.rows;
      const int row = s.row0 + rr;
      const int tok = row / A.G;
      AttnNode node{0, 0};
      if constexpr (TREE) {
        // Every part's CTA looks at all the request's parents, so that a torn tree
        // fails in all of them.
        const int32_t* parents = A.parent + s.t_off;
        bool torn = false;
        if (tid > 0 && tid <= s.R.k && !s.R.code) {
          const int up = parents[tid];
          torn = up < 0 || up >= tid;
        }
        if (softmax_any(torn) && tid == 0) {
          S.bad[unit % kSegs] = 1;
          S.first_torn = min(S.first_torn, s.b);
        }
        node = attn_node(A, parents, s.R.n, min(tok, s.R.k));
      }
      const int at = TREE ? node.at : s.R.at0 + tok;
      const int row_hi =
          live ? (s.R.code ? 0 : TREE ? s.R.n : min(at + 1, s.R.hi)) : INT32_MAX;
      const int row_lo = live && A.window > 0 ? max(0, at - A.window + 1) : 0;
      // behind row_hi: nodes that the row sees
      const uint64_t row_path = TREE && live && !s.R.code ? node.path : 0;
      // the range that every row of the unit sees: tiles inside it need no mask
      const int at_first = s.R.at0 + s.row0 / A.G;
      // a tree is no deeper than its nodes are many
      const int at_last = TREE ? s.R.n + s.R.k : s.R.at0 + (s.row0 + s.rows - 1) / A.G;
      const int all_hi = s.R.code ? 0 : TREE ? s.R.n : min(at_first + 1, s.R.hi);
      const int all_lo = A.window > 0 ? max(0, at_last - A.window + 1) : 0;
      float m = -INFINITY, l = 0.f;   // m: the maximum that the sum and O refer to
      for (int t = 0; t < s.count; ++t, ++g, v_slot.step(), done = bf, bf.step()) {
        const int p0 = (s.R.tile0 + s.first + t) * TN;
        const int buf = bf.at;
        const bool edge = p0 < all_lo || p0 + TN > all_hi;
        const uint32_t scol = lanes + uint32_t(buf) * TN;
        if (!tc_wait_warp(&S.sfull[buf], bf.phase, S)) {
          stop = true;
          break;
        }
        tc_fence_after();
        uint32_t signs[2 * D / 32];   // non-finite values that the row sees
        bool dirty = false;
        if (edge) {
          // V of this tile: 128 bytes a thread
          const uint32_t slot = v_slot.at;
          if (!tc_wait_warp(&S.full[slot], v_slot.phase, S)) {
            stop = true;
            break;
          }
          uint4* v = reinterpret_cast<uint4*>(smem_p + C::kQBufs * C::kQBytes + slot * kSlotBytes);
          bool found = false;
#pragma unroll
          for (int i = 0; i < kSlotBytes / 16 / 128; ++i) {
            const uint4 w = v[i * 128 + tid];
            found |= any_nonfinite<T>(w.x) | any_nonfinite<T>(w.y) | any_nonfinite<T>(w.z) |
                     any_nonfinite<T>(w.w);
          }
          if (found) S.dirty[buf] = g + 1;
          if (!tc_sync(&S.looked[0], looked, S)) {
            stop = true;
            break;
          }
          looked ^= 1;
          dirty = *reinterpret_cast<volatile int*>(&S.dirty[buf]) == g + 1;
          if (dirty) {
            // each copy has the signs of its own columns: one without weight has none
            const int first = copy * (TN / s.copies);
            collect_signs<T, D, TN>(reinterpret_cast<const uint32_t*>(v), first,
                                    live ? first + TN / s.copies : first, row_lo - p0,
                                    row_hi - p0, row_path, row_hi - p0, signs);
            if (!tc_sync(&S.looked[1], collected, S)) {
              stop = true;
              break;
            }
            collected ^= 1;
#pragma unroll 1
            for (int i = 0; i < kSlotBytes / 16 / 128; ++i) {
              uint32_t* w = reinterpret_cast<uint32_t*>(v + i * 128 + tid);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t e = ((w[x] & Bits<T>::kExp) + Bits<T>::kOne) & 0x80008000u;
                w[x] &= ~((e >> 15) * 0xffffu);
              }
            }
            fence_async_proxy();
          }
        }
        // The warp's copy's share of the columns, N at a time (two rounds where
        // it has all of 128: the first round's scores are read again after the
        // maximum over both)
        auto weigh = [&](auto columns, auto rounds) -> bool {
          constexpr int N = decltype(columns)::value, ROUNDS = decltype(rounds)::value;
          const int c0 = copy * N;
          float x[N];
          auto fetch = [&](int round) {
#pragma unroll
            for (int c = 0; c < N / 32; ++c)
              tmem_ld32(scol + c0 + round * N + c * 32,
                        *reinterpret_cast<uint32_t(*)[32]>(&x[c * 32]));
            tmem_ld_wait();
            if (edge) {
              const int p = p0 + c0 + round * N;
              if constexpr (TREE) {
#pragma unroll
                for (int i = 0; i < N / 32; ++i) {
                  // a bit per column: cached positions, then nodes
                  const int q = p + i * 32, shift = row_hi - q;
                  uint32_t w = shift >= 32 ? ~0u : shift > 0 ? (1u << shift) - 1 : 0u;
                  if (row_lo > q) w = row_lo - q >= 32 ? 0u : w & (~0u << (row_lo - q));
                  if (shift < 32 && shift > -64)
                    w |= shift >= 0 ? uint32_t(row_path) << shift : uint32_t(row_path >> -shift);
#pragma unroll
                  for (int c = 0; c < 32; ++c)
                    x[i * 32 + c] = (w >> c) & 1 ? x[i * 32 + c] : -INFINITY;
                }
              } else {
#pragma unroll
                for (int c = 0; c < N; ++c)
                  x[c] = p + c >= row_lo && p + c < row_hi ? x[c] : -INFINITY;
              }
            }
          };
          float high = -INFINITY;
#pragma unroll
          for (int round = 0; round < ROUNDS; ++round) {
            fetch(round);
#pragma unroll
            for (int c = 0; c < N; ++c) high = fmaxf(high, x[c]);
          }
          const float grown = fmaxf(m, high * A.scale2);   // scale2 > 0
          const bool rescale = live && grown > m + kRescaleLog2;
          if (__any_sync(0xffffffffu, rescale)) {
            // all rows of the warp move to their present maximum
            const float f = m == -INFINITY ? 0.f : exp2f(m - grown);
            if (t > 0) {
              if (!tc_wait_warp(&S.pvdone[done.at], done.phase, S)) return false;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < dim / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(lanes + C::kOCol + c * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(lanes + C::kOCol + c * 16, o);
              }
            }
            l *= f;
            m = grown;
          }
          const float sh = (m == -INFINITY ? 0.f : m) - Bits<T>::kLift;
          const uint64_t sc2 = pk2(A.scale2, A.scale2), sh2 = pk2(-sh, -sh);
          uint64_t sum = pk2(0.f, 0.f);
          // the last round's scores are still there; P of a round lies over
          // scores that are read by then (of this or an earlier round)
          uint32_t held[ROUNDS > 1 ? N / 2 : 1];
#pragma unroll
          for (int round = ROUNDS - 1; round >= 0; --round) {
            if (round != ROUNDS - 1) fetch(round);
            uint32_t pw[N / 2];
#pragma unroll
            for (int c = 0; c < N; c += 2) {
              float e0, e1;
              upk2(fma2(pk2(x[c], x[c + 1]), sc2, sh2), e0, e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              sum = add2(sum, pk2(e0, e1));
              pw[c / 2] = Bits<T>::pack(e0, e1);
            }
            if (ROUNDS > 1 && round == 1) {
#pragma unroll
              for (int c = 0; c < N / 2; ++c) held[c] = pw[c];
            } else {
              // the other copies' columns are theirs: zeros here
              uint32_t zero[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) zero[c] = 0;
#pragma unroll
              for (int i = 0; i < TN / N / ROUNDS; ++i)
#pragma unroll
                for (int c = 0; c < N / 32; ++c) {
                  const uint32_t to = scol + i * (N / 2) + c * 16;
                  if (i == copy) tmem_st16(to, *reinterpret_cast<uint32_t(*)[16]>(&pw[c * 16]));
                  else tmem_st16(to, zero);
                }
              if constexpr (ROUNDS > 1) {
#pragma unroll
                for (int c = 0; c < N / 32; ++c)
                  tmem_st16(scol + N / 2 + c * 16,
                            *reinterpret_cast<uint32_t(*)[16]>(&held[c * 16]));
              }
            }
          }
          float s0, s1;
          upk2(sum, s0, s1);
          l += s0 + s1;
          tmem_st_wait();
          return true;
        };
        if (active) {
          bool ok;
          using One = std::integral_constant<int, 1>;
          if (s.copies == 1)
            ok = weigh(std::integral_constant<int, 64>(), std::integral_constant<int, TN / 64>());
          else if (s.copies == 2)
            ok = weigh(std::integral_constant<int, TN / 2>(), One());
          else
            ok = weigh(std::integral_constant<int, 32>(), One());
          if (!ok) {
            stop = true;
            break;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&S.pfull[buf]));
        if (dirty) {
          if (!tc_wait_warp(&S.pvdone[buf], bf.phase, S)) {
            stop = true;
            break;
          }
          tc_fence_after();
          if (active) add_signs<D>(lanes + C::kOCol, dim, signs);
          tc_fence_before();
        }
      }
      // ------------------------------------------------- the unit's rows
      if (!stop)
        stop = !tc_wait_two(&S.pvdone[done.at], done.phase, &S.noted[unit % kSegs],
                            (unit / kSegs) & 1, S);
      if (softmax_any(stop)) break;
      tc_fence_after();
      const bool bad = *reinterpret_cast<volatile int*>(&S.bad[unit % kSegs]) != 0;
      const float nan = __int_as_float(0x7fc00000);
      const int slot = s.first == 0 ? 1 : 0;
      const int64_t pr = (int64_t(blockIdx.x) * 2 + slot) * kTcMr;
      float top = m, total = l;
      auto place = [&](int r, int64_t* t, int* hq) {   // token and head of row r of the unit
        const int x = s.row0 + r;
        *t = int64_t(s.t_off) + x / A.G;
        *hq = s.h * A.G + x % A.G;
      };
      // Weights that are 0 in M's other copies, or too small for the type, times an
      // infinite value give NaN where the formula gives the infinity.  So where a
      // row of proper weights has NaN, the part's values are looked through once
      // more, and what their signs say takes its place.  Tiles [in0, in1) are seen
      // by every row; what the others hold is looked up row by row.  Looking for
      // NaN costs 1 % with 15 drafts (115.4 -> 116.9 us).
      const int part0 = s.R.tile0 + s.first, part1 = part0 + s.count;
      const int in0 = max(part0, (all_lo + TN - 1) / TN);
      const int in1 = max(in0, min(part1, all_hi / TN));
      auto value_of = [&](int p) -> const uint16_t* {
        int64_t v_off;
        const char* k = attn_key(A, s.b, s.R.n, p, &v_off);
        return k ? reinterpret_cast<const uint16_t*>(k + v_off) + int64_t(s.h) * dim : nullptr;
      };
      auto settle = [&](float v, int r, int d) {
        if (!isnan(v)) return v;
        uint32_t seen = ((S.signs[0][d >> 5] >> (d & 31)) & 1) |
                        (((S.signs[1][d >> 5] >> (d & 31)) & 1) << 1);
        const int t = (s.row0 + r) / A.G;
        const AttnNode node = TREE ? attn_node(A, A.parent + s.t_off, s.R.n, t) : AttnNode{0, 0};
        const int row_at = TREE ? node.at : s.R.at0 + t;
        const int lo = max(part0 * TN, A.window > 0 ? max(0, row_at - A.window + 1) : 0);
        const int hi = min(part1 * TN, TREE ? s.R.hi : min(row_at + 1, s.R.hi));
        for (int p = lo; p < hi && seen != 3; ++p) {
          if (p == in0 * TN) p = in1 * TN;
          if (TREE && p >= s.R.n && p < hi && !((node.path >> (p - s.R.n)) & 1)) continue;
          const uint16_t* x = p < hi ? value_of(p) : nullptr;
          if (x) seen |= value_signs<T>(x[d]);
        }
        return seen == 1 ? INFINITY : seen == 2 ? -INFINITY : v;
      };
      bool staged = s.copies > 1, settled = false;
      for (;;) {
        bool odd = false;   // a value of this thread's that is no number
        if (!staged) {
          const float inv = bad ? nan : total == 0.f ? 0.f : 1.f / total;
          int64_t trow;
          int hq;
          place(rr, &trow, &hq);
          if (active) {
#pragma unroll 1
            for (int c = 0; c * 32 < dim; ++c) {
              uint32_t o[32];
              tmem_ld32(lanes + C::kOCol + c * 32, o);
              tmem_ld_wait();
              if (!live) continue;
              bool any = false;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                any |= !(PART && c * 32 + e >= dim) && isnan(__uint_as_float(o[e]));
              odd |= any && inv == inv;
              if (s.whole) {
                T* out = static_cast<T*>(A.out) + trow * A.o_ts + int64_t(hq) * A.o_hs + c * 32;
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  w[e] = Bits<T>::pack(__uint_as_float(o[2 * e]) * inv,
                                       __uint_as_float(o[2 * e + 1]) * inv);
                if (A.out_vec) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    if (PART && c * 32 + e * 8 >= dim) break;
                    *reinterpret_cast<uint4*>(out + e * 8) =
                        make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                  }
                } else {
#pragma unroll
                  for (int e = 0; e < 32; ++e) {
                    if (PART && c * 32 + e >= dim) break;
                    const uint16_t h = uint16_t(w[e / 2] >> (16 * (e & 1)));
                    out[e] = *reinterpret_cast<const T*>(&h);
                  }
                }
              } else {
                uint4* po = reinterpret_cast<uint4*>(A.part_o + (pr + rr) * dim + c * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  if (PART && c * 32 + e * 4 >= dim) break;
                  po[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
              }
            }
          }
        } else {
          // The copies' sums and outputs add up at their common maximum, as many
          // columns of O at a time as fit; all threads then write them.
          Stage& stage = *reinterpret_cast<Stage*>(
              smem_p + (C::kOwnStage ? C::kQBufs * C::kQBytes + C::kSlots * kSlotBytes
                                     : unit % C::kQBufs * C::kQBytes));
          stage.ml[tid] = make_float2(m, l);
          softmax_sync();
          for (int c = 0; c < s.copies; ++c) top = fmaxf(top, stage.ml[rr + c * apart].x);
          total = 0.f;
          for (int c = 0; c < s.copies; ++c) {
            const float2 x = stage.ml[rr + c * apart];
            if (x.x > -INFINITY || x.y != x.y) total = fmaf(x.y, ex2_approx(x.x - top), total);
          }
          const float f = m > -INFINITY ? ex2_approx(m - top) : 0.f;
          if (live && copy == 0) {
            int64_t t;
            int hq;
            place(rr, &t, &hq);
            stage.out[rr] = t * A.o_ts + int64_t(hq) * A.o_hs;
            stage.inv[rr] = bad ? nan : total == 0.f ? 0.f : 1.f / total;
          }
          int cols = D;
          while (s.rows * s.copies * (cols + 1) > kStageFloats) cols >>= 1;
          const int half = cols / 2, shift = 31 - __clz(half);
#pragma unroll 1
          for (int c0 = 0; c0 < dim; c0 += cols) {
            if (active) {
              float* to = stage.o + (copy * s.rows + rr) * (cols + 1);
#pragma unroll 1
              for (int c = 0; c < cols; c += 32) {   // 32 columns fit whatever the rows
                uint32_t o[32];
                tmem_ld32(lanes + C::kOCol + c0 + c, o);
                tmem_ld_wait();
                if (live) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) to[c + e] = __uint_as_float(o[e]) * f;
                }
              }
            }
            softmax_sync();
            for (int i = tid; i < s.rows * half; i += 128) {
              const int r = i >> shift, e = (i & (half - 1)) * 2;
              if (PART && c0 + e >= dim) continue;
              float v0 = 0.f, v1 = 0.f;
              for (int k = 0; k < s.copies; ++k) {
                const float* from = stage.o + (k * s.rows + r) * (cols + 1) + e;
                v0 += from[0];
                v1 += from[1];
              }
              if ((isnan(v0) || isnan(v1)) && stage.inv[r] == stage.inv[r]) {
                if (settled) {
#pragma unroll 1
                  for (int x = 0; x < 2; ++x) {
                    const float v = settle(x ? v1 : v0, r, c0 + e + x);
                    (x ? v1 : v0) = v;
                  }
                }
                odd = true;
              }
              if (s.whole) {
                T* out = static_cast<T*>(A.out) + stage.out[r] + c0 + e;
                const uint32_t w = Bits<T>::pack(v0 * stage.inv[r], v1 * stage.inv[r]);
                if (A.out_vec) {
                  *reinterpret_cast<uint32_t*>(out) = w;
                } else {
                  const uint16_t h0 = uint16_t(w), h1 = uint16_t(w >> 16);
                  out[0] = *reinterpret_cast<const T*>(&h0);
                  out[1] = *reinterpret_cast<const T*>(&h1);
                }
              } else {
                *reinterpret_cast<float2*>(A.part_o + (pr + r) * dim + c0 + e) =
                    make_float2(v0, v1);
              }
            }
            if (c0 + cols < dim) softmax_sync();   // the last columns: the barrier below
          }
        }
        if (settled || !softmax_any(odd)) break;
        // signs of the infinite and NaN values that every row sees
        if (tid < 2 * D / 32) S.signs[tid / (D / 32)][tid % (D / 32)] = 0;
        softmax_sync();
        for (int p = in0 * TN + tid; p < in1 * TN; p += 128) {
          const uint4* v = reinterpret_cast<const uint4*>(value_of(p));
          for (int c = 0; v && c < dim / 8; ++c) {
            const uint4 x = v[c];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            for (int i = 0; i < 8; ++i) {
              const uint32_t seen = value_signs<T>(w[i / 2] >> (16 * (i & 1)));
              const int d = c * 8 + i;
              if (seen & 1) atomicOr(&S.signs[0][d >> 5], 1u << (d & 31));
              if (seen & 2) atomicOr(&S.signs[1][d >> 5], 1u << (d & 31));
            }
          }
        }
        softmax_sync();
        staged = settled = true;
      }
      if (live && copy == 0) {
        int64_t trow;
        int hq;
        place(rr, &trow, &hq);
        const float ref = top - Bits<T>::kLift;   // what O and the sum refer to
        if (s.whole)
          A.lse[trow * A.Hq + hq] =
              bad ? nan : (ref == -INFINITY ? 0.f : ref * kAttnLn2) + logf(total);
        else
          A.part_ml[pr + rr] = make_float2(bad ? nan : ref, total);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_addr(&S.ofree));
        mbar_arrive(smem_addr(&S.qempty[unit % C::kQBufs]));
      }
      if (tid == 0 && !s.whole && s.first == 0) begin_split(A, P, s);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (S.abort) give_up<T, D>(A, S);
  if (tid == 0)
    A.status[A.B + blockIdx.x] = S.abort ? -SV_ERR_TIMEOUT : S.first_bad;
  if (TREE && tid == 0) A.status[A.B + A.ctas + blockIdx.x] = S.first_torn;
  if (warp == kValueWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
  }
}

template <class T, int D, bool PART, bool TREE>
cudaError_t run(const AttnArgs& A, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(attn_tc_kernel<T, D, PART, TREE>, Shape<D>::kSmem, configured))
    return e;
  CUtensorMap map;
  AttnArgs B = A;
  B.box_rows = box_rows(A.S, Shape<D>::TN, D, 32);
  if (!rows_map(&map, B, Bits<T>::kFmt != 0)) return cudaErrorInvalidValue;
  attn_tc_kernel<T, D, PART, TREE><<<A.ctas, kTcThreads, Shape<D>::kSmem, s>>>(map, B);
  return cudaGetLastError();
}

template <class T, bool TREE>
cudaError_t run_dim(const AttnArgs& A, cudaStream_t s) {
  if (A.D == 64) return run<T, 64, false, TREE>(A, s);
  if (A.D <= 128)
    return A.D == 128 ? run<T, 128, false, TREE>(A, s) : run<T, 128, true, TREE>(A, s);
  return A.D == 256 ? run<T, 256, false, TREE>(A, s) : run<T, 256, true, TREE>(A, s);
}

template <bool TREE>
cudaError_t run_type(const AttnArgs& A, int dtype, cudaStream_t s) {
  return dtype == SV_BF16 ? run_dim<__nv_bfloat16, TREE>(A, s) : run_dim<__half, TREE>(A, s);
}

}  // namespace
}  // namespace sv
