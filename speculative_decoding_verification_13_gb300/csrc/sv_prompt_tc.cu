// Causal attention over packed prompts on the fifth-generation tensor cores, for
// bf16 and fp16 and heads of up to 256 elements that lie on 16 bytes (taken at D,
// the next of 64, 128 and 256; what lies behind a head is filled with zeros by the
// copy engine).
//
// A row tile is 128 / G tokens of one KV head with the G query heads that share
// it, the M of the products: row r is token r / G, head r % G, and the rows of a
// tile are one box of the copy engine.  A unit is NQ row tiles that follow one
// another (two, one for heads of 256, whose output takes half of TMEM) over the
// tiles of TN positions that they see: S = Q K^T (128 x TN x D), P = exp S, O += P V
// (128 x D x TN).  With two row tiles one's softmax runs during the other's
// products, and every tile of K and V serves both.
//
// One CTA per SM, over units u = c, 2 n - 1 - c, 2 n + c, ... (n CTAs, forth and back)
// in the order of the tokens' place in their sequence, the last first: what a unit
// costs falls with its number, so that the CTAs' sums stay close without a queue (24
// sequences of 1 to 4000 tokens: the most 97 tiles a CTA, the mean 93).
//   warps 0-3, 4-7  softmax of the first and the second row tile, one row a thread
//                   (the lanes of TMEM): scores from TMEM, running maximum, P rounded
//                   to the type (half a step of it, the one rounding of a weight;
//                   sums stay in 32 bits) back over the scores, where the second
//                   product reads it as its A operand.  O is rescaled only when a
//                   row's maximum has grown by more than 2^8 since the last time.
//   warp 8          finds the units, announces them, and has the copy engine load Q,
//                   K and V into rings of slots, 128-byte swizzled.
//   warp 9          issues the products.  The tensor cores run them in the order of
//                   issue, so that S of the next tile may follow the product that
//                   reads P in the same place.  A warp for each row tile instead, with
//                   or without turns, 1350 us -> 1480 to 1680 on the case below: their
//                   products come between one another's.
//   warps 10, 11    look through V of the tiles that some row of the unit sees in
//                   part: masked weights are 0, but 0 times an infinite or NaN value
//                   would still reach the row.  If such a tile holds any, each row
//                   collects the signs of those that it sees, they are replaced by 0,
//                   and added to the row's O afterwards.  (A weight that is 0 in the
//                   type, more than 2^126 below its row's largest, 2^31 in fp16, times
//                   an infinite value in any other tile is NaN.)
//
// Every wait is bounded; on expiry the CTA's status records it, its copies and
// products land, TMEM is freed, and the rows of all its units become NaN.
//
// Measured, 32 + 8 heads of 128 in bf16: 16001 tokens 1.34 ms, 1560 TFLOP/s of what the
// visible pairs take; 4 times 2048 tokens 120 us, 1140; 201 tokens 12 us.  Heads of 64
// 960 TFLOP/s, of 256 1300 (8 to 16 thousand tokens).  Bound by a row tile's round:
// softmax 1200 to 1300 cycles, products 1050, and about 600 from barrier to barrier,
// 2950 where the products of both row tiles take 2050; then by a unit's end (its last
// product, 2500 cycles of output, the next unit's first scores: 6000 in all).  Heads of
// 64: a product with V takes as long for 64 columns as for 128.
#include <type_traits>

#include "sv_attn_tc.cuh"
#include "sv_prompt.cuh"

namespace sv {
namespace {

constexpr int kPtThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLookWarp = 10;
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

// One unit.  The load warp finds them, a few ahead, and announces them to the
// others; n 0 is the end.
struct PtSeg {
  int row0;       // first row of the sequence
  int h;          // KV head
  int tok0;       // first token
  int tile0, n;   // tiles of positions
  int cnt[2];     // of them what each row tile sees, from the first on
  int live[2];    // tokens of each row tile
};

struct PtShared {
  PtSeg seg[kSegs];
  uint64_t announced[kSegs], taken[kSegs];
  uint64_t full[10], empty[10];
  uint64_t looked[10], clean[10];   // of V slots: looked through; nothing to be kept out
  uint64_t qfull[2], qempty[2], ofree[2];
  // Per S accumulator: with two, a warp may be a tile ahead of another, and a tile's
  // product two tiles behind the scores, whose barriers' parities would be alike.
  uint64_t sfull[2][2], pfull[2][2], pvdone[2][2];
  uint64_t collected[2];            // the row tile has the signs of a dirty tile
  uint64_t drain, never;
  int dirty[10][2];                 // per V slot and looking warp
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

__device__ __forceinline__ bool pt_next_seg(PtShared& S, int unit, PtSeg& s) {
  if (!tc_wait_warp(&S.announced[unit % kSegs], (unit / kSegs) & 1, S)) return false;
  s = S.seg[unit % kSegs];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&S.taken[unit % kSegs]));
  return s.n > 0;
}

// A thread's signs of the infinite (NaN: both) values among the columns lo .. hi - 1
// of a tile of V: bits of columns of the head, +inf then -inf.
template <class T, int D, int TN>
__device__ __noinline__ void collect_signs(const uint32_t* v, int lo, int hi, uint32_t* signs) {
  for (int i = 0; i < 2 * D / 32; ++i) signs[i] = 0;
  for (int c = max(lo, 0); c < min(hi, TN); ++c)
    for (int d = 0; d < D; d += 2) {
      const uint32_t w =
          v[(d >> 6) * (TN * 32) + c * 32 + ((((d & 63) >> 3) ^ (c & 7)) << 2) + ((d & 7) >> 1)];
      if (!any_nonfinite<T>(w)) continue;
      for (int x = 0; x < 2; ++x) {
        const uint32_t y = (w >> (16 * x)) & 0xffffu;
        if ((y & Bits<T>::kExp1) != Bits<T>::kExp1) continue;
        const bool isnan = (y & Bits<T>::kMan1) != 0;
        const uint32_t bit = 1u << ((d + x) & 31);
        if (isnan || !(y & 0x8000u)) signs[d >> 5] |= bit;
        if (isnan || (y & 0x8000u)) signs[D / 32 + (d >> 5)] |= bit;
      }
    }
}

// Adds them to the thread's row of O.
template <int D>
__device__ __noinline__ void add_signs(uint32_t o_at, int dim, const uint32_t* signs) {
  for (int c = 0; c * 16 < dim; ++c) {
    uint32_t o[16];
    tmem_ld16(o_at + c * 16, o);
    tmem_ld_wait();
    const uint32_t plus = signs[c >> 1] >> (16 * (c & 1)),
                   minus = signs[D / 32 + (c >> 1)] >> (16 * (c & 1));
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float x = __uint_as_float(o[e]);
      if ((plus >> e) & 1) x += INFINITY;
      if ((minus >> e) & 1) x -= INFINITY;
      o[e] = __float_as_uint(x);
    }
    tmem_st16(o_at + c * 16, o);
  }
  tmem_st_wait();
}

// All threads, after a wait of the CTA expired and every warp has left its loop:
// what was issued has landed; every row of the CTA's units becomes NaN.
template <class T, int D>
__device__ __noinline__ void pt_give_up(const PromptArgs& A, PtShared& S) {
  using C = PtShape<D>;
  const float nan = __int_as_float(0x7fc00000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PtWalk<C::NQ> walk(A, S.top);
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

template <class T, int D, bool PART>
__global__ void __launch_bounds__(kPtThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map,
                     const __grid_constant__ PromptArgs A) {
  using C = PtShape<D>;
  constexpr int TN = C::TN, NQ = C::NQ, NB = C::NB;
  constexpr int kSlotBytes = C::kSlotBytes;
  extern __shared__ unsigned char pt_smem_raw[];
  __shared__ PtShared S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_addr(pt_smem_raw) + 1023u) & ~1023u;
  unsigned char* smem_p = pt_smem_raw + (smem0 - smem_addr(pt_smem_raw));
  const uint32_t ring0 = smem0 + NQ * C::kQBytes;
  const int dim = PART ? A.D : D;
  const int parts = PART ? (A.D + 63) / 64 : D / 64;
  const int toks = kM / A.G;

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_addr(&S.full[i]), 1);
      mbar_init(smem_addr(&S.empty[i]), 1);
      mbar_init(smem_addr(&S.looked[i]), 2);
      mbar_init(smem_addr(&S.clean[i]), 2);
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
      mbar_init(smem_addr(&S.taken[i]), 4 * NQ + 3);   // every warp but the load warp
    }
    for (int g = 0; g < 2; ++g) mbar_init(smem_addr(&S.collected[g]), 4);
    mbar_init(smem_addr(&S.drain), 1);
    mbar_init(smem_addr(&S.never), 1);
    fence_mbar_init();
    S.abort = S.bad = S.top = 0;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&S.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncthreads();
  // the sequences, looked through by every CTA
  {
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
  const bool go = S.bad == 0;
  if (!go) prompt_fail<T>(A);

  if (go && warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ------------------------------------------------------- units and loads
      Ring kr(0, C::kKSlots, 1), vr(C::kKSlots, C::kSlots - C::kKSlots, 1);
      int kfilled = 0, vfilled = 0, quse[2] = {0, 0};
      bool stop = false;
      const uint32_t lead = lane == 0;
      PtWalk<NQ> walk(A, S.top);
      PtSeg next;
      walk.template next<TN>(A, next);
      for (int unit = 0;; ++unit) {
        const PtSeg s = next;
        // this entry's unit before has been taken over by every warp
        stop = !tc_wait_warp(&S.taken[unit % kSegs], ((unit / kSegs) & 1) ^ 1, S);
        if (stop) break;
        if (lead) {
          S.seg[unit % kSegs] = s;
          mbar_arrive(smem_addr(&S.announced[unit % kSegs]));
        }
        __syncwarp();
        if (s.n == 0) break;
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
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          if (s.cnt[g] == 0 || stop) continue;
          stop = !tc_wait_warp(&S.qempty[g], (quse[g]++ & 1) ^ 1, S);
          if (lead && !stop) {
            const uint32_t bar = smem_addr(&S.qfull[g]);
            mbar_arrive_expect_tx(bar, uint32_t(parts * toks * A.G * 128));
            for (int p = 0; p < parts; ++p)
              box_load3(smem0 + g * C::kQBytes + p * (kM * 128), &q_map, p * 64, s.h * A.G,
                        s.row0 + s.tok0 + g * toks, bar);
          }
          __syncwarp();
        }
        for (int t = 0; t < s.n && !stop; ++t) {
          stop = !load(kr, &k_map, t);
          kfilled += !stop;
          if (!stop) {
            stop = !load(vr, &v_map, t);
            vfilled += !stop;
          }
          if (t == 0) walk.template next<TN>(A, next);   // while the first tile is on its way
        }
        if (stop) break;
      }
      if (stop) {   // let the copies that were issued land
        ring_land(kr, kfilled, S.full);
        ring_land(vr, vfilled, S.full);
        for (int g = 0; g < NQ; ++g)
          if (quse[g] > 0) mbar_wait_for(smem_addr(&S.qfull[g]), (quse[g] - 1) & 1, kTestWaitNs);
      }
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
      auto score = [&](int g, const PtSeg& s, int t) {   // S of row tile g
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
        PtSeg s;
        ok = pt_next_seg(S, unit, s);
        if (!ok) break;
        ok = tc_wait_warp(&S.full[kr.at], kr.phase, S);
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          if (!ok || s.cnt[g] == 0) continue;
          ok = tc_wait_warp(&S.qfull[g], quse[g]++ & 1, S);
          if (!ok) break;
          tc_fence_after();
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
            tc_fence_after();
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
            ok = tc_wait_two(&S.full[vr.at], vr.phase, &S.clean[vr.at], vr.phase, S) &&
                 tc_wait_warp(&S.pfull[g][buf], (NB == 2 ? pcount[g] >> 1 : pcount[g]) & 1, S);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = v_desc + vr.at * (kSlotBytes >> 4);
            const uint32_t p = tmem + (g * NB + buf) * TN;
#pragma unroll
            for (int c = 0; c < TN / 16; ++c)
              mma_ts(lead, tmem + C::kOCol + g * D, p + c * 8, v + c * (2048 >> 4), idesc_o,
                     (c != 0) || t > 0);
            mma_commit(lead, &S.pvdone[g][buf]);
            ++pcount[g];
            if (NB == 1 && t + 1 < s.cnt[g]) {
              ok = tc_wait_warp(&S.full[kr.at], kr.phase, S);
              if (!ok) break;
              tc_fence_after();
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
      const int w = warp - kLookWarp;
      Ring vr(C::kKSlots, C::kSlots - C::kKSlots, 0);
      uint32_t dirties[2] = {0, 0};
      bool ok = true;
      for (int unit = 0; ok; ++unit) {
        PtSeg s;
        ok = pt_next_seg(S, unit, s);
        if (!ok) break;
        const int last = s.tok0 + s.live[0] + s.live[1] - 1;
        const int all_hi = s.tok0 + 1, all_lo = A.window > 0 ? max(0, last - A.window + 1) : 0;
        for (int t = 0; t < s.n; ++t, vr.step()) {
          const int p0 = (s.tile0 + t) * TN;
          ok = tc_wait_warp(&S.full[vr.at], vr.phase, S);
          if (!ok) break;
          const bool edge = p0 < all_lo || p0 + TN > all_hi;
          if (!edge) {
            if (lane == 0) {
              mbar_arrive(smem_addr(&S.looked[vr.at]));
              mbar_arrive(smem_addr(&S.clean[vr.at]));
            }
            continue;
          }
          constexpr int kVecs = kSlotBytes / 16 / 2;   // a warp's half
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
      PtSeg s;
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
      const int row_hi = live ? tok + 1 : INT32_MAX;
      const int row_lo = live && A.window > 0 ? max(0, tok - A.window + 1) : 0;
      // what all rows of the unit see, and all of this row tile
      const int last = s.tok0 + s.live[0] + s.live[1] - 1;
      const int all_hi = s.tok0 + 1, all_lo = A.window > 0 ? max(0, last - A.window + 1) : 0;
      const int own_hi = tok0 + 1,
                own_lo = A.window > 0 ? max(0, tok0 + s.live[g] - A.window) : 0;
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
        if (p0 < all_lo || p0 + TN > all_hi) {
          ok = tc_wait_warp(&S.looked[vr.at], vr.phase, S);
          if (!ok) break;
          const volatile int* d = S.dirty[vr.at];
          dirty = (d[0] | d[1]) != 0;
          if (dirty) {
            collect_signs<T, D, TN>(
                reinterpret_cast<const uint32_t*>(smem_p + NQ * C::kQBytes + vr.at * kSlotBytes),
                row_lo - p0, live ? row_hi - p0 : 0, signs);
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
        if (p0 + TN > own_hi) {
          const int hi = row_hi - p0;
#pragma unroll
          for (int c = 0; c < TN; ++c) x[c] = c < hi ? x[c] : -INFINITY;
        }
        if (p0 < own_lo) {
          const int lo = row_lo - p0;
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
      if (cnt == 0) continue;
      // ------------------------------------------------- the row tile's rows
      ok = product_done(count - 1);
      if (!ok) break;
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
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
          // w[i]: the lane's row's piece i, then row i's (of the four lanes') piece `piece`
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
          const int col = c * 32 + piece * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < live_rows && !(PART && col >= dim))
              *reinterpret_cast<uint4*>(unit_out + int64_t(quad_row[i]) * A.D + col) =
                  make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c * 32 < dim; ++c) {
          uint32_t o[32];
          tmem_ld32(o_at + c * 32, o);
          tmem_ld_wait();
          if (!live) continue;
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] =
                Bits<T>::pack(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (PART && c * 32 + e >= dim) break;
            const uint16_t y = uint16_t(w[e / 2] >> (16 * (e & 1)));
            out[c * 32 + e] = *reinterpret_cast<const T*>(&y);
          }
        }
      }
      if (live) {
        const float ref = m - Bits<T>::kLift;   // what O and the sum refer to
        A.lse[to] = (ref == -INFINITY ? 0.f : ref * kAttnLn2) + logf(l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&S.ofree[g]));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (go && S.abort) pt_give_up<T, D>(A, S);
  if (tid == 0) A.status[1 + blockIdx.x] = S.abort ? -SV_ERR_TIMEOUT : INT32_MAX;
  if (blockIdx.x == 0 && tid == 0) prompt_header(A, !go, gridDim.x);
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

template <class T, int D, bool PART>
cudaError_t run(const PromptArgs& A, int sms, cudaStream_t s) {
  using C = PtShape<D>;
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(prompt_tc_kernel<T, D, PART>, C::kSmem, configured)) return e;
  const bool bf16 = Bits<T>::kFmt != 0;
  CUtensorMap q, k, v;
  if (!heads_map(&q, A.q, bf16, A.D, A.Hq, A.rows, A.q_ts, A.q_hs, A.G, kM / A.G) ||
      !heads_map(&k, A.k, bf16, A.D, A.Hkv, A.rows, A.k_ts, A.k_hs, 1, C::TN) ||
      !heads_map(&v, A.v, bf16, A.D, A.Hkv, A.rows, A.v_ts, A.v_hs, 1, C::TN))
    return cudaErrorInvalidValue;
  prompt_tc_kernel<T, D, PART><<<unsigned(sms), kPtThreads, C::kSmem, s>>>(q, k, v, A);
  return cudaGetLastError();
}

template <class T>
cudaError_t run_dim(const PromptArgs& A, int sms, cudaStream_t s) {
  if (A.D <= 64) return A.D == 64 ? run<T, 64, false>(A, sms, s) : run<T, 64, true>(A, sms, s);
  if (A.D <= 128) return A.D == 128 ? run<T, 128, false>(A, sms, s) : run<T, 128, true>(A, sms, s);
  return A.D == 256 ? run<T, 256, false>(A, sms, s) : run<T, 256, true>(A, sms, s);
}

}  // namespace

// Types, heads and addresses that the copy engine and the products take.  The
// largest score is found before the scaling, so the scale has to be positive.
bool prompt_on_tensor_cores(const PromptArgs& A, int dtype) {
  auto boxes = [&](const void* p, int64_t ts, int64_t hs, int heads) {
    auto stride = [](int64_t x) { return x > 0 && x % 8 == 0 && x < (int64_t(1) << 38); };
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (A.rows == 1 || stride(ts)) &&
           (heads == 1 || stride(hs));
  };
  return dtype != SV_F32 && A.D % 8 == 0 && A.D <= 256 && A.G <= kM && A.scale2 > 0.0f &&
         boxes(A.q, A.q_ts, A.q_hs, A.Hq) && boxes(A.k, A.k_ts, A.k_hs, A.Hkv) &&
         boxes(A.v, A.v_ts, A.v_hs, A.Hkv);
}

cudaError_t launch_prompt_tc(const PromptArgs& A, int dtype, int sms, cudaStream_t s) {
  return dtype == SV_BF16 ? run_dim<__nv_bfloat16>(A, sms, s) : run_dim<__half>(A, sms, s);
}

}  // namespace sv
