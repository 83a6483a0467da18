// What the tensor-core kernels of attention and of its weights share: rings of
// tiles, waits, products, and the loading of a tile of keys or values from the
// paged cache and the speculative entries.
#pragma once

#include "sv_attn.cuh"
#include "sv_tcgen05.cuh"

namespace sv {

// A place in a ring of slots and the phase of its barriers.  K and V have rings
// of their own: with one for both, a load warp could meet a barrier two phases
// behind, whose parity is that of the phase it waits for.
struct Ring {
  uint32_t at, phase, base, end;
  __device__ __forceinline__ Ring(uint32_t first, uint32_t n, uint32_t phase_)
      : at(first), phase(phase_), base(first), end(first + n) {}
  __device__ __forceinline__ void step() {
    if (++at == end) {
      at = base;
      phase ^= 1;
    }
  }
};

// After a wait expired: waits (bounded) until the copies into the ring's last
// slots have landed, since the shared memory that they are to fill is the block's
// only until it ends.  `at`: where the next tile would have gone, its phase that of
// the slot's empty barrier; a slot's tile before ended the full barrier's phase of
// the opposite parity.
__device__ __forceinline__ void ring_land(Ring at, int filled, uint64_t* full) {
  for (int i = min(filled, int(at.end - at.base)); i > 0; --i) {
    if (at.at == at.base) {
      at.at = at.end;
      at.phase ^= 1;
    }
    --at.at;
    mbar_wait_for(smem_addr(&full[at.at]), at.phase ^ 1);
  }
  __syncwarp();
}

// A type's bits, and kLift: weights are held 2^kLift times as large.  The
// smallest normal number of fp16 is 2^-14, so that weights of long contexts
// would lose bits; with the lift and at most 2^8 above the stored maximum they
// stay below its largest, 65504, and are normal down to 2^-21 of the maximum.
template <class T> struct Bits;
template <> struct Bits<__nv_bfloat16> {
  static constexpr float kLift = 0.f;
  static constexpr uint32_t kFmt = 1, kExp = 0x7f807f80u, kOne = 0x00800080u, kExp1 = 0x7f80u,
                            kMan1 = 0x007fu;
  __device__ static uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Bits<__half> {
  static constexpr float kLift = 7.f;
  static constexpr uint32_t kFmt = 0, kExp = 0x7c007c00u, kOne = 0x04000400u, kExp1 = 0x7c00u,
                            kMan1 = 0x03ffu;
  __device__ static uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
// any of the two 16-bit values of w infinite or NaN
template <class T>
__device__ __forceinline__ bool any_nonfinite(uint32_t w) {
  return (((w & Bits<T>::kExp) + Bits<T>::kOne) & 0x80008000u) != 0;
}

// The products and their commits are issued by one lane of a warp that runs
// them as a whole: predicated instructions, no branch, so that descriptors stay
// in the warp's uniform registers (one lane in a branch of its own had to move
// every operand there: about 100 cycles a product).
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 e, %5, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 e, %5, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(bar)),
      "r"(lead)
      : "memory");
}

// 8 elements of a head of q, in one load where they lie on 16 bytes.
template <bool VEC, class T>
__device__ __forceinline__ uint4 load_chunk(const T* p) {
  if (VEC) return __ldg(reinterpret_cast<const uint4*>(p));
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = uint32_t(h[2 * i]) | uint32_t(h[2 * i + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// This lane's arrival on a barrier, made when its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

constexpr uint32_t kPollsPerLook = 256;

// Whether a wait that has polled `polls` times, and its CTA, should give up: looked at
// now and then.  Not inlined: a wait's own instructions are few, and a kernel has dozens
// of them.
template <class Sh>
__device__ __noinline__ bool tc_expired(uint32_t polls, uint64_t* since, Sh& S) {
  if (*reinterpret_cast<volatile int*>(&S.abort)) return true;
  const uint64_t now = global_ns();
  if (polls == kPollsPerLook) *since = now;
  if (now - *since <= kWaitNs && polls < kWaitPolls) return false;
  *reinterpret_cast<volatile int*>(&S.abort) = 1;
  return true;
}

// Bounded wait on a barrier of a CTA whose shared record is S; false, with its
// abort flag set, on expiry.
template <class Sh>
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, Sh& S) {
  const uint32_t at = smem_addr(bar);
  uint64_t since;
#pragma unroll 1
  for (uint32_t polls = 1;; ++polls) {
    if (mbar_try_wait(at, parity)) return true;
    if (polls % kPollsPerLook == 0 && tc_expired(polls, &since, S)) return false;
  }
}
// The same for a whole warp, one answer for all its lanes.
template <class Sh>
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, Sh& S) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, S));
}
// Two barriers at once: their polls overlap (a poll that succeeds still takes
// about 100 cycles between two products).
template <class Sh>
__device__ __forceinline__ bool tc_wait_two(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                            Sh& S) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p, q;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      "and.pred p, p, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(a)), "r"(pa), "r"(smem_addr(b)), "r"(pb)
      : "memory");
  if (__all_sync(0xffffffffu, ok != 0)) return true;
  return tc_wait_warp(a, pa, S) && tc_wait_warp(b, pb, S);
}
// Barrier of the four warps that count on `bar`, bounded like every other wait
// (a warp that gave up would leave a hardware barrier waiting for ever).
template <class Sh>
__device__ __forceinline__ bool tc_sync(uint64_t* bar, uint32_t parity, Sh& S) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(bar));
  return tc_wait_warp(bar, parity, S);
}


// Heads of any multiple of 16 from 64 on are taken at D, the next of 64, 128 and
// 256: PART says that the head is narrower than D.  What lies behind it in a slot
// (entries of the next head, or nothing) is in no product: scores end at the
// head's last 16 elements, and products with V have its columns only.
template <int D, bool PART>
__device__ __forceinline__ int head_width(const AttnArgs& A) {
  return PART ? A.D : D;
}
// 128-byte parts of a row
template <int D, bool PART>
__device__ __forceinline__ int row_parts(const AttnArgs& A) {
  return PART && D > 128 ? (A.D + 63) / 64 : D / 64;
}

// The pages of one tile: of this lane's box (the first), or of its rows lane +
// 32 i where the tile does not come in boxes.  SHARES warps may load a tile
// together, each every SHARES-th box or its share of the rows.
template <int TN, int SHARES>
struct TilePages {
  int page[TN / 32 / SHARES];
};

__device__ __forceinline__ int page_column(const AttnArgs& A, int p) {
  return int(uint64_t(uint32_t(p)) * A.s_mul >> A.s_shift);
}

// A tile comes in boxes where it is whole and pages hold a multiple of 8 of its
// positions.
template <int TN>
__device__ __forceinline__ bool tile_boxed(const AttnArgs& A, int cached, int p0) {
  return A.box_rows > 0 && p0 + TN <= cached;
}

template <int TN, int SHARES>
__device__ __forceinline__ TilePages<TN, SHARES> row_pages(const AttnArgs& A, const int32_t* table,
                                                        int cached, int p0, int share) {
  TilePages<TN, SHARES> t;
#pragma unroll
  for (int i = 0; i < TN / 32 / SHARES; ++i) {
    const int p = p0 + share * (TN / SHARES) + (threadIdx.x & 31) + 32 * i;
    t.page[i] = p < cached ? __ldg(table + page_column(A, p)) : 0;
  }
  return t;
}

template <int D, bool PART, int TN, int SHARES = 1>
__device__ __forceinline__ TilePages<TN, SHARES> tile_pages(const AttnArgs& A,
                                                            const int32_t* table, int cached,
                                                            int p0, int share = 0) {
  const int lane = threadIdx.x & 31;
  if (!tile_boxed<TN>(A, cached, p0)) return row_pages<TN, SHARES>(A, table, cached, p0, share);
  TilePages<TN, SHARES> t;
  const int box0 = (lane * SHARES + share) / row_parts<D, PART>(A) * A.box_rows;
  t.page[0] = box0 < TN ? __ldg(table + page_column(A, p0 + box0)) : 0;
  return t;
}

// The rows of a tile that does not come in boxes, 16 bytes at a time.  Like row_pages not
// inlined: they are most of a load's instructions, and most tiles come in boxes.
template <int D, bool PART, int TN, int SHARES>
__device__ __noinline__ void load_rows(const AttnArgs& A, TilePages<TN, SHARES> pages, int b, int n,
                                       int cached, int hi, int p0, int h, int kv, uint32_t dst,
                                       int share) {
  const int lane = threadIdx.x & 31;
  const int dim = head_width<D, PART>(A);
  // addresses of the lane's own rows; each round's lanes then fetch theirs from
  // the lane that has it
  constexpr int kOwn = TN / 32 / SHARES;
  const int first = share * (TN / SHARES);
  uint64_t own[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int p = p0 + first + lane + 32 * i;
    const char* a = nullptr;   // stays null for a row that is filled with zeros
    if (p >= cached) {
      if (p < hi)
        a = A.spec + int64_t(b) * A.spec_req + int64_t(p - n) * A.spec_tok + kv * A.entry_bytes;
    } else if (pages.page[i] >= 0) {
      a = A.cache + pages.page[i] * A.page_bytes + kv * A.v_off +
          (p - page_column(A, p) * A.S) * A.entry_bytes;
    }
    own[i] = a ? reinterpret_cast<uint64_t>(a + int64_t(h) * dim * 2) : 0;
  }
  constexpr int kChunks = D / 8, kStep = 32 / kChunks;   // 16-byte chunks of a row, rows a round
  const int ch = lane % kChunks;
  const char* none = A.spec ? A.spec : A.cache;   // not read, but on 16 bytes
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
#pragma unroll 4
    for (int j = 0; j < 32; j += kStep) {
      const int from = j + lane / kChunks, r = first + 32 * i + from;
      const uint64_t a = (uint64_t(__shfl_sync(0xffffffffu, uint32_t(own[i] >> 32), from)) << 32) |
                         __shfl_sync(0xffffffffu, uint32_t(own[i]), from);
      if (PART && ch * 8 >= dim) continue;
      cp_async16(dst + (ch >> 3) * (TN * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                 a ? reinterpret_cast<const char*>(a) + ch * 16 : none, a ? 16u : 0u);
    }
}

// A warp loads its share of K (kv 0) or V (kv 1) of head h and positions p0 ..
// p0 + TN - 1 of request b into the slot at dst: [D / 64][TN][64] of 16 bits,
// 128-byte swizzled.  `full` counts 32 arrivals a share; `copied` tells how the
// tile came.  missing(page) is true, and notes it, for a page that is not in the
// pool.
template <int D, bool PART, int TN, int SHARES, class F>
__device__ __forceinline__ void load_tile(const AttnArgs& A, const CUtensorMap& map,
                                          const TilePages<TN, SHARES>& pages, int b, int n,
                                          int cached, int hi, int p0, int h, int kv, uint32_t dst,
                                          uint64_t* full, int* copied, uint64_t policy, int share,
                                          F missing) {
  const int lane = threadIdx.x & 31;
  const uint32_t bar = smem_addr(full);
  const int dim = head_width<D, PART>(A);
  if (tile_boxed<TN>(A, cached, p0)) {
    const int parts = row_parts<D, PART>(A);
    if (lane == 0) {
      const int boxes = (TN / A.box_rows * parts - share + SHARES - 1) / SHARES;
      *copied = 0;
      mbar_arrive_expect_tx(bar, uint32_t(boxes * A.box_rows * 128));
    } else {
      mbar_arrive(bar);
    }
    __syncwarp();
    const int box = lane * SHARES + share;   // this lane's box
    const int part = box % parts, box0 = box / parts * A.box_rows;
    if (box0 < TN) {
      const int p = p0 + box0, pg = pages.page[0];
      // a missing page: a box outside the matrix is all zeros
      const int row = missing(pg)
                          ? -A.box_rows
                          : pg * A.page_rows + kv * A.S + (p - page_column(A, p) * A.S);
      box_load(dst + part * (TN * 128) + box0 * 128, &map, h * dim + part * 64, row, bar, policy);
    }
    return;
  }
  TilePages<TN, SHARES> rows = pages;   // a missing page: -1
#pragma unroll
  for (int i = 0; i < TN / 32 / SHARES; ++i) {
    const int p = p0 + share * (TN / SHARES) + (threadIdx.x & 31) + 32 * i;
    if (p < cached && missing(rows.page[i])) rows.page[i] = -1;
  }
  load_rows<D, PART, TN, SHARES>(A, rows, b, n, cached, hi, p0, h, kv, dst, share);
  if (lane == 0) *copied = 1;
  cp_async_arrive(bar);
}

// Rows of a page that lie in one tile of `tile` positions, 0 unless they are
// whole groups of 8 of the swizzled layout and the loading lanes can take a box
// each.
inline int box_rows(int page_size, int tile, int head_dim, int lanes) {
  int rows = page_size, rest = tile;
  while (rest) {
    const int r = rows % rest;
    rows = rest;
    rest = r;
  }
  return rows % 8 == 0 && tile / rows * (head_dim / 64) <= lanes ? rows : 0;
}

// The cache from the layer's first entry on as a matrix of entries of E
// elements, moved in boxes of 128 bytes by box_rows entries.
inline bool rows_map(CUtensorMap* map, const AttnArgs& A, bool bf16) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  const uint64_t elems = uint64_t(A.entry_bytes) / 2;
  const cuuint64_t dims[2] = {elems, cuuint64_t(A.num_pages > 0 ? A.num_pages : 1) *
                                         cuuint64_t(A.page_rows) - cuuint64_t(A.layer_row)};
  const cuuint64_t strides[1] = {cuuint64_t(A.entry_bytes)};
  const cuuint32_t box[2] = {64, cuuint32_t(A.box_rows > 0 ? A.box_rows : 8)}, step[2] = {1, 1};
  // an empty pool has no page that a row could come from: any address will do
  const void* base = A.num_pages > 0 ? static_cast<const void*>(A.cache) : A.spec;
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A thread's signs of the infinite (NaN: both) values in a tile of V, of its positions
// first .. last - 1 those from lo to hi - 1 and those of path's bits from node0 on: bits
// of columns of the head, +inf then -inf.  This and add_signs are not inlined: what is
// rare stands apart from what every tile runs, whose instructions then come from the
// caches (230 KB of them with everything in one piece).
template <class T, int D, int TN>
__device__ __noinline__ void collect_signs(const uint32_t* v, int first, int last, int lo, int hi,
                                           uint64_t path, int node0, uint32_t* signs) {
  for (int i = 0; i < 2 * D / 32; ++i) signs[i] = 0;
  for (int c = first; c < last; ++c) {
    const bool node = c >= node0 && c - node0 < 64 && ((path >> (c - node0)) & 1);
    if (!node && (c < lo || c >= hi)) continue;
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

}  // namespace sv
