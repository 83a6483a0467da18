// Accumulated attention weights on the fifth-generation tensor cores, for bf16
// and fp16 and heads of 64 to 256, multiples of 16.
//
//   score[b][p] += sum over heads h and counted rows r of exp(s - lse[r])
//
// Here the keys are the M of the product, S^T = K Q^T (128 positions x up to 64
// rows x D): a thread then owns a position and sums the weights of a head's
// rows in its own registers, with no exchange between threads and one order of
// the sum.  K is read once (the floor: 2 D bytes a position and head); the rows'
// Q and lse come from L2, once per 128 positions.
//
// One CTA per SM over an even piece of all requests' tiles of 128 positions;
// per tile a step for every head and 64 rows of it:
//   warps 4, 5 load K of a head and tile into a ring, half a tile each (as attention
//              loads it);
//   warps 7-9  load the steps' Q, the N of the product, in turn, with each row's
//              lse and the position of its token; the first also finds the parts
//              of the piece and announces them.
//   warp 6     issues the products into four accumulators in TMEM;
//   warps 0-3  one position a thread: exp(s - lse) summed over the rows.
// Every wait is bounded, as in attention; scores that an expired one left out
// stay as they are.
//
// Measured, bf16, 8 KV heads of 128 with 4 query heads each, pages of 16: 32
// requests of 2001 to 8190 positions with up to 15 drafts 58 us (5.2 TB/s; one row
// warp with an address per copy 299, three with branches in their loops 70); 24
// of 500 to 9001, one token, 34 us (4.5 TB/s, of which about 8 us until the first
// product).
#include "sv_attn_tc.cuh"

namespace sv {
namespace {

constexpr int kWtThreads = 320;
constexpr int kWtTile = 128;      // positions
constexpr int kWtRows = 64;       // rows per step
constexpr int kAccs = 4;
constexpr int kKeyWarp = 4, kProductWarp = 6, kRowWarp = 7;  // two key, three row warps
constexpr int kParts = 4;         // parts announced ahead

template <int D>
struct WtShape {
  static constexpr int kSlotBytes = kWtTile * D * 2;
  static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 5 : 2;
  static constexpr int kQBytes = kWtRows * D * 2;
  static constexpr int kQBufs = D == 256 ? 2 : 3;
  static constexpr size_t kSmem = 1024 + size_t(kSlots) * kSlotBytes + size_t(kQBufs) * kQBytes;
};
constexpr uint32_t kWtTmem = kAccs * kWtRows;

struct Part {                     // consecutive tiles of one request; count 0: the end
  int b, t_off, tile, count;
  AttnReq R;
};

struct WtShared {
  Part part[kParts];
  uint64_t announced[kParts], taken[kParts];
  uint64_t full[8], empty[8], qfull[3], qempty[3], lfull[6], lempty[6], sfull[kAccs],
      sempty[kAccs], drain, never;   // never: nothing arrives, the test of an expired wait
  struct {
    uint32_t at, phase;
    int filled;
  } loaded[2];                    // the ring of K as each of its warps left it
  uint32_t tmem;
  int abort, first_bad;
  int copied[8];
  // of the rows of a step: lse in the log2 domain, +inf for a row that does not
  // count, and their tokens' positions.  Two for each Q buffer: the sums are
  // still at them when the product is done with Q
  alignas(16) float lse[6][kWtRows];
  alignas(16) int at[6][kWtRows];
};

// Steps per head of a part; none for a tile in front of every row's window.
__device__ __forceinline__ int row_steps(const AttnArgs& A, const AttnReq& R, int p0) {
  if (A.window > 0 && p0 + kWtTile <= R.at0 - A.window + 1) return 0;
  return (R.take * A.G + kWtRows - 1) / kWtRows;
}

__device__ __forceinline__ bool next_part(WtShared& S, int i, Part& p) {
  if (!tc_wait_warp(&S.announced[i % kParts], (i / kParts) & 1, S)) return false;
  p = S.part[i % kParts];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&S.taken[i % kParts]));
  return p.count > 0;
}

// All threads, after a wait of the CTA expired and every warp has left its loop:
// copies and products that were issued finish, whichever warp gave up and when.
// Of a slot that only one of its two warps filled the wait runs out.
template <int D>
__device__ __noinline__ void give_up(WtShared& S) {
  const int warp = threadIdx.x >> 5;
  if (warp == kKeyWarp || warp == kKeyWarp + 1) {
    const int share = warp - kKeyWarp;
    Ring at(0, WtShape<D>::kSlots, S.loaded[share].phase);
    at.at = S.loaded[share].at;
    ring_land(at, S.loaded[share].filled, S.full);
  } else if (warp == kProductWarp) {
    mma_commit((threadIdx.x & 31) == 0, &S.drain);
    mbar_wait_for(smem_addr(&S.drain), 0);
    __syncwarp();
  }
  __syncthreads();
}

template <class T, int D, bool PART>
__global__ void __launch_bounds__(kWtThreads, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap keys_map, const AttnArgs A) {
  using C = WtShape<D>;
  extern __shared__ unsigned char wt_smem_raw[];
  __shared__ WtShared S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_addr(wt_smem_raw) + 1023u) & ~1023u;
  unsigned char* smem_p = wt_smem_raw + (smem0 - smem_addr(wt_smem_raw));
  constexpr uint32_t kQ0 = uint32_t(C::kSlots) * C::kSlotBytes;  // the Q buffers behind the ring

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_addr(&S.full[i]), 64);
      mbar_init(smem_addr(&S.empty[i]), 1);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(smem_addr(&S.qfull[i]), 1);
      mbar_init(smem_addr(&S.qempty[i]), 1);
    }
    for (int i = 0; i < 2 * C::kQBufs; ++i) {
      mbar_init(smem_addr(&S.lfull[i]), 1);
      mbar_init(smem_addr(&S.lempty[i]), 4);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(smem_addr(&S.sfull[i]), 1);
      mbar_init(smem_addr(&S.sempty[i]), 4);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(smem_addr(&S.announced[i]), 1);
      mbar_init(smem_addr(&S.taken[i]), 6 + C::kQBufs);  // all warps but the first row warp
    }
    mbar_init(smem_addr(&S.drain), 1);
    mbar_init(smem_addr(&S.never), 1);
    fence_mbar_init();
    S.abort = 0;
    S.first_bad = INT32_MAX;
  }
  if (warp == kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&S.tmem)),
                 "r"(kWtTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  const AttnPlan P = attn_plan<kWtTile, kWtTile, true, kWtThreads>(A);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const bool go = P.code == 0 && P.start < P.end;

  if (go && warp >= kKeyWarp && warp < kProductWarp) {
    // ------------------------------------------------------------------ keys
    const int share = warp - kKeyWarp;
    const uint64_t policy = l2_evict_first_policy();
    Part w;
    Ring at(0, C::kSlots, 1);
    bool stop = false;
    int filled = 0;
    for (int i = 0; !stop && next_part(S, i, w); ++i) {
      const int cached = min(w.R.n, w.R.hi);
      const int32_t* table = A.table + int64_t(w.b) * A.max_pages;
      // a missing page is noted where its scores would be written
      auto missing = [&](int page) { return page < 0 || page >= A.num_pages; };
      TilePages<kWtTile, 2> next =
          tile_pages<D, PART, kWtTile, 2>(A, table, cached, w.tile * kWtTile, share);
      for (int t = 0; t < w.count && !stop; ++t) {
        const int p0 = (w.tile + t) * kWtTile;
        const TilePages<kWtTile, 2> pages = next;
        if (t + 1 < w.count) next = tile_pages<D, PART, kWtTile, 2>(A, table, cached, p0 + kWtTile, share);
        if (row_steps(A, w.R, p0) == 0) continue;
        for (int h = 0; h < A.Hkv; ++h) {
          if (!tc_wait_warp(&S.empty[at.at], at.phase, S)) {
            stop = true;
            break;
          }
          load_tile<D, PART, kWtTile, 2>(A, keys_map, pages, w.b, w.R.n, cached, w.R.hi, p0, h, 0,
                                   smem0 + at.at * C::kSlotBytes, &S.full[at.at],
                                   &S.copied[at.at], policy, share, missing);
          at.step();
          ++filled;
        }
      }
    }
    if (lane == 0) {
      S.loaded[share].at = at.at;
      S.loaded[share].phase = at.phase;
      S.loaded[share].filled = filled;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (go && warp >= kRowWarp && warp < kRowWarp + C::kQBufs) {
    // --------------------------------------------------- parts, and their rows
    constexpr int kChunks = D / 8, kStep = 32 / kChunks;
    const int mine = warp - kRowWarp;   // this warp's buffer: every kQBufs-th step
    const int ch = lane % kChunks;
    const T* q = static_cast<const T*>(A.q);
    unsigned char* buf = smem_p + kQ0 + mine * C::kQBytes;
    const uint32_t buf_at = smem0 + kQ0 + mine * C::kQBytes;
    int64_t pos = P.start, base = P.base;
    int b = P.b, t_off = P.t_off;
    AttnReq R = attn_request<kWtTile, kWtTile, true>(A, b);
    uint32_t phase = 1, lphase = 1;
    int turn = 0;
    int step = 0;                       // of the piece, modulo kQBufs
    bool stop = false;
    for (int i = 0; !stop; ++i) {
      Part w;
      w.count = 0;
      if (mine > 0) {
        if (!next_part(S, i, w)) break;
      } else {
        if (pos < P.end) {
          while (pos >= base + R.ntiles) {
            base += R.ntiles;
            t_off += R.k + 1;
            R = attn_request<kWtTile, kWtTile, true>(A, ++b);
          }
          w.b = b;
          w.t_off = t_off;
          w.tile = R.tile0 + int(pos - base);
          const int64_t left = P.end - pos, rest = base + R.ntiles - pos;
          w.count = int(left < rest ? left : rest);
          w.R = R;
          pos += w.count;
        }
        if (!tc_wait_warp(&S.taken[i % kParts], ((i / kParts) & 1) ^ 1, S)) break;
        if (lane == 0) {
          S.part[i % kParts] = w;
          mbar_arrive(smem_addr(&S.announced[i % kParts]));
        }
        if (w.count == 0) break;
      }
      const int nrows = w.R.take * A.G;
      for (int t = 0; t < w.count && !stop; ++t) {
        const int steps = row_steps(A, w.R, (w.tile + t) * kWtTile);
        for (int h = 0; h < A.Hkv && !stop; ++h)
          for (int c = 0; c < steps; ++c) {
            const bool other = step != mine;
            step = step + 1 == C::kQBufs ? 0 : step + 1;
            if (other) continue;
            const int lb = mine + turn * C::kQBufs;   // this step's lse buffer
            if (!tc_wait_warp(&S.lempty[lb], lphase, S)) {
              stop = true;
              break;
            }
            turn ^= 1;
            lphase ^= turn ^ 1;
            const int row0 = c * kWtRows, rows = min(kWtRows, nrows - row0);
            const int padded = (rows + 15) & ~15;
            // Rows lane and lane + 32: their addresses, lse and tokens' positions.  The
            // product's N is a multiple of 16: the last row again fills it up, under an
            // lse that leaves it no weight.  Its products are numbers wherever the
            // row's own are; those of a zero query and an infinite key are not.
            // (Leaving such rows out of the sums instead: 58 -> 64 us with 15 drafts.)
            uint64_t own[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int r = lane + 32 * x, row = row0 + min(r, rows - 1);
              const int tok = row / A.G, hq = h * A.G + row % A.G;
              own[x] = reinterpret_cast<uint64_t>(q + int64_t(w.t_off + tok) * A.q_ts +
                                                  int64_t(hq) * A.q_hs);
              float v = INFINITY;
              if (r < rows) {
                v = A.lse[int64_t(w.t_off + tok) * A.Hq + hq] * kAttnLog2e;
                if (v == -INFINITY) v = INFINITY;   // a row that saw nothing weighs nothing
              }
              S.lse[lb][r] = v;
              S.at[lb][r] = w.R.at0 + tok;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&S.lfull[lb]));
            if (!tc_wait_warp(&S.qempty[mine], phase, S)) {
              stop = true;
              break;
            }
            phase ^= 1;
            // without branches, which take a lone warp as long as ten other instructions
            auto fill = [&](auto vec) {
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll 1
                for (int j0 = 0; j0 < min(32, padded - 32 * x); j0 += 8 * kStep)
#pragma unroll
                  for (int j = 0; j < 8 * kStep; j += kStep) {
                    const int from = j0 + j + lane / kChunks, r = 32 * x + from;
                    const uint64_t a =
                        (uint64_t(__shfl_sync(0xffffffffu, uint32_t(own[x] >> 32), from)) << 32) |
                        __shfl_sync(0xffffffffu, uint32_t(own[x]), from);
                    const T* src = reinterpret_cast<const T*>(a) +
                                   (PART && ch * 8 >= A.D ? 0 : ch * 8);
                    const uint32_t off =
                        (ch >> 3) * (kWtRows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                    if (decltype(vec)::value) {
                      cp_async16(buf_at + off, src, 16u);
                    } else {
                      T* dst = reinterpret_cast<T*>(buf + off);
                      for (int e = 0; e < 8; ++e) dst[e] = src[e];
                    }
                  }
            };
            if (A.q_vec) fill(std::true_type());
            else fill(std::false_type());
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&S.qfull[mine]));
          }
      }
    }
  } else if (go && warp == kProductWarp) {
    // -------------------------------------------------------------- products
    constexpr uint32_t kBase = (1u << 4) | (Bits<T>::kFmt << 7) | (Bits<T>::kFmt << 10) |
                               (uint32_t(kWtTile >> 4) << 24);
    const uint32_t lead = lane == 0;
    const uint64_t k_desc = sw128_desc(smem0), q_desc = sw128_desc(smem0 + kQ0);
    Part w;
    Ring at(0, C::kSlots, 0), qb(0, C::kQBufs, 0), acc(0, kAccs, 0);
    bool ok = true;
    for (int i = 0; ok && next_part(S, i, w); ++i) {
      const int nrows = w.R.take * A.G;
      for (int t = 0; ok && t < w.count; ++t) {
        const int steps = row_steps(A, w.R, (w.tile + t) * kWtTile);
        for (int h = 0; ok && steps > 0 && h < A.Hkv; ++h) {
          ok = tc_wait_warp(&S.full[at.at], at.phase, S);
          if (!ok) break;
          if (*reinterpret_cast<volatile int*>(&S.copied[at.at])) fence_async_proxy();
          const uint64_t k = k_desc + at.at * (C::kSlotBytes >> 4);
          for (int c = 0; c < steps; ++c) {
            // the rows there, and the accumulator read (the first round passes at once)
            ok = tc_wait_two(&S.qfull[qb.at], qb.phase, &S.sempty[acc.at], acc.phase ^ 1, S);
            if (!ok) break;
            tc_fence_after();
            const uint32_t n = (min(kWtRows, nrows - c * kWtRows) + 15) & ~15;
            const uint32_t idesc = kBase | (n >> 3 << 17);
            const uint64_t q = q_desc + qb.at * (C::kQBytes >> 4);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              if (PART && x * 16 >= A.D) break;
              mma_ss(lead, tmem + acc.at * kWtRows,
                     k + (((x >> 2) * (kWtTile * 128) + (x & 3) * 32) >> 4),
                     q + (((x >> 2) * (kWtRows * 128) + (x & 3) * 32) >> 4), idesc, x != 0);
            }
            mma_commit(lead, &S.sfull[acc.at]);
            mma_commit(lead, &S.qempty[qb.at]);
            qb.step();
            acc.step();
          }
          if (ok) mma_commit(lead, &S.empty[at.at]);
          at.step();
        }
      }
    }
  } else if (go && warp < kKeyWarp) {
    // ------------------------------------------------------------------ sums
    const uint32_t lanes = tmem + (uint32_t(warp * 32) << 16);
    Part w;
    Ring acc(0, kAccs, 0), lb(0, 2 * C::kQBufs, 0);
    bool ok = true;
    for (int i = 0; ok && next_part(S, i, w); ++i) {
      if (i == 0 && A.test_expire == int(blockIdx.x) + 1 &&
          !mbar_wait_for(smem_addr(&S.never), 0, kTestWaitNs)) {
        *reinterpret_cast<volatile int*>(&S.abort) = 1;
        break;
      }
      const int nrows = w.R.take * A.G;
      for (int t = 0; ok && t < w.count; ++t) {
        const int p0 = (w.tile + t) * kWtTile, p = p0 + tid;
        const int steps = row_steps(A, w.R, p0);
        // whether some row does not see some position of the tile
        const bool edge = p0 + kWtTile - 1 > w.R.at0 || p0 + kWtTile > w.R.hi ||
                          (A.window > 0 && p0 <= w.R.at0 + w.R.take - 1 - A.window);
        float sum = 0.f;
        for (int h = 0; ok && h < A.Hkv; ++h)
          for (int c = 0; c < steps; ++c) {
            ok = tc_wait_two(&S.sfull[acc.at], acc.phase, &S.lfull[lb.at], lb.phase, S);
            if (!ok) break;
            tc_fence_after();
            const int n = (min(kWtRows, nrows - c * kWtRows) + 15) & ~15;
            const uint32_t col = lanes + acc.at * kWtRows;
            for (int x0 = 0; x0 < n; x0 += 16) {
              uint32_t s[16];
              float z[16];
              tmem_ld16(col + x0, s);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<float4*>(&z[4 * x]) =
                    *reinterpret_cast<const float4*>(&S.lse[lb.at][x0 + 4 * x]);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) z[x] = fmaf(__uint_as_float(s[x]), A.scale2, -z[x]);
              if (edge) {
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const int at = S.at[lb.at][x0 + x];
                  if (p <= at && (A.window <= 0 || p > at - A.window)) sum += ex2_approx(z[x]);
                }
              } else {
                float part = 0.f;   // 16 rows on their own: short chains of additions
#pragma unroll
                for (int x = 0; x < 16; x += 2) part += ex2_approx(z[x]) + ex2_approx(z[x + 1]);
                sum += part;
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(smem_addr(&S.sempty[acc.at]));
              mbar_arrive(smem_addr(&S.lempty[lb.at]));
            }
            lb.step();
            acc.step();
          }
        if (ok && p < w.R.hi) {
          int64_t voff;
          if (attn_key(A, w.b, w.R.n, p, &voff))
            A.out_score[int64_t(w.b) * A.out_stride + p] =
                A.score[int64_t(w.b) * A.score_stride + p] + sum;
          else
            atomicMin(&S.first_bad, w.b);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (S.abort) give_up<D>(S);
  if (tid == 0) A.status[A.B + blockIdx.x] = S.abort ? -SV_ERR_TIMEOUT : S.first_bad;
  if (warp == kProductWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kWtTmem));
  }
}

template <class T, int D, bool PART>
cudaError_t run(const AttnArgs& A, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  if (cudaError_t e = allow_smem(weights_tc_kernel<T, D, PART>, WtShape<D>::kSmem, configured)) return e;
  CUtensorMap map;
  AttnArgs B = A;
  B.box_rows = box_rows(A.S, kWtTile, D, 64);
  if (!rows_map(&map, B, Bits<T>::kFmt != 0)) return cudaErrorInvalidValue;
  weights_tc_kernel<T, D, PART><<<A.ctas, kWtThreads, WtShape<D>::kSmem, s>>>(map, B);
  return cudaGetLastError();
}

template <class T>
cudaError_t run_dim(const AttnArgs& A, cudaStream_t s) {
  if (A.D == 64) return run<T, 64, false>(A, s);
  if (A.D <= 128) return A.D == 128 ? run<T, 128, false>(A, s) : run<T, 128, true>(A, s);
  return A.D == 256 ? run<T, 256, false>(A, s) : run<T, 256, true>(A, s);
}

}  // namespace

cudaError_t launch_attn_weights_tc(const AttnArgs& A, int dtype, cudaStream_t s) {
  return dtype == SV_BF16 ? run_dim<__nv_bfloat16>(A, s) : run_dim<__half>(A, s);
}

}  // namespace sv
