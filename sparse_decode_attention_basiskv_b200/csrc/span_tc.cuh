// Attention of many query rows over a sliding window with sinks on the
// 5th-generation tensor cores: prompt chunks, and drafts of more rows than
// the streaming kernel takes (instances: span_tc_bf16.cu, span_tc_e4m3.cu,
// span_tc_q4.cu).
//
//   a[row] = sum_t p_t z_t,  p = softmax over the row's tokens of
//   (q . K_t) / sqrt(d)
//
// A work item is (sequence, KV head, two tiles of 128 rows).  A row is a query
// token and a head of the group (token-major), so the group's heads share each
// Key and latent that is loaded, and a tile spans only 128 / G tokens of the
// band.  KV comes in tiles of 128 tokens and is multiplied in steps of 64: per
// step and row tile S = Q K^T (tcgen05), P = exp2(S - m) (registers), O += P Z,
// Q and P as A operands in tensor memory.  Two row tiles and 128 tokens take
// 2 * 128 * 128 * (d + r_v) multiply-adds and 2 * 128 * 128 exponentials: at d
// 128, r_v 64 the tensor cores need 1600 clocks (a 128 x 64 x 16 product takes
// 33; 49 with both operands in shared memory, whose bandwidth then bounds it)
// and the 16 exponentials a clock 2050.
//
// Roles (16 warps, one CTA an SM): warps 0 and 1 issue the MMAs of one row tile
// each; warps 4-7 and 8-11 hold the softmax of one row tile each, a thread a
// row (no shuffles): the step's 64 scores in registers, their maximum, the
// weights.  The weights are taken against a reference that only moves where a
// row's maximum has passed it by a wide margin; then the warp rescales O.
// Warps 12-15 bring in the KV tiles page by page into the swizzled layout (bf16
// by cp.async; E4M3 and 4-bit rows widened to f16 on the way, exactly), a tile
// ahead of what they hand over.
//
// Precision: scores, maxima and sums in fp32.  Over E4M3 and 4-bit caches the weights
// are rounded to f16 for P Z (2^-11 of a weight).  Over bf16 ones a weight is its bf16
// rounding and a rounding of the rest (16 bits, a second product), so that a prompt is
// as accurate as a token.  With weights of 8 bits the chunk below takes 270 us instead
// of 300 (the same inputs again and again), and its error against 64 bits is 2.2e-3
// instead of 1.7e-3, the output's own rounding.
//
// Tensor memory: per row tile two slots of 64 columns for S, P over its S (bf16:
// 32 tokens' weights, their remainders, the other 32 tokens'), r_v for O, and Q in
// what is left (all of it for r_v up to 64, d 128, half at 96, none at 128; the other
// k-steps read Q from shared memory).  Q K^T of step i + 2 follows P Z of step i on
// the tensor cores into the same slot, while the softmax has step i + 1 before it,
// so its latency is hidden.  A product's end needs no barrier of its own: S of step
// i + 2 is behind P Z of step i, so its barrier tells both (a wait costs some 270
// clocks even when the phase is over; one a step less was worth 8%).
//
// Measured (4096-token chunk, Llama-8B layer, window 4096, inputs past L2): bf16 326
// us, 633 TFLOP/s; the same inputs again and again 300, r_v 128 405, E4M3 285, r_v 128
// 416, 4 bits 286, r_v 128 321.  Three ragged sequences of 1023 tokens, Qwen3-32B
// layer, window 2000, 4 bits: 275 us, 641 TFLOP/s.  Bound by the softmax's chain of a
// step: load, maximum, weights, store, two barriers, some 1950 clocks (bf16) where its
// exponentials take 1020: with weights of 8 bits (1750 clocks, 282 us) the chunk took
// 255 without the exponentials, 273 with a quarter of the products and 262 without
// the copies.  An item's start (queries to tensor memory, the first tile) costs some
// 10,000 clocks.  One slot of 128 columns a row tile, the softmax waiting for each
// product, was 7% slower.
//
// Tokens whose block-table entry is out of range have no part in the softmax: the
// issuing warp, which looks the run's entries up at the start, sets their scores to
// -infinity in tensor memory behind Q K^T.  A run with such an entry takes a loop
// of its own.  (Tests in the softmax, whose registers are full, took 7 to 11% of
// every call, one in the issuing warps' common loop up to 7%; this way the calls
// without such entries take -2 to +3%.)
//
// The items that would not fill a last round of the SMs (all of them, where
// there are fewer items than SMs) have their KV tiles cut into runs, a block
// each, whose partial sums span_tc_merge_kernel joins.
#pragma once

#include <type_traits>

#include "cache4.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tcgen05.cuh"

namespace basiskv {
namespace {

constexpr int kTcThreads = 512;
constexpr int kTcRows = 256;  // two row tiles
// How far (log2) scores may pass the reference before it moves: the weights then
// reach 2^15 in f16, 2^32 in bf16, at the same relative precision, and their products
// and sums stay inside fp32's range: over bf16 caches for latents up to 2^64 and 2^30
// tokens.  (2^64, at the same times, overflowed from latents of 2^60 on.)
template <int FMT>
constexpr float tc_slack() {
  return FMT == kSpanBf16 ? 32.f : 15.f;
}

template <int D, int RV>
struct TcGeom {
  static constexpr int kQBytes = kTcRows * D * 2;
  static constexpr int kKBytes = 128 * D * 2;
  static constexpr int kZBlocks = (RV + 63) / 64;  // 64-column blocks
  static constexpr int kZBytes = kZBlocks * 128 * 128;
  static constexpr int kStages = RV <= 64 ? 3 : 2;
  // k-steps of Q whose A operand lies in tensor memory (32 columns hold 4)
  static constexpr int kRoom = (128 - RV) / 32 * 4;
  static constexpr int kQSteps = kRoom < D / 16 ? kRoom : D / 16;
  // its columns: S of row tile t at 128 t, then O, then Q
  static constexpr int kO = 256, kQ = kO + 2 * RV;
  static_assert(kQ + 16 * kQSteps <= 512, "");
  // (d 128, r_v 128: 12 KB more left the rows that the loaders widen half the L1, and
  // took an E4M3 chunk from 417 to 484 us)
  static constexpr size_t kSmem = 1024 + kQBytes + kStages * (size_t)(kKBytes + kZBytes);
};

// One item's place and its KV tiles (128 tokens each): the sinks', then the
// window's.
struct TcItem {
  int b, g, j0;         // first query token of the item
  int pos0;             // its position
  int live_end;         // no row sees a token from here on
  int lo_first;         // first window token of the first row
  int n_sink, tile0, n; // KV tiles
};
__device__ __forceinline__ TcItem tc_place(const SpanArgs& a, int item) {
  TcItem x;
  const int tq2 = kTcRows >> a.logG, njt = (a.n_tot + tq2 - 1) >> (8 - a.logG);
  const int groups = a.B * a.Hkv, jt = item / groups, bg = item - jt * groups;
  // the last tiles of a chunk see the most tokens: they go first
  x.j0 = (njt - 1 - jt) * tq2;
  x.b = bg / a.Hkv;
  x.g = bg - x.b * a.Hkv;
  return x;
}
__device__ __forceinline__ void tc_span(const SpanArgs& a, TcItem& x) {
  int T = __ldg(a.seq_lens + x.b);
  if (T < 0 || T > a.max_seq_len) {
    if (threadIdx.x == 0) raise_status(a.status, BASISKV_DEV_BAD_LENGTH);
    T = 0;
  }
  x.pos0 = T - a.n_tot + x.j0;
  const int last = min(x.pos0 + (kTcRows >> a.logG), T) - 1;
  x.live_end = T > 0 ? last + 1 : 0;
  x.lo_first = a.window > 0 ? max(0, max(x.pos0, 0) - a.window + 1) : 0;
  if (x.live_end <= 0) {
    x.n_sink = x.tile0 = x.n = 0;
  } else {
    x.tile0 = x.lo_first >> 7;
    x.n_sink = min((a.sink + 127) >> 7, x.tile0);
    x.n = x.n_sink + (last >> 7) - x.tile0 + 1;
  }
}
__device__ __forceinline__ int tc_tile(const TcItem& x, int i) {
  return i < x.n_sink ? i : x.tile0 + i - x.n_sink;
}

// Byte offset of 16-byte chunk c of row r in a tile of 128-byte swizzled rows
// (64 16-bit columns each; the 64-column blocks lie 16 KB apart).
__device__ __forceinline__ uint32_t tc_off(int r, int c) {
  return (uint32_t)((c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z,
                                       uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}

// Two fp32 lanes an instruction: a * b + c and a + b on register pairs.
__device__ __forceinline__ uint64_t pack2(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two bf16 roundings in a word, and what a pair of values has beyond the bf16 values
// of a word (exact for its own roundings).
__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void less_bf16_pair(float x, float y, uint32_t w, float& rx, float& ry) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2;"
      " fma.rn.f32.bf16 %0, l, %5, %3; fma.rn.f32.bf16 %1, h, %5, %4; }"
      : "=f"(rx), "=f"(ry)
      : "r"(w), "f"(x), "f"(y), "h"((uint16_t)0xbf80));  // -1
}

// One arrival for the whole warp, after all its lanes' work before it.
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

template <int FMT, int D, int RV>
__global__ void __launch_bounds__(kTcThreads, 1) span_tc_kernel(SpanArgs a, TcPlan plan) {
  using Gm = TcGeom<D, RV>;
  constexpr int NST = Gm::kStages;
  constexpr bool BF = FMT == kSpanBf16;
  extern __shared__ uint8_t tc_smem_raw[];
  uint8_t* smem = align_smem_1k(tc_smem_raw);
  __shared__ uint64_t bars[4 * NST + 11];
  __shared__ __align__(128) uint32_t no_score[128];  // -infinity, 32 rows of 4 columns
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float row_scale[kTcRows];
  uint64_t *kfull = bars, *kempty = bars + NST, *zfull = bars + 2 * NST, *zempty = bars + 3 * NST;
  // [row tile][slot]: S of step u is there and O has step u - 2 (two phases more
  // than there are steps); P is there
  uint64_t *sfull = bars + 4 * NST, *pfull = sfull + 4, *qfull = sfull + 8;
  uint64_t* scored = qfull + 1;  // [row tile]: Q K^T of a step with missing tokens is done
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
  const uint32_t sq = smem_u32(smem), sk = sq + Gm::kQBytes, sz = sk + NST * Gm::kKBytes;

  // the first plan.full blocks take whole items, the others one of plan.ns runs
  const bool whole = (int)blockIdx.x < plan.full;
  const int part = (int)blockIdx.x - plan.full;
  TcItem it = tc_place(a, whole ? (int)blockIdx.x : plan.full + part / plan.ns);
  const int split = whole ? 0 : part % plan.ns, nsplit = whole ? 1 : plan.ns;
  const int rows = min(kTcRows, (a.n_tot - it.j0) << a.logG);  // live rows of the item
  const int nt = rows > 128 ? 2 : 1;                           // row tiles
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&kfull[s], 4);  // one arrival a warp
      mbar_init(&zfull[s], 4);
      mbar_init(&kempty[s], nt);  // one commit a row tile
      mbar_init(&zempty[s], nt);
    }
    for (int t = 0; t < 4; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pfull[t], 4);
    }
    mbar_init(qfull, 8);
    mbar_init(&scored[0], 1);
    mbar_init(&scored[1], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 2) {
    sts128(smem_u32(no_score + 4 * lane), 0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
    fence_proxy_async();
  }
  pdl_wait();
  pdl_launch_dependents();

  // the first batch of the item's queries, under the length's round trip
  constexpr int QC = D / 8, QN = kTcRows * QC / 256, QB = QN < 8 ? QN : 8;
  const uint16_t* q0 = a.q + ((size_t)it.b * a.n_tot + it.j0) * a.Hq * D + it.g * a.G * D;
  auto load_q = [&](uint4 (&qv)[QB], int x0) {
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      const int y = (x0 + x) * 256 + tid - 128, r = y / QC;
      qv[x] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)  // a token's heads of the group lie one behind the other
        qv[x] = __ldg(reinterpret_cast<const uint4*>(
            q0 + (size_t)(r >> a.logG) * a.Hq * D + (r & (a.G - 1)) * D + 8 * (y % QC)));
    }
  };
  uint4 qv[QB];
  if (warp >= 4 && warp < 12) load_q(qv, 0);
  tc_span(a, it);
  const int i0 = (int)((long long)it.n * split / nsplit);
  const int n = (int)((long long)it.n * (split + 1) / nsplit) - i0;
  const int tq = 128 >> a.logG;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  volatile int* abrt = &abort_flag;
  // The block-table entry of logical page p, or -1 where it is out of range.
  auto entry = [&](int p) {
    const int pp = p < a.max_pages ? __ldg(a.block_table + (size_t)it.b * a.max_pages + p) : -1;
    return pp < a.num_phys ? pp : -1;
  };
  // steps of 64 tokens; the last tile's second half may be past every row
  const int n2 = n == 0 ? 0
                        : 2 * n - (i0 + n == it.n && ((it.live_end - 1) & 127) < 64 ? 1 : 0);

  if (warp < 2) {
    // --------------------------------------- MMA issue, one warp a row tile
    const int t = warp;
    if (n > 0 && t < nt) {
      constexpr uint32_t id_qk = tc_idesc(128, 64, BF, false);
      constexpr uint32_t id_pv = tc_idesc(128, RV, BF, true);
      const uint64_t dq = tc_sdesc(sq + t * (Gm::kQBytes / 2)), dk = tc_sdesc(sk),
                     dz = tc_sdesc(sz, 16384);
      const uint32_t tm_s = tmem + 128 * t, tm_o = tmem + Gm::kO + RV * t;
      const uint32_t tm_q = tmem + Gm::kQ + 8 * Gm::kQSteps * t;
      const bool lead = elect_one();
      auto wait = [&](uint64_t* bar, int parity) {
        return mbar_poll(bar, parity, a.status, abrt);
      };
      // is the page of a token among t .. t + count - 1 (of one page) needed and not there?
      auto missing = [&](int t, int count) {
        return t < it.live_end && (t + count > it.lo_first || t < a.sink) &&
               entry(t >> a.logS) < 0;
      };
      bool gap = false;  // (looked up while the first tile is on its way)
      const int lp = 7 - a.logS;  // log2 of a tile's pages
      for (int x = lane; x < n << lp; x += 32) {
        const int page = x & ((1 << lp) - 1);
        gap |= missing(tc_tile(it, i0 + (x >> lp)) * 128 + (page << a.logS), a.S);
      }
      gap = __any_sync(0xffffffffu, gap);
      int scored_ph = 0;
      auto issue = [&](auto gaps) {
        constexpr bool GAPS = decltype(gaps)::value;
        // step u of KV tile u / 2 in ring stage st: rows 64 (u % 2) .. of the tile
        auto qk = [&](int u, int st) -> bool {
          bool ok = true;
          tc_fence_after_sync();
          if (lead) {
            const uint64_t k0 = dk + st * (Gm::kKBytes >> 4) + (u & 1) * (64 * 128 >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t kk = k0 + (k >> 2) * 1024 + (k & 3) * 2;
              if (k < Gm::kQSteps)
                tc_mma_ts(tm_s + 64 * (u & 1), tm_q + 8 * k, kk, id_qk, k > 0);
              else
                tc_mma_ss(tm_s + 64 * (u & 1), dq + (k >> 2) * 1024 + (k & 3) * 2, kk, id_qk,
                          k > 0);
            }
          }
          if constexpr (GAPS) {
            // 8 tokens a lane: they lie in one page
            const int t8 = tc_tile(it, i0 + (u >> 1)) * 128 + 64 * (u & 1) + 8 * (lane & 7);
            const uint32_t miss = __ballot_sync(0xffffffffu, lane < 8 && missing(t8, 8));
            if (miss) {
              if (lead) tc_commit_to(&scored[t]);
              ok = wait(&scored[t], scored_ph);
              scored_ph ^= 1;
              tc_fence_after_sync();
              if (lead && ok) {
                for (int c = 0; c < 16; ++c)
                  if (miss >> (c >> 1) & 1)
                    tc_cp_32x4(tm_s + 64 * (u & 1) + 4 * c, tc_sdesc_plain(smem_u32(no_score)));
              }
            }
          }
          if (lead) {
            tc_commit_to(&sfull[2 * t + (u & 1)]);
            if (u & 1) tc_commit_to(&kempty[st]);
          }
          __syncwarp();
          return ok;
        };
        int kst = 0, kph = 0, zst = 0, zph = 0;  // stages of the next Key and latent tiles
        auto next = [](int& st, int& ph) {
          if (++st == NST) {
            st = 0;
            ph ^= 1;
          }
        };
        bool ok = wait(qfull, 0) && wait(&kfull[0], 0);
        if (ok) {
          ok = qk(0, 0) && (n2 == 1 || qk(1, 0));
          next(kst, kph);
        }
        for (int u = 0; ok && u < n2; ++u) {
          if (!(u & 1)) ok = wait(&zfull[zst], zph);
          ok = ok && wait(&pfull[2 * t + (u & 1)], (u >> 1) & 1);
          if (!ok) break;
          tc_fence_after_sync();
          if (lead) {
            const uint64_t z = dz + zst * (Gm::kZBytes >> 4) + (u & 1) * (64 * 128 >> 4);
#pragma unroll
            for (int k = 0; k < (BF ? 8 : 4); ++k) {
              const int zk = BF ? (k & 1) + 2 * (k >> 2) : k;  // (remainders: k 2, 3, 6, 7)
              tc_mma_ts(tm_o, tm_s + 64 * (u & 1) + 8 * k, z + zk * 128, id_pv, u > 0 || k > 0);
            }
            if (u + 2 >= n2) tc_commit_to(&sfull[2 * t + (u & 1)]);
            if (u & 1) tc_commit_to(&zempty[zst]);
          }
          __syncwarp();
          if (u & 1) next(zst, zph);
          if (u + 2 < n2) {
            if (!(u & 1)) ok = wait(&kfull[kst], kph);
            if (!ok) break;
            ok = qk(u + 2, kst);  // in the slot of step u
            if (u & 1) next(kst, kph);
          }
        }
        if (!ok) {  // a wait has run out: tensor memory goes once the products are done
          if (lead) tc_commit_to(&scored[t]);
          mbar_wait(&scored[t], scored_ph, a.status, kDrainNs);
        }
      };
      if (gap)
        issue(std::true_type{});
      else
        issue(std::false_type{});
    }
  } else if (warp >= 12) {
    // -------------------------------------------------------------- loaders
    const int lt = tid - 384;  // 0 .. 127
    // tokens some row of the item sees; the rest of a tile is zeroed
    auto seen = [&](int t) { return t < it.live_end && (t >= it.lo_first || t < a.sink); };
    // The tile row of token t, -1 when there is nothing to read.
    auto tile_row = [&](int t) -> int {
      if (!seen(t)) return -1;
      const int p = t >> a.logS;
      const int pp = p < a.max_pages ? __ldg(a.block_table + (size_t)it.b * a.max_pages + p) : -1;
      if (pp < 0 || pp >= a.num_phys) {
        raise_status(a.status, BASISKV_DEV_BAD_PAGE);
        return -1;
      }
      return ((pp * a.Hkv + it.g) << a.logS) + (t & (a.S - 1));
    };
    if constexpr (BF) {
      // Rows 32 w .. 32 w + 31 of a tile are warp w's: lane l looks row l's
      // place up, and the lanes then copy whole rows together.
      const int w = lt >> 5;
      constexpr int KC = D / 8, ZC = RV / 8;
      auto copy_k = [&](int i, int row) {
        const uint32_t dst = sk + (i % NST) * Gm::kKBytes + 32 * w * 128;
        const uint8_t* src = a.K + (lane % KC) * 16;
#pragma unroll 4
        for (int x = 0; x < KC; ++x) {
          const int r = (32 * x + lane) / KC, c = lane % KC;
          const int tr = __shfl_sync(0xffffffffu, row, r);
          cp_async16_or_zero(dst + tc_off(r, c), src + (tr < 0 ? 0 : (int64_t)tr * (D * 2)),
                             tr >= 0);
        }
      };
      auto copy_z = [&](int i, int row) {
        const uint32_t dst = sz + (i % NST) * Gm::kZBytes + 32 * w * 128;
        if (a.zsplit == RV) {
#pragma unroll 4
          for (int x = 0; x < ZC; ++x) {
            const int y = 32 * x + lane, r = y / ZC, c = y % ZC;
            const int tr = __shfl_sync(0xffffffffu, row, r);
            cp_async16_or_zero(dst + tc_off(r, c),
                               a.Z + c * 16 + (tr < 0 ? 0 : (int64_t)tr * (RV * 2)), tr >= 0);
          }
        } else {  // a narrow router's split tiles
#pragma unroll 1
          for (int x = 0; x < ZC; ++x) {
            const int y = 32 * x + lane, r = y / ZC, c = y % ZC;
            const int tr = __shfl_sync(0xffffffffu, row, r);
            size_t off = 0;
            if (tr >= 0)
              off = ((size_t)(tr >> a.logS) * a.S * RV +
                     split_off(tr & (a.S - 1), 8 * c, a.S, RV, a.zsplit)) * 2;
            cp_async16_or_zero(dst + tc_off(r, c), a.Z + off, tr >= 0);
          }
        }
      };
      // groups in flight: K_0, Z_0, K_1, Z_1, ...; a part is handed over when
      // the next tile's has been requested
      int row = n > 0 ? tile_row(tc_tile(it, i0) * 128 + lt) : -1;
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int next = i + 1 < n ? tile_row(tc_tile(it, i0 + i + 1) * 128 + lt) : -1;
        if (i >= NST) ok = mbar_poll(&kempty[i % NST], ((i / NST) & 1) ^ 1, a.status, abrt);
        if (!ok) break;
        copy_k(i, row);
        cp_async_commit();
        if (i > 1) {
          cp_async_wait_group<2>();
          fence_proxy_async();
          arrive_warp(&kfull[(i - 1) % NST]);
        }
        if (i >= NST) ok = mbar_poll(&zempty[i % NST], ((i / NST) & 1) ^ 1, a.status, abrt);
        if (!ok) break;
        copy_z(i, row);
        cp_async_commit();
        if (i == 0) {  // nothing is under way yet: the first Keys at once
          cp_async_wait_group<1>();
          fence_proxy_async();
          arrive_warp(&kfull[0]);
        }
        if (i > 0) {
          cp_async_wait_group<2>();
          fence_proxy_async();
          arrive_warp(&zfull[(i - 1) % NST]);
        }
        row = next;
      }
      cp_async_wait_all();
      fence_proxy_async();
      if (n > 0 && ok) {
        if (n > 1) arrive_warp(&kfull[(n - 1) % NST]);
        arrive_warp(&zfull[(n - 1) % NST]);
      }
    } else {
      // A thread widens one row of each tile; the next tile's bytes are
      // requested before the current ones are converted, and its place in the
      // cache was looked up a tile earlier.
      constexpr int KW = FMT == kSpanQ4 ? D / 8 : D / 4;    // 32-bit words of codes a row
      constexpr int ZW = FMT == kSpanQ4 ? RV / 8 : RV / 4;
      constexpr int KS = D / 64, ZS = (RV / 16 + 3) / 4;    // words of scales (4 bits only)
      auto load = [&](const uint8_t* base, int row, int wdt, uint32_t* dst, int nw, uint32_t* sc,
                      bool z) {
        if (row < 0) return;
        if constexpr (FMT == kSpanQ4) {
          const int tile = row >> a.logS, r = row & (a.S - 1);
          const uint8_t* tp = base + (size_t)tile * q4_tile_bytes(a.S, wdt);
          const uint8_t* cp = tp + r * (wdt / 2);
#pragma unroll
          for (int x = 0; x < nw; x += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(cp + 4 * x));
            dst[x] = v.x, dst[x + 1] = v.y, dst[x + 2] = v.z, dst[x + 3] = v.w;
          }
          const uint8_t* sp = tp + a.S * (wdt / 2) + r * (wdt / 16);
          // rows of 2 (w 32) to 8 scale bytes, 2-byte aligned
#pragma unroll
          for (int x = 0; x < wdt / 16; x += 2) {
            const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(sp + x));
            if (x % 4 == 0)
              sc[x / 4] = h;
            else
              sc[x / 4] |= h << 16;
          }
        } else {
          const size_t tile = row >> a.logS;
          const int r = row & (a.S - 1);
#pragma unroll
          for (int x = 0; x < nw; x += 4) {
            const size_t off = z ? tile * a.S * wdt + split_off(r, 4 * x, a.S, wdt, a.zsplit)
                                 : (size_t)row * wdt + 4 * x;
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(base + off));
            dst[x] = v.x, dst[x + 1] = v.y, dst[x + 2] = v.z, dst[x + 3] = v.w;
          }
        }
      };
      auto put = [&](uint32_t dst, bool there, const uint32_t* src, int wdt, const uint32_t* sc) {
#pragma unroll
        for (int c = 0; c < wdt / 8; ++c) {  // 8 columns, 16 bytes of f16
          uint32_t o[4] = {0u, 0u, 0u, 0u};
          if (there) {
            if constexpr (FMT == kSpanQ4) {
              const uint32_t s = q4_scale_x2(sc[c / 8] >> (8 * ((c / 2) & 3)) & 255u);
              q4_unpack8(src[c], o);
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] = hmul2(o[k], s);
            } else {
              e4m3x4_to_f16(src[2 * c], o[0], o[1]);
              e4m3x4_to_f16(src[2 * c + 1], o[2], o[3]);
            }
          }
          sts128(dst + tc_off(lt, c), o[0], o[1], o[2], o[3]);
        }
      };
      struct Raw {
        int row;
        uint32_t kw[KW], zw[ZW], ks[KS], zs[ZS];
      };
      auto place = [&](int i) { return i < n ? tile_row(tc_tile(it, i0 + i) * 128 + lt) : -1; };
      auto fetch = [&](Raw& x, int row) {
        x.row = row;
        load(a.K, row, D, x.kw, KW, x.ks, false);
        load(a.Z, row, RV, x.zw, ZW, x.zs, true);
      };
      bool ok = true;
      auto hand_over = [&](const Raw& x, int i) {
        if (i >= NST) ok = mbar_poll(&kempty[i % NST], ((i / NST) & 1) ^ 1, a.status, abrt);
        if (!ok) return false;
        put(sk + (i % NST) * Gm::kKBytes, x.row >= 0, x.kw, D, x.ks);
        fence_proxy_async();
        arrive_warp(&kfull[i % NST]);
        if (i >= NST) ok = mbar_poll(&zempty[i % NST], ((i / NST) & 1) ^ 1, a.status, abrt);
        if (!ok) return false;
        put(sz + (i % NST) * Gm::kZBytes, x.row >= 0, x.zw, RV, x.zs);
        fence_proxy_async();
        arrive_warp(&zfull[i % NST]);
        return true;
      };
      Raw x0, x1;
      fetch(x0, place(0));
      int next = place(1);
      for (int i = 0; i < n; i += 2) {
        fetch(x1, next);
        next = place(i + 2);
        if (!hand_over(x0, i) || i + 1 == n) break;
        fetch(x0, next);
        next = place(i + 3);
        if (!hand_over(x1, i + 1)) break;
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- softmax
    // queries into the swizzled layout first, D / 8 lanes a row
    {
#pragma unroll
      for (int x0 = 0; x0 < QN; x0 += QB) {
        if (x0 > 0) load_q(qv, x0);
#pragma unroll
        for (int x = 0; x < QB; ++x) {
          const int y = (x0 + x) * 256 + tid - 128, r = y / QC, c = y % QC;
          uint32_t u[4] = {qv[x].x, qv[x].y, qv[x].z, qv[x].w};
          if constexpr (!BF) {
            // f16 of the row times a power of two (largest magnitude in [2^14, 2^15))
            float mq = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = bf16x2_to_f2(u[k]);
              mq = fmaxf(mq, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
#pragma unroll
            for (int o = 1; o < QC; o <<= 1) mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
            const int ex = mq > 0.f ? (int)((__float_as_uint(mq) >> 23) & 0xffu) - 126 : 15;
            const int sh = max(-126, min(126, 15 - ex));
            const float sc = __uint_as_float((uint32_t)(127 + sh) << 23);
            if (c == 0) row_scale[r] = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = bf16x2_to_f2(u[k]);
              const __half2 hh = __floats2half2_rn(f.x * sc, f.y * sc);
              u[k] = *reinterpret_cast<const uint32_t*>(&hh);
            }
          }
          sts128(sq + (r >> 7) * (Gm::kQBytes / 2) + tc_off(r & 127, c), u[0], u[1], u[2], u[3]);
        }
      }
      fence_proxy_async();
      if (!BF || Gm::kQSteps > 0) named_bar_sync(1, 256);  // the rows and row_scale
    }
    const int t = (warp >> 2) - 1, r = tid & 127, row = t * 128 + r;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + Gm::kO + RV * t;
    if constexpr (Gm::kQSteps > 0) {  // the thread's row, from shared to tensor memory
      const uint32_t tq = tmem + lanes + Gm::kQ + 8 * Gm::kQSteps * t;
#pragma unroll
      for (int x = 0; x < Gm::kQSteps / 4; ++x) {
        uint32_t u[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = lds128(sq + t * (Gm::kQBytes / 2) + tc_off(r, 8 * x + c));
          u[4 * c] = v.x, u[4 * c + 1] = v.y, u[4 * c + 2] = v.z, u[4 * c + 3] = v.w;
        }
        tc_st32(tq + 32 * x, u);
      }
      tc_wait_st();
      tc_fence_before_sync();
    }
    arrive_warp(qfull);
    if (t < nt) {
      const int j = row >> a.logG, h = row & (a.G - 1);
      const bool live = row < rows;
      const int pos = live ? it.pos0 + j : -1;
      const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      // the row tile's first and last positions
      const int pos_a = it.pos0 + t * tq, pos_b = min(it.pos0 + (t + 1) * tq, it.live_end) - 1;
      const int lo_b = a.window > 0 ? max(0, pos_b - a.window + 1) : 0;
      const float sl = BF ? a.scale_log2 : a.scale_log2 * row_scale[row];
      const uint64_t sl2 = pack2(__float_as_uint(sl), __float_as_uint(sl));
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int u = 0; u < n2; ++u) {
        const uint32_t tu = ts + 64 * (u & 1);
        ok = mbar_poll(&sfull[2 * t + (u & 1)], (u >> 1) & 1, a.status, abrt);
        if (!ok) break;
        tc_fence_after_sync();
        const int t0 = tc_tile(it, i0 + (u >> 1)) * 128 + 64 * (u & 1);
        const bool all_seen = t0 + 63 <= pos_a && (t0 >= lo_b || t0 + 63 < a.sink);
        // Where a row's maximum has outgrown its reference, the warp moves that, rescales
        // O, and reads S again.
        uint64_t sum = 0;
#pragma unroll 1
        while (ok) {
          uint32_t sa[32], sb[32];
          tc_ld32(tu, sa);
          tc_ld32(tu + 32, sb);
          tc_wait_ld(sa);
          tc_wait_ld(sb);
          if (!all_seen) {
            // column x holds token t0 + x: visible up to pos, from lo on or below
            // the sinks' end
            const int me = pos - t0, mf = lo - t0, mg = a.sink - t0;
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              if (x > me || (x < mf && x >= mg)) sa[x] = 0xff800000u;
              if (x + 32 > me || (x + 32 < mf && x + 32 >= mg)) sb[x] = 0xff800000u;
            }
          }
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int x = 0; x < 32; ++x)
            mx4[x & 3] = max3(mx4[x & 3], __uint_as_float(sa[x]), __uint_as_float(sb[x]));
          const float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]) * sl;
          const bool grow = mx > m + tc_slack<FMT>();
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? ex2(m - mx) : 1.f;
            if (grow) m = mx;
            if (u > 0) {
              l *= f;
              // the next S comes behind P Z of the step before this one
              ok = mbar_poll(&sfull[2 * t + ((u + 1) & 1)], ((u + 1) >> 1) & 1, a.status, abrt);
              if (!ok) break;
              tc_fence_after_sync();
#pragma unroll 1
              for (int x = 0; x < RV; x += 32) {
                uint32_t o[32];
                tc_ld32(to + x, o);
                tc_wait_ld(o);
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                tc_st32(to + x, o);
              }
            }
            continue;  // (no row grows again)
          }
          const uint32_t nb = __float_as_uint(m == -INFINITY ? 0.f : -m);
          const uint64_t nbase = pack2(nb, nb);
          // two weights a word; bf16: the remainders of 32 tokens behind their weights
          auto weights = [&](const uint32_t (&s)[32], uint32_t* out) {
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              float p0, p1;
              unpack2(fma2(pack2(s[y], s[y + 1]), sl2, nbase), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum = add2(sum, pack2(__float_as_uint(p0), __float_as_uint(p1)));
              if constexpr (BF) {
                // the roundings, and roundings of what they leave
                out[y / 2] = bf16_pair(p0, p1);
                float r0, r1;
                less_bf16_pair(p0, p1, out[y / 2], r0, r1);
                out[16 + y / 2] = bf16_pair(r0, r1);
              } else {
                const __half2 v = __floats2half2_rn(p0, p1);
                out[y / 2] = *reinterpret_cast<const uint32_t*>(&v);
              }
            }
          };
          if constexpr (BF) {
            uint32_t p[32];
            weights(sa, p);
            tc_st32(tu, p);  // over S
            weights(sb, p);
            tc_st32(tu + 32, p);
          } else {
            uint32_t p[32];
            weights(sa, p);
            weights(sb, p + 16);
            tc_st32(tu, p);
          }
          break;
        }
        if (!ok) break;
        float sum0, sum1;
        unpack2(sum, sum0, sum1);
        l += sum0 + sum1;
        tc_wait_st();
        tc_fence_before_sync();
        arrive_warp(&pfull[2 * t + (u & 1)]);
      }
      if (n2 > 1 && ok) ok = mbar_poll(&sfull[2 * t + (n2 & 1)], (n2 >> 1) & 1, a.status, abrt);
      if (n2 > 0 && ok)
        ok = mbar_poll(&sfull[2 * t + ((n2 + 1) & 1)], ((n2 + 1) >> 1) & 1, a.status, abrt);
      if (ok) {
        tc_fence_after_sync();
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const size_t slot = part;
        float* po = a.partial + (slot * kTcRows + row) * RV;
        float* pm = a.partial + (size_t)plan.tail * plan.ns * kTcRows * RV + (slot * kTcRows + row) * 2;
        uint16_t* out =
            a.out + (((size_t)it.b * a.n_tot + it.j0 + j) * a.Hq + it.g * a.G + h) * RV;
#pragma unroll
        for (int x = 0; x < RV / 32; ++x) {
          uint32_t o[32];
          if (n > 0) {
            tc_ld32(to + 32 * x, o);
            tc_wait_ld(o);
          } else {
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = 0u;
          }
          if (live && nsplit == 1) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 u =
                    __floats2bfloat162_rn(__uint_as_float(o[y + 2 * k]) * inv,
                                          __uint_as_float(o[y + 2 * k + 1]) * inv);
                v[k] = *reinterpret_cast<const uint32_t*>(&u);
              }
              *reinterpret_cast<uint4*>(out + 32 * x + y) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          } else if (live) {
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              *reinterpret_cast<uint4*>(po + 32 * x + y) =
                  make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
        }
        if (live && nsplit > 1) {
          pm[0] = m;
          pm[1] = l;
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

// Joins the plan.ns partial sums of every row of the split items: a thread 4
// columns.
template <int RV>
__global__ void __launch_bounds__(256) span_tc_merge_kernel(SpanArgs a, TcPlan plan) {
  pdl_wait();
  pdl_launch_dependents();
  const TcItem it = tc_place(a, plan.full + blockIdx.x);
  const int rows = min(kTcRows, (a.n_tot - it.j0) << a.logG), nsplit = plan.ns;
  const float* ml = a.partial + (size_t)plan.tail * nsplit * kTcRows * RV;
  for (int o = blockIdx.y * 256 + threadIdx.x; o < rows * (RV / 4); o += gridDim.y * 256) {
    const int row = o / (RV / 4), c = (o - row * (RV / 4)) * 4;
    float M = -INFINITY, L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < nsplit; ++s) {
      const size_t slot = ((size_t)blockIdx.x * nsplit + s) * kTcRows + row;
      const float2 v = __ldcg(reinterpret_cast<const float2*>(ml + slot * 2));
      if (v.x == -INFINITY) continue;
      const float4 x = __ldcg(reinterpret_cast<const float4*>(a.partial + slot * RV + c));
      const float mn = fmaxf(M, v.x);
      const float f0 = M == -INFINITY ? 0.f : ex2(M - mn), f1 = ex2(v.x - mn);
      L = fmaf(L, f0, v.y * f1);
      A.x = fmaf(A.x, f0, x.x * f1);
      A.y = fmaf(A.y, f0, x.y * f1);
      A.z = fmaf(A.z, f0, x.z * f1);
      A.w = fmaf(A.w, f0, x.w * f1);
      M = mn;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const int j = row >> a.logG, h = row & (a.G - 1);
    const __nv_bfloat162 u = __floats2bfloat162_rn(A.x * inv, A.y * inv);
    const __nv_bfloat162 w = __floats2bfloat162_rn(A.z * inv, A.w * inv);
    *reinterpret_cast<uint2*>(
        a.out + (((size_t)it.b * a.n_tot + it.j0 + j) * a.Hq + it.g * a.G + h) * RV + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&w));
  }
}

template <int FMT, int D, int RV>
cudaError_t launch_span_tc_t(const SpanArgs& a, cudaStream_t st, bool pdl) {
  const TcPlan plan = tc_plan(a.B, a.Hkv, a.G, a.n_tot, a.max_seq_len, a.sink, a.window, a.r_v);
  cudaError_t e = cudaFuncSetAttribute(span_tc_kernel<FMT, D, RV>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)TcGeom<D, RV>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_k(span_tc_kernel<FMT, D, RV>, dim3(plan.full + plan.tail * plan.ns),
               dim3(kTcThreads), TcGeom<D, RV>::kSmem, st, pdl, a, plan);
  if (e != cudaSuccess || plan.ns == 1) return e;
  const int rows = a.n_tot * a.G < kTcRows ? a.n_tot * a.G : kTcRows;
  return launch_k(span_tc_merge_kernel<RV>, dim3(plan.tail, (rows * (RV / 4) + 255) / 256),
                  dim3(256), 0, st, pdl, a, plan);
}

template <int FMT>
cudaError_t launch_span_tc_fmt(const SpanArgs& a, cudaStream_t st, bool pdl) {
#define BKV_SPAN_TC_RV(DD)                                          \
  switch (a.r_v) {                                                  \
    case 32: return launch_span_tc_t<FMT, DD, 32>(a, st, pdl);      \
    case 64: return launch_span_tc_t<FMT, DD, 64>(a, st, pdl);      \
    case 96: return launch_span_tc_t<FMT, DD, 96>(a, st, pdl);      \
    default: return launch_span_tc_t<FMT, DD, 128>(a, st, pdl);     \
  }
  if (a.d == 64) {
    BKV_SPAN_TC_RV(64)
  } else {
    BKV_SPAN_TC_RV(128)
  }
#undef BKV_SPAN_TC_RV
}

}  // namespace
}  // namespace basiskv
