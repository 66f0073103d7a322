// Attention of a few query rows over a long span of one sequence's tokens,
// streamed once: a sliding window with sinks, the whole context, or the
// pages of a selection (instances: span_bf16.cu, span_e4m3.cu, span_q4.cu).
//
//   a[row] = sum_t p_t z_t,  p = softmax over the row's tokens of
//   (q . K_t) / sqrt(d)
//
// Rows: query token j and head h of KV head g make row j * G + h; up to 32 rows
// (one to four N tiles of mma.m16n8k16) share every Key and latent that is
// read.
// Bound by HBM: 2 (d + r_v) multiply-adds a row and (d + r_v) cached columns a token;
// over 4-bit caches as much by the chain of a unit, in which the codes are widened (a
// conversion and a multiplication for two columns).
//
// Split: the unit of work is 16 tokens (4-bit caches: 32).  All units of all
// (sequence, KV head) items form one line in (b, g, unit) order, cut into
// equal contiguous runs, one a CTA, so that ragged lengths load every SM
// alike; each CTA finds its run from a scan of the sequences' lengths.  A
// CTA's 8 warps take every 8th unit of the run, keep their own running
// maximum, sum and accumulators, and meet in shared memory where the run
// passes from one item to the next.  An item that lies in one CTA is written
// there; the others leave one partial a CTA, which span_merge_kernel joins
// (the second launch, scheduled early).
//
// Data path: each warp brings its units into its own ring of shared memory,
// kStages - 1 units ahead and across item borders; no other warp waits for
// it.  E4M3 and 4-bit units are one or a few contiguous pieces: one lane
// hands them to the copy engine (cp.async.bulk), which costs a few
// instructions a unit where 16-byte copies by all lanes cost 40 (a gather of
// 1152 + 576 byte tiles alone runs at 6.2 TB/s this way).  bf16 units are
// copied 16 bytes a lane, swizzled for ldmatrix.  The Keys are the A operand
// of QK (rows = tokens, the head dimension in the order the lanes hold it) and
// the latents PV's A operand (rows = latent columns: a lane reads the same
// columns of neighbouring tokens and pairs them); the scores, [token][row],
// become PV's B operand with one 8x8 transposition per 8 tokens.
//
// The running reference moves only when a score passes it by a wide margin
// (2^15 or 2^32 in the weights, which the operands' types hold): then the warp
// takes the rows' maxima over their lanes and rescales; all other units cost
// one vote.
//
// Precision: scores and sums in fp32.  The weights of PV are rounded to f16
// (2^-11 of each weight, an eighth of the output's own rounding) where the
// operands are f16, and held as bf16 roundings plus bf16 remainders (16
// significant bits, a second product) where they are bf16.
//
// Measured (16 x 32K tokens, 8 KV heads, d 128, r_v 64, G 4): bf16, window 4096
// (202 MB) 42 us, 4.8 TB/s; E4M3, the same 30 us, all tokens (806 MB) 135, 6.0 TB/s; 4
// bits, all tokens (453 MB) 110 us, 4.1 TB/s, with neither HBM nor the issue slots
// (62%) full: without the conversions 107, without the scales' products 94; 128 selected
// pages of 4 bits (28 MB) 19 us, a start of 8 us and one turn of the ring;
// E4M3, 7 ragged sequences, window 8192, 20 rows (89 MB) 41 us against 69 on
// the prompt kernel.  Joining the partials of an item with one CTA took 23 us
// longer there; one output a thread, over more CTAs, about 2.
//
// Formats: bf16 (bf16 products), E4M3 and 4 bits (widened to f16, which is
// exact; each row's query is brought to f16 by a power of two that puts its
// largest magnitude into [2^14, 2^15), divided out of the scores again).
#pragma once

#include "cache4.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "line_scan.cuh"

namespace basiskv {
namespace {

constexpr int kSpThreads = kLineMaxSeqs;  // a thread scans a sequence's length
constexpr int kSpWarps = kSpThreads / 32;
// How far (log2) scores may pass the reference before it moves: the weights then
// reach 2^15 in f16, 2^32 in bf16, at the same relative precision, and their products
// and sums stay inside fp32's range: over bf16 caches for latents up to 2^64 and 2^30
// tokens.  (2^64, at the same times, overflowed from latents of 2^60 on.)
template <int FMT>
constexpr float sp_slack() {
  return FMT == kSpanBf16 ? 32.f : 15.f;
}

// Tokens of a unit: 32 over 4-bit caches, and over E4M3 ones where 17 to 32 rows
// leave a warp a scheduler and a half (two steps of 16 tokens side by side: 46
// -> 43 us with 20 rows over 89 MB; pages of 8 tokens are not halves of such a unit).
template <int FMT, int NR>
constexpr int sp_unit() {
  return FMT == kSpanQ4 || (FMT == kSpanE4m3 && NR > 2) ? 32 : 16;
}

// What one sequence contributes: its live length, and the units of one KV
// head (n_sink units of sink tokens, then the window's from lo_unit on).
struct SpanSeq {
  int T, n_sink, lo_unit, n;
};
template <int UT>
__device__ __forceinline__ SpanSeq span_seq(const SpanArgs& a, int len) {
  SpanSeq s;
  s.T = len;
  const int last = len - 1;
  if (len <= 0 || len > a.max_seq_len) {
    s.T = 0;
    s.n_sink = s.lo_unit = s.n = 0;
  } else if (a.sel) {
    s.n_sink = s.lo_unit = 0;
    s.n = a.S >= UT ? a.top_k * (a.S / UT) : (a.top_k + 1) >> 1;
  } else {
    const int lo = a.window > 0 ? max(0, max(len - a.n_tot, 0) - a.window + 1) : 0;
    s.lo_unit = lo / UT;
    s.n_sink = min((a.sink + UT - 1) / UT, s.lo_unit);
    s.n = s.n_sink + last / UT - s.lo_unit + 1;
  }
  return s;
}

// pre[b] = units of one KV head of the sequences before b; pre[B] = all.  The
// lengths are left in lens for the lookups that follow, where that is given.
template <int UT>
__device__ __forceinline__ void span_scan(const SpanArgs& a, long long* pre, bool report,
                                          int* lens = nullptr) {
  line_scan(a.B, pre, [&](int b) -> long long {
    const int len = a.seq_lens[b];
    if (lens) lens[b] = len;
    if (report && (len < 0 || len > a.max_seq_len)) raise_status(a.status, BASISKV_DEV_BAD_LENGTH);
    return span_seq<UT>(a, len).n;
  });
}

// x / n for line positions, which seldom need 64 bits.
__device__ __forceinline__ long long line_div(long long x, int n) {
  return (unsigned long long)x >> 32 ? x / n : (long long)((unsigned)x / (unsigned)n);
}

// CTAs that share the line: all of the grid, or fewer when the lengths at hand
// leave less than kSpMinUnits units for each (so each of them has units).
constexpr int kSpMinUnits = kSpWarps;
__device__ __forceinline__ int span_ctas(long long total, int grid) {
  const long long c = total / kSpMinUnits > 0 ? total / kSpMinUnits : 1;
  return (int)(c < grid ? c : grid);
}
__device__ __forceinline__ int span_cta_of(long long x, long long total, int C) {
  const long long c = ((x + 1) * C - 1) / total;
  return (int)(c < C - 1 ? c : C - 1);
}

// Bytes of one unit in a warp's ring, and of the ring's part of shared memory.
template <int FMT, int D, int RV, int NR>
constexpr int sp_unit_bytes() {
  return sp_unit<FMT, NR>() * (D + RV) * (FMT == kSpanBf16 ? 32 : (FMT == kSpanE4m3 ? 16 : 9)) / 16;
}
// CTAs an SM: two, except where the queries' and accumulators' registers (more
// than 8 rows) or the ring (bf16) allow one.
template <int FMT, int NR>
constexpr int sp_ctas() {
  return FMT == kSpanBf16 || NR >= 2 ? 1 : 2;
}
// The warps meet with at most 16 rows at a time.  A row: its accumulators in the
// lanes' order (position 8 t + n: tile t, lane column n; the pad keeps the lanes'
// writes on different banks), then maximum, sum, factor and joint sum.
constexpr int kSpRowPad = kSpanRowPad;
template <int FMT, int D, int RV, int NR>
constexpr size_t sp_meet_bytes() {
  return (size_t)kSpWarps * 8 * (NR < 2 ? NR : 2) * (RV + kSpRowPad) * 4;
}
// Ring depth: 4 units, fewer where shared memory ends (2 at least).
template <int FMT, int D, int RV, int NR>
constexpr int sp_stages() {
  const size_t room = 224 * 1024 / sp_ctas<FMT, NR>() - 6 * 1024 - sp_meet_bytes<FMT, D, RV, NR>();
  const size_t n = room / ((size_t)kSpWarps * sp_unit_bytes<FMT, D, RV, NR>());
  return n < 4 ? (int)n : 4;
}
template <int FMT, int D, int RV, int NR>
constexpr size_t sp_smem() {
  return (size_t)kSpWarps * sp_stages<FMT, D, RV, NR>() * sp_unit_bytes<FMT, D, RV, NR>() +
         sp_meet_bytes<FMT, D, RV, NR>();
}

// The latent column that lane column n (0..7) of accumulator tile t holds:
// the order in which the lanes read a latent row.
template <int FMT, int RV>
__device__ __forceinline__ int sp_col(int t, int n) {
  if (FMT == kSpanBf16) return 8 * t + n;
  if (FMT == kSpanE4m3) return 32 * (t >> 2) + 4 * n + (t & 3);
  if (t < 8 * (RV / 64)) return 64 * (t >> 3) + 8 * n + (t & 7);
  return 64 * (RV / 64) + 4 * n + (t & 3);
}
// Swizzled 16-byte chunk of a bf16 latent row in shared memory.
template <int RV>
__device__ __forceinline__ int sp_zchunk(int r, int ch) {
  if (RV == 32) return ch ^ ((r >> 1) & 3);
  if (RV == 96 && ch >= 8) return 8 + ((ch ^ (r >> 1)) & 3);
  return ch ^ (r & 7);
}

__device__ __forceinline__ void mbar_arrive_only(uint32_t bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(bar)
               : "memory");
}

// ONE (4-bit caches): a unit is one page of 32 tokens, else two of 16.
template <int FMT, int D, int RV, int NR, bool ONE>
__global__ void __launch_bounds__(kSpThreads, sp_ctas<FMT, NR>()) span_kernel(SpanArgs a) {
  constexpr int UT = sp_unit<FMT, NR>(), HT = UT / 2;  // tokens of a unit, of its halves
  constexpr int VT = UT / 16;                      // 16-token steps
  constexpr int MT = RV / 16, KS = D / 16, NST = sp_stages<FMT, D, RV, NR>();
  constexpr int UB = sp_unit_bytes<FMT, D, RV, NR>();
  constexpr int RS = RV + kSpRowPad;
  constexpr bool BULK = FMT != kSpanBf16;
  static_assert(NST >= 2 && (D + RV) * UT / 16 * 9 % 16 == 0, "");
  extern __shared__ __align__(128) uint8_t sp_smem_raw[];
  __shared__ long long pre[257];
  __shared__ int lens[kLineMaxSeqs];
  __shared__ uint2 tags[kSpWarps][NST];      // a unit's halves: first tokens (~0: absent)
  __shared__ uint64_t bars[kSpWarps * NST];  // a unit has landed
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(sp_smem_raw) + warp * NST * UB;
  const uint32_t bar = smem_u32(bars + warp * NST);
  // [warp][row][RS] where the warps meet after an item
  float* meet = reinterpret_cast<float*>(sp_smem_raw + kSpWarps * NST * UB);
  const int R = a.n_tot * a.G;

  if (BULK && tid < kSpWarps * NST) mbar_init(bars + tid, 1);
  if (BULK) fence_barrier_init();
  pdl_wait();
  pdl_launch_dependents();
  span_scan<UT>(a, pre, blockIdx.x == 0, lens);
  const long long total = pre[a.B] * a.Hkv;
  const int C = span_ctas(total, gridDim.x);
  if ((int)blockIdx.x >= C) return;
  // the run [start, start + run) of the line; `start` stays in shared memory
  __shared__ long long start;
  int run;
  {
    const long long s0 = line_div(total * blockIdx.x, C);
    run = (int)(line_div(total * (blockIdx.x + 1), C) - s0);
    if (tid == 0) start = s0;
  }
  __syncthreads();
  if (run <= 0) return;

  // ---- the warp's units: warp + 8 k of the run, k < n_units, whatever their items
  const int n_units = warp < run ? (run - warp + kSpWarps - 1) / kSpWarps : 0;
  // Ids of 32 units ahead, one a lane: the first token of the unit's halves and
  // their tile rows (physical page and KV head * S + row; -1: not there).
  int id_ta = 0, id_tb = 0, id_ra = -1, id_rb = -1, id_base = 0;
  auto fetch_ids = [&](int base) {
    id_base = base;
    id_ra = id_rb = -1;
    const int k = base + lane;
    if (k >= n_units) return;
    const long long x = start + warp + (long long)kSpWarps * k;
    const int b = line_find(a.B, pre, a.Hkv, x);
    const SpanSeq sq = span_seq<UT>(a, lens[b]);
    const long long y = x - pre[b] * a.Hkv;
    const int g = (int)line_div(y, sq.n), u = (int)(y - (long long)g * sq.n);
    const int lo = a.window > 0 ? max(0, max(sq.T - a.n_tot, 0) - a.window + 1) : 0;
    auto tile_row = [&](int t) -> int {
      // no row sees tokens between the sinks and the window: their pages are
      // not looked up
      if (t >= sq.T || (t + HT <= lo && t >= a.sink)) return -1;
      const int p = t >> a.logS;
      const int pp = p < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + p) : -1;
      if (pp < 0 || pp >= a.num_phys) {
        raise_status(a.status, BASISKV_DEV_BAD_PAGE);
        return -1;
      }
      return ((pp * a.Hkv + g) << a.logS) + (t & (a.S - 1));
    };
    auto selected = [&](int e) -> int {  // first token of selected page e, -1: none
      const int lp = e < a.top_k
                         ? __ldg(a.sel + (size_t)(b * a.Hkv + g) * a.top_k + e) : -1;
      if (lp >= a.max_pages) raise_status(a.status, BASISKV_DEV_BAD_PAGE);
      return lp >= 0 && lp < a.max_pages ? lp << a.logS : -1;
    };
    if (a.sel) {
      if (a.S >= UT) {
        id_ta = selected(u);
        id_tb = id_ta + HT;
      } else {
        id_ta = selected(2 * u);
        id_tb = selected(2 * u + 1);
      }
      if (id_ta >= 0) id_ra = tile_row(id_ta);
      if ((FMT == kSpanQ4 ? ONE : a.S >= UT) ? id_ta >= 0 : id_tb >= 0) id_rb = tile_row(id_tb);
    } else {
      id_ta = UT * (u < sq.n_sink ? u : sq.lo_unit + u - sq.n_sink);
      id_tb = id_ta + HT;
      id_ra = tile_row(id_ta);
      id_rb = tile_row(id_tb);
    }
  };
  // Requests unit k into ring slot `slot` (k grows by one from call to call).
  auto issue = [&](int k, int slot) {
    if (k < n_units) {
      if (k - id_base >= 32) fetch_ids(k);
      const uint32_t st = ring + slot * UB;
      if constexpr (BULK) {
        if (lane == k - id_base) {  // the lane that knows the unit
          tags[warp][slot] = make_uint2(id_ra >= 0 ? (uint32_t)id_ta : ~0u,
                                        id_rb >= 0 ? (uint32_t)id_tb : ~0u);
          const uint32_t b = bar + 8 * slot;
          auto copy = [&](uint32_t dst, const uint8_t* src, uint32_t bytes) {
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], "
                "%2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(b)
                : "memory");
          };
          auto expect = [&](uint32_t bytes) {
            asm volatile(
                "{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(b),
                "r"(bytes)
                : "memory");
          };
          const int present = (id_ra >= 0) + (id_rb >= 0);
          if (!present) {
            mbar_arrive_only(b);
          } else if constexpr (FMT == kSpanQ4) {
            if constexpr (ONE) {  // the unit is one tile: codes and scales of 32 rows
              const size_t tile = (id_ra >= 0 ? id_ra : id_rb - HT) >> a.logS;
              expect(UB);
              copy(st, a.K + tile * (2 * 9 * D), 2 * 9 * D);
              copy(st + 2 * 9 * D, a.Z + tile * (2 * 9 * RV), 2 * 9 * RV);
            } else {  // two tiles of 16 rows, one behind the other
              expect(present * (UB / 2));
              if (id_ra >= 0) {
                copy(st, a.K + (size_t)(id_ra >> a.logS) * (9 * D), 9 * D);
                copy(st + 2 * 9 * D, a.Z + (size_t)(id_ra >> a.logS) * (9 * RV), 9 * RV);
              }
              if (id_rb >= 0) {
                copy(st + 9 * D, a.K + (size_t)(id_rb >> a.logS) * (9 * D), 9 * D);
                copy(st + 2 * 9 * D + 9 * RV, a.Z + (size_t)(id_rb >> a.logS) * (9 * RV), 9 * RV);
              }
            }
          } else {  // E4M3 rows; latents [rows][F] and then [rows][RV - F]
            const int F = a.zsplit;
            expect(present * HT * (D + RV));
            auto half = [&](int row, int at, int rows) {
              copy(st + at * D, a.K + (size_t)row * D, rows * D);
              const uint8_t* tile = a.Z + (size_t)(row >> a.logS) * a.S * RV;
              const int r = row & (a.S - 1);
              copy(st + UT * D + at * F, tile + r * F, rows * F);
              if (F < RV)
                copy(st + UT * D + UT * F + at * (RV - F), tile + a.S * F + r * (RV - F),
                     rows * (RV - F));
            };
            if (a.S >= UT && present == 2) {
              half(id_ra, 0, UT);
            } else {
              if (id_ra >= 0) half(id_ra, 0, HT);
              if (id_rb >= 0) half(id_rb, HT, HT);
            }
          }
        }
      } else {
        const int src = k - id_base;
        const int ra = __shfl_sync(0xffffffffu, id_ra, src);
        const int rb = __shfl_sync(0xffffffffu, id_rb, src);
        if (lane == src)
          tags[warp][slot] = make_uint2(id_ra >= 0 ? (uint32_t)id_ta : ~0u,
                                        id_rb >= 0 ? (uint32_t)id_tb : ~0u);
        constexpr int KC = D / 8, ZC = RV / 8;
#pragma unroll
        for (int x = 0; x < 16 * KC; x += 32) {
          const int i = x + lane, r = i / KC, ch = i % KC;
          const int tr = r < HT ? ra + r : rb + r - HT;
          if (r < HT ? ra >= 0 : rb >= 0)
            cp_async16_or_zero(st + (r * KC + (ch ^ (r & 7))) * 16,
                               a.K + ((size_t)tr * D + ch * 8) * 2);
        }
#pragma unroll
        for (int x = 0; x < 16 * ZC; x += 32) {
          const int i = x + lane, r = i / ZC, ch = i % ZC;
          const int tr = r < HT ? ra + r : rb + r - HT;
          if (r < HT ? ra >= 0 : rb >= 0)
            cp_async16_or_zero(
                st + 32 * D + (r * ZC + sp_zchunk<RV>(r, ch)) * 16,
                a.Z + ((size_t)(tr >> a.logS) * a.S * RV +
                       split_off(tr & (a.S - 1), ch * 8, a.S, RV, a.zsplit)) * 2);
        }
      }
    }
    if constexpr (!BULK) cp_async_commit();
  };

  int k_next = 0, slot_next = 0;  // the next unit to request, and its slot
  bool landing = true;  // no wait has run out yet (the others would, too)
  auto request = [&]() {
    if (!landing) return;
    issue(k_next++, slot_next);
    slot_next = slot_next + 1 == NST ? 0 : slot_next + 1;
  };
  if (n_units > 0) fetch_ids(0);
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) request();
  int slot = 0;
  uint32_t phase = 0;  // of the slots' barriers in this turn of the ring

  // 4-bit units: byte offsets of half 1's codes and of the halves' scales
  // (Keys; the latents' are the same with RV for D), and of the lane in them
  constexpr int H1 = ONE ? 8 : 9, S0 = ONE ? 16 : 8, S1 = 17;
  const uint32_t lane_k = n * (D / 2) + (D / 8) * c, lane_ks = n * (D / 16) + (D / 64) * c;
  const uint32_t lane_z = 2 * c * (RV / 2) + 4 * n, lane_zs = 2 * c * (RV / 16) + (n >> 1);

  int seg = 0;  // the run's next unit
  while (seg < run) {
    int b, g, count, item_end;
    bool alone;  // the whole item is in this run
    SpanSeq sq;
    {
      const long long x = start + seg;
      b = line_find(a.B, pre, a.Hkv, x);
      sq = span_seq<UT>(a, lens[b]);
      const long long y = x - pre[b] * a.Hkv;
      g = (int)line_div(y, sq.n);
      const int u = (int)(y - (long long)g * sq.n);  // the item's unit at seg
      item_end = min(run, seg + sq.n - u);
      alone = u == 0 && item_end == seg + sq.n;
      // the run's warps take turns from its start on, whatever the item
      const int w0 = seg + ((warp - seg) & (kSpWarps - 1));
      count = w0 < item_end ? (item_end - w0 + kSpWarps - 1) / kSpWarps : 0;
    }
    const int bg = b * a.Hkv + g;
    const int pos0 = sq.T - a.n_tot, p_last = sq.T - 1;  // the rows' positions
    const int lo_first = a.window > 0 ? max(0, max(pos0, 0) - a.window + 1) : 0;
    const int lo_last = a.window > 0 ? max(0, p_last - a.window + 1) : 0;

    // ---- queries (B operand of QK): lane (n, c) holds columns of rows n, n + 8
    uint32_t qb[KS][NR][2];
    // of rows 2c, 2c + 1 (+ 8), whose scores the lane gets: score factor, position
    float sl[NR][2];
    int pos[NR][2];
    auto column = [&](int k, int e) {  // of the pair in qb[k][.][e]
      return FMT == kSpanBf16 ? 16 * k + 8 * e + 2 * c
             : FMT == kSpanE4m3 ? 64 * (k >> 2) + 16 * c + 4 * (k & 3) + 2 * e
                                : (D / 4) * c + 4 * k + 2 * e;
    };
#pragma unroll
    for (int i = 0; i < NR; ++i) {  // all loads before the first use
      const int r = n + 8 * i, j = r >> a.logG, h = r & (a.G - 1);
      const bool ok = r < R;
      const uint16_t* qr =
          a.q + (((size_t)b * a.n_tot + (ok ? j : 0)) * a.Hq + g * a.G + (ok ? h : 0)) * D;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if constexpr (FMT == kSpanBf16) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qb[k][i][e] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qr + column(k, e))) : 0u;
        } else {
          const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(qr + column(k, 0)))
                             : make_uint2(0u, 0u);
          qb[k][i][0] = w.x;
          qb[k][i][1] = w.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * i + 2 * c + e;
        pos[i][e] = row < R ? pos0 + (row >> a.logG) : -1;
        sl[i][e] = a.scale_log2;
      }
      if constexpr (FMT != kSpanBf16) {
        float mq = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = bf16x2_to_f2(qb[k][i][e]);
            mq = fmaxf(mq, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 1));
        mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 2));
        const int ex = mq > 0.f ? (int)((__float_as_uint(mq) >> 23) & 0xffu) - 126 : 15;
        const int sh = max(-126, min(126, 15 - ex));
        const float sc = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = bf16x2_to_f2(qb[k][i][e]);
            const __half2 hh = __floats2half2_rn(f.x * sc, f.y * sc);
            qb[k][i][e] = *reinterpret_cast<const uint32_t*>(&hh);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int sh2 = __shfl_sync(0xffffffffu, sh, 4 * (2 * c + e));
          sl[i][e] *= __uint_as_float((uint32_t)(127 - sh2) << 23);
        }
      }
    }

    // m: the rows' reference (log2 units); thr: the raw score that moves it
    float m[NR][2], thr[NR][2], l[NR][2], acc[MT][NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) m[i][e] = thr[i][e] = -INFINITY, l[i][e] = 0.f;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < NR; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;

    for (int it = 0; it < count; ++it) {
      __syncwarp();  // every lane is done with the slot that is filled next
      request();
      if constexpr (BULK) {
        landing = landing && mbar_poll(bars + warp * NST + slot, phase, a.status);
      } else {
        cp_async_wait_group<NST - 1>();
        __syncwarp();
      }
      const uint2 tag = tags[warp][slot];
      const uint32_t ks = ring + slot * UB, zs = ks + UT * D * (FMT == kSpanBf16 ? 32 : FMT == kSpanE4m3 ? 16 : 9) / 16;
      if (++slot == NST) {
        slot = 0;
        phase ^= 1;
      }
      if ((tag.x & tag.y) == ~0u) continue;  // nothing there
      const int ta = (int)tag.x, tb = (int)tag.y;  // first tokens of the halves
      auto half_seen = [&](int t0) {
        return t0 >= 0 && t0 + HT - 1 <= pos0 && (t0 >= lo_last || t0 + HT - 1 < a.sink);
      };
      const bool all_seen = half_seen(ta) && half_seen(tb);
      // the unit's token u (negative: absent)
      auto token = [&](int u) {
        const int first = u < HT ? ta : tb;
        return first < 0 ? -1 : first + (u < HT ? u : u - HT);
      };
      if (!all_seen) {
        // Latents of tokens that no row sees may hold anything, and 0 * NaN
        // would poison the sums: they (4 bits: their scales) are zeroed here.
        if (lane < UT) {
          const int tt = token(lane);
          if (!(tt >= 0 && tt <= p_last && (tt >= lo_first || tt < a.sink))) {
            if constexpr (FMT == kSpanQ4) {
              const uint32_t at = zs + (lane < 16 ? S0 : S1) * RV + (lane & 15) * (RV / 16);
#pragma unroll
              for (int k = 0; k < RV / 16; k += 2)
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + k), "h"((unsigned short)0)
                             : "memory");
            } else if constexpr (FMT == kSpanE4m3) {
              const int F = a.zsplit;
#pragma unroll
              for (int k = 0; k < RV; k += 16) {
                const uint32_t at = zs + (k < F ? lane * F + k : UT * F + lane * (RV - F) + k - F);
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u)
                             : "memory");
              }
            } else {
#pragma unroll
              for (int k = 0; k < RV / 8; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 zs + lane * (2 * RV) + 16 * k),
                             "r"(0u)
                             : "memory");
            }
            if (BULK) fence_proxy_async();  // the slot's next bytes come from the copy engine
          }
        }
        __syncwarp();
      }
      // ---- scores: s[v][i] = tokens 16 v + n (e < 2) and + 8, rows 8 i + 2c, + 1
      float s[VT][NR][4];
#pragma unroll
      for (int v = 0; v < VT; ++v)
#pragma unroll
        for (int i = 0; i < NR; ++i) s[v][i][0] = s[v][i][1] = s[v][i][2] = s[v][i][3] = 0.f;
      auto qk = [&](int v, int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          if constexpr (FMT == kSpanBf16)
            mma_bf16_16816(s[v][i], a0, a1, a2, a3, qb[k][i][0], qb[k][i][1]);
          else
            mma_f16_16816(s[v][i], a0, a1, a2, a3, qb[k][i][0], qb[k][i][1]);
        }
      };
      if constexpr (FMT == kSpanBf16) {
        const int row = lane & 15;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int ch = (2 * k + (lane >> 4)) ^ (row & 7);
          uint32_t a0, a1, a2, a3;
          ldmatrix_x4(ks + row * (2 * D) + ch * 16, a0, a1, a2, a3);
          qk(0, k, a0, a1, a2, a3);
        }
      } else if constexpr (FMT == kSpanE4m3) {
#pragma unroll
        for (int k4 = 0; k4 < KS / 4; ++k4)
#pragma unroll
          for (int v = 0; v < VT; ++v) {
            // 16 columns of tokens n and n + 8
            const uint4 x = lds128(ks + (16 * v + n) * D + (c + 4 * k4) * 16);
            const uint4 y = lds128(ks + (16 * v + n + 8) * D + (c + 4 * k4) * 16);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(xw[w], a0, a2);
              e4m3x4_to_f16(yw[w], a1, a3);
              qk(v, 4 * k4 + w, a0, a1, a2, a3);
            }
          }
      } else {
        // D / 4 columns of tokens n and n + 8: D / 8 bytes, one scale per 16
        const uint32_t kl = ks + lane_k, kls = ks + lane_ks;
#pragma unroll
        for (int v = 0; v < VT; ++v) {
          uint32_t xw[2][D / 32], sx[2][D / 64];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t row = kl + v * H1 * D + y * 8 * (D / 2);
            const uint32_t scl = kls + (v ? S1 : S0) * D + y * 8 * (D / 16);
            if constexpr (D == 128) {
              const uint4 x = lds128(row);
              xw[y][0] = x.x, xw[y][1] = x.y, xw[y][2] = x.z, xw[y][3] = x.w;
              const uint32_t u = lds16(scl);
              sx[y][0] = __byte_perm(u, 0u, 0x4040) << 7;
              sx[y][D / 64 - 1] = __byte_perm(u, 0u, 0x4141) << 7;
            } else {
              const uint2 x = lds64(row);
              xw[y][0] = x.x, xw[y][1] = x.y;
              sx[y][0] = q4_scale_x2(lds8(scl));
            }
          }
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            uint32_t x[4], y[4];
            q4_unpack8(xw[0][w], x);
            q4_unpack8(xw[1][w], y);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              qk(v, 2 * w + e, hmul2(x[2 * e], sx[0][w / 2]), hmul2(y[2 * e], sx[1][w / 2]),
                 hmul2(x[2 * e + 1], sx[0][w / 2]), hmul2(y[2 * e + 1], sx[1][w / 2]));
          }
        }
      }
      // ---- softmax weights
      if (!all_seen) {
#pragma unroll
        for (int v = 0; v < VT; ++v)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int tt = token(16 * v + n + 8 * y);
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int p = pos[i][e], lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
                if (!(tt >= 0 && tt <= p && (tt >= lo || tt < a.sink)))
                  s[v][i][2 * y + e] = -INFINITY;
              }
          }
      }
      bool grow = false;
      float mx[NR][2];
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[i][e] = fmaxf(s[0][i][e], s[0][i][2 + e]);
#pragma unroll
          for (int v = 1; v < VT; ++v)
            mx[i][e] = fmaxf(mx[i][e], fmaxf(s[v][i][e], s[v][i][2 + e]));
          grow |= mx[i][e] > thr[i][e];
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = mx[i][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            const float mn = fmaxf(m[i][e], x * sl[i][e]);
            f[e] = mn == -INFINITY ? 1.f : ex2(m[i][e] - mn);
            m[i][e] = mn;
            thr[i][e] = (mn + sp_slack<FMT>()) / sl[i][e];
            l[i][e] *= f[e];
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            acc[t][i][0] *= f[0];
            acc[t][i][1] *= f[1];
            acc[t][i][2] *= f[0];
            acc[t][i][3] *= f[1];
          }
        }
      }
      // B operand of PV: rows n (+ 8 i), tokens 16 v + 2c, + 1 and + 8, + 9
      uint32_t pb[VT][NR][2], pr[VT][NR][2];  // roundings; remainders (bf16)
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float base0 = m[i][0] == -INFINITY ? 0.f : m[i][0];
        const float base1 = m[i][1] == -INFINITY ? 0.f : m[i][1];
#pragma unroll
        for (int v = 0; v < VT; ++v)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p0 = ex2(fmaf(s[v][i][2 * y], sl[i][0], -base0));
            const float p1 = ex2(fmaf(s[v][i][2 * y + 1], sl[i][1], -base1));
            l[i][0] += p0;
            l[i][1] += p1;
            if constexpr (FMT == kSpanBf16) {
              uint32_t hi, rest;
              split_bf16x2(p0, p1, hi, rest);
              pb[v][i][y] = movmatrix_trans(hi);
              pr[v][i][y] = movmatrix_trans(rest);
            } else {
              const __half2 hh = __floats2half2_rn(p0, p1);
              pb[v][i][y] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&hh));
            }
          }
      }
      // ---- latents (A operand of PV), 16 columns and 16 tokens a product
#pragma unroll
      for (int v = 0; v < VT; ++v) {
        auto pv = [&](int t, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            if constexpr (FMT == kSpanBf16) {
              mma_bf16_16816(acc[t][i], a0, a1, a2, a3, pb[v][i][0], pb[v][i][1]);
              mma_bf16_16816(acc[t][i], a0, a1, a2, a3, pr[v][i][0], pr[v][i][1]);
            } else {
              mma_f16_16816(acc[t][i], a0, a1, a2, a3, pb[v][i][0], pb[v][i][1]);
            }
          }
        };
        if constexpr (FMT == kSpanQ4) {
          const uint32_t zl = zs + lane_z + v * H1 * RV, zls = zs + lane_zs + (v ? S1 : S0) * RV;
          // scale pairs of a block for tokens (2c, 2c + 1) and (+ 8, + 9)
          auto scales = [&](uint32_t at, uint32_t& s01, uint32_t& s89) {
            s01 = __byte_perm(lds8(at), lds8(at + RV / 16), 0x5410) << 7;
            s89 = __byte_perm(lds8(at + 8 * (RV / 16)), lds8(at + 9 * (RV / 16)), 0x5410) << 7;
          };
          // the 8 columns of two tokens, paired
          auto pairs = [&](uint32_t x0, uint32_t y0, uint32_t (&f)[8]) {
            uint32_t lo4[4], hi4[4];
            q4_unpack8((x0 & 0x0f0f0f0fu) | ((y0 << 4) & 0xf0f0f0f0u), lo4);
            q4_unpack8(((x0 >> 4) & 0x0f0f0f0fu) | (y0 & 0xf0f0f0f0u), hi4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[2 * j] = lo4[j];
              f[2 * j + 1] = hi4[j];
            }
          };
#pragma unroll
          for (int w = 0; w < RV / 64; ++w) {
            uint32_t x[4], f0[8], f1[8], s01, s89;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = lds32(zl + ((e & 1) + 8 * (e >> 1)) * (RV / 2) + 32 * w);
            pairs(x[0], x[1], f0);
            pairs(x[2], x[3], f1);
            scales(zls + 4 * w, s01, s89);
#pragma unroll
            for (int j = 0; j < 8; j += 2)
              pv(4 * w + j / 2, hmul2(f0[j], s01), hmul2(f0[j + 1], s01), hmul2(f1[j], s89),
                 hmul2(f1[j + 1], s89));
          }
          if constexpr (RV % 64 != 0) {  // 32 more columns, 4 a lane
            constexpr int W0 = RV / 64;
            uint32_t x[4], f0[8], f1[8], s01, s89;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = lds16(zl - 2 * n + ((e & 1) + 8 * (e >> 1)) * (RV / 2) + 32 * W0);
            pairs(x[0], x[1], f0);
            pairs(x[2], x[3], f1);
            scales(zls - (n >> 1) + (n >> 2) + 4 * W0, s01, s89);
#pragma unroll
            for (int j = 0; j < 4; j += 2)
              pv(4 * W0 + j / 2, hmul2(f0[j], s01), hmul2(f0[j + 1], s01), hmul2(f1[j], s89),
                 hmul2(f1[j + 1], s89));
          }
        } else if constexpr (FMT == kSpanBf16) {
          // matrices: tokens 0-7 | 8-15 (lanes 16 on) of columns 16 t | + 8
          const int row = (lane & 7) + 8 * (lane >> 4);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t a0, a1, a2, a3;
            ldmatrix_x4_trans(
                zs + row * (2 * RV) + sp_zchunk<RV>(row, 2 * t + ((lane >> 3) & 1)) * 16, a0, a1,
                a2, a3);
            pv(t, a0, a1, a2, a3);
          }
        } else {
          const int F = a.zsplit;
#pragma unroll
          for (int w = 0; w < RV / 32; ++w) {
            const int col = 32 * w + 4 * n;
            const int pitch = col < F ? F : RV - F;
            const uint32_t at = zs + (col < F ? col : UT * F + col - F) + 16 * v * pitch;
            uint32_t x[4], f[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = lds32(at + (2 * c + (e & 1) + 8 * (e >> 1)) * pitch);
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // token pairs of each column
              e4m3x4_to_f16(__byte_perm(x[2 * e], x[2 * e + 1], 0x5140), f[e][0], f[e][1]);
              e4m3x4_to_f16(__byte_perm(x[2 * e], x[2 * e + 1], 0x7362), f[e][2], f[e][3]);
            }
#pragma unroll
            for (int j = 0; j < 4; j += 2)
              pv(2 * w + j / 2, f[0][j], f[0][j + 1], f[1][j], f[1][j + 1]);
          }
        }
      }
    }

    // ---- the warps meet, two row tiles at a time
    float* part = a.partial + (size_t)(blockIdx.x + bg) * R * RS;
#pragma unroll
    for (int i0 = 0; i0 < NR; i0 += 2) {
      constexpr int MR = 8 * (NR < 2 ? NR : 2);
#pragma unroll
      for (int i = i0; i < i0 + 2 && i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
          float* row = meet + (size_t)(warp * MR + 8 * (i - i0) + 2 * c + e) * RS;
          if (n == 0) {
            row[RV] = m[i][e];
            row[RV + 1] = l[i][e];
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            row[16 * t + n] = acc[t][i][e];
            row[16 * t + 8 + n] = acc[t][i][2 + e];
          }
        }
      __syncthreads();
      const int rows = min(R - 8 * i0, MR);
      if (tid < kSpWarps * MR) {  // the warps' factors, the joint maximum and sum
        const int w = tid / MR, rr = tid - w * MR;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int x = 0; x < kSpWarps; ++x) M = fmaxf(M, meet[(size_t)(x * MR + rr) * RS + RV]);
        const float ref = M == -INFINITY ? 0.f : M;
        float* row = meet + (size_t)(w * MR + rr) * RS;
        row[RV + 2] = ex2(row[RV] - ref);
        if (w == 0) {
#pragma unroll
          for (int x = 0; x < kSpWarps; ++x) {
            const float* other = meet + (size_t)(x * MR + rr) * RS;
            L = fmaf(other[RV + 1], ex2(other[RV] - ref), L);
          }
          row[RV + 3] = L;
          if (!alone && rr < rows) {
            part[(8 * i0 + rr) * RS + RV] = M;
            part[(8 * i0 + rr) * RS + RV + 1] = L;
          }
        }
      }
      __syncthreads();
      for (int o = tid; o < rows * (RV / 4); o += kSpThreads) {
        const int rr = o / (RV / 4), at = 4 * (o - rr * (RV / 4)), r = 8 * i0 + rr;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSpWarps; ++w) {
          const float* row = meet + (size_t)(w * MR + rr) * RS;
          const float4 x = *reinterpret_cast<const float4*>(row + at);
          const float f = row[RV + 2];
          A.x = fmaf(x.x, f, A.x);
          A.y = fmaf(x.y, f, A.y);
          A.z = fmaf(x.z, f, A.z);
          A.w = fmaf(x.w, f, A.w);
        }
        if (alone) {
          const float L = meet[(size_t)rr * RS + RV + 3], inv = L > 0.f ? 1.f / L : 0.f;
          const int j = r >> a.logG, h = r & (a.G - 1);
          uint16_t* dst = a.out + (((size_t)b * a.n_tot + j) * a.Hq + g * a.G + h) * RV;
          const float v[4] = {A.x * inv, A.y * inv, A.z * inv, A.w * inv};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            dst[sp_col<FMT, RV>(at >> 3, (at & 7) + x)] = f_to_bf16(v[x]);
        } else {
          *reinterpret_cast<float4*>(part + r * RS + at) = A;
        }
      }
      __syncthreads();  // the meeting place is free again
    }
    seg = item_end;
  }
  // a wait has run out: no copy may still be on its way into this block's memory
  if (BULK && !landing)
    for (int k = max(0, k_next - NST); k < min(k_next, n_units); ++k)
      mbar_wait(bars + warp * NST + k % NST, (k / NST) & 1, a.status, kDrainNs);
}

// Joins the partials of the items that several CTAs share; rows of items
// without units are zero.  A thread joins one output: CTA (x, y) has outputs
// 256 y .. of (sequence, KV head) x, so the joins of a few items are not one
// CTA's chain of loads.  The lengths are read before the grid-dependency wait:
// the launch before this one let it in after its own wait, and does not write
// them.
template <int FMT, int RV, int UT>
__global__ void __launch_bounds__(kSpThreads) span_merge_kernel(SpanArgs a, int grid) {
  constexpr int RS = RV + kSpRowPad;
  __shared__ long long pre[257];
  span_scan<UT>(a, pre, false);
  const int bg = blockIdx.x, b = bg / a.Hkv, g = bg - b * a.Hkv, R = a.n_tot * a.G;
  const long long total = pre[a.B] * a.Hkv, u = pre[b + 1] - pre[b];
  const long long x0 = pre[b] * a.Hkv + g * u;
  int c0 = 0, c1 = -1;
  if (u > 0) {
    const int C = span_ctas(total, grid);
    c0 = span_cta_of(x0, total, C);
    c1 = span_cta_of(x0 + u - 1, total, C);
  }
  const int o = blockIdx.y * kSpThreads + threadIdx.x, r = o / RV, at = o - r * RV;
  pdl_wait();
  pdl_launch_dependents();
  if ((u > 0 && c0 == c1) || r >= R) return;  // written by its one CTA
  float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll 8
  for (int c = c0; c <= c1; ++c) {
    const float* s = a.partial + ((size_t)(c + bg) * R + r) * RS;
    const float mc = __ldcg(s + RV), lc = __ldcg(s + RV + 1), ac = __ldcg(s + at);
    const float mn = fmaxf(M, mc);
    const float f0 = M == -INFINITY ? 0.f : ex2(M - mn), f1 = mc == -INFINITY ? 0.f : ex2(mc - mn);
    L = fmaf(L, f0, lc * f1);
    A = fmaf(A, f0, ac * f1);
    M = mn;
  }
  const int j = r >> a.logG, h = r & (a.G - 1), col = sp_col<FMT, RV>(at >> 3, at & 7);
  a.out[(((size_t)b * a.n_tot + j) * a.Hq + g * a.G + h) * RV + col] =
      f_to_bf16(L > 0.f ? A / L : 0.f);
}

template <int FMT, int D, int RV, int NR, bool ONE = false>
cudaError_t launch_span_t(const SpanArgs& a, cudaStream_t st, bool pdl) {
  constexpr int UT = sp_unit<FMT, NR>();
  // Units of the longest context this call may meet; fewer CTAs when they do
  // not suffice for kSpMinUnits each.
  long long most = (long long)a.max_seq_len + UT;
  if (a.sel)
    most = (long long)a.top_k * a.S;
  else if (a.window > 0 && (long long)a.window + a.n_tot + a.sink + 3 * UT < most)
    most = (long long)a.window + a.n_tot + a.sink + 3 * UT;
  const long long units = (most + UT - 1) / UT * a.B * a.Hkv;
  long long grid = (long long)num_sms() * sp_ctas<FMT, NR>();
  if (grid > kSpanMaxCtas) grid = kSpanMaxCtas;
  if (grid > units / kSpMinUnits) grid = units / kSpMinUnits > 0 ? units / kSpMinUnits : 1;
  constexpr size_t smem = sp_smem<FMT, D, RV, NR>();
  cudaError_t e = cudaFuncSetAttribute(span_kernel<FMT, D, RV, NR, ONE>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_k(span_kernel<FMT, D, RV, NR, ONE>, dim3((unsigned)grid), dim3(kSpThreads), smem, st, pdl,
               a);
  if (e != cudaSuccess) return e;
  const int outs = a.n_tot * a.G * RV;
  return launch_k(span_merge_kernel<FMT, RV, UT>, dim3(a.B * a.Hkv, (outs + kSpThreads - 1) / kSpThreads),
                  dim3(kSpThreads), 0, st, pdl, a, (int)grid);
}

template <int FMT, int D, int RV, bool ONE>
cudaError_t launch_span_rows(const SpanArgs& a, cudaStream_t st, bool pdl) {
  switch ((a.n_tot * a.G + 7) / 8) {  // tiles of 8 rows
    case 1: return launch_span_t<FMT, D, RV, 1, ONE>(a, st, pdl);
    case 2: return launch_span_t<FMT, D, RV, 2, ONE>(a, st, pdl);
    case 3: return launch_span_t<FMT, D, RV, 3, ONE>(a, st, pdl);
    default:
      if constexpr (FMT == kSpanBf16 && RV > 64)
        return cudaErrorInvalidValue;  // not streamed
      else
        return launch_span_t<FMT, D, RV, 4, ONE>(a, st, pdl);
  }
}

template <int FMT, int D, bool ONE>
cudaError_t launch_span_width(const SpanArgs& a, cudaStream_t st, bool pdl) {
  switch (a.r_v) {
    case 32: return launch_span_rows<FMT, D, 32, ONE>(a, st, pdl);
    case 64: return launch_span_rows<FMT, D, 64, ONE>(a, st, pdl);
    case 96: return launch_span_rows<FMT, D, 96, ONE>(a, st, pdl);
    default: return launch_span_rows<FMT, D, 128, ONE>(a, st, pdl);
  }
}

template <int FMT, bool ONE = false>
cudaError_t launch_span_fmt(const SpanArgs& a, cudaStream_t st, bool pdl) {
  return a.d == 64 ? launch_span_width<FMT, 64, ONE>(a, st, pdl)
                   : launch_span_width<FMT, 128, ONE>(a, st, pdl);
}

}  // namespace
}  // namespace basiskv
