// Attention of a few query rows over a long span of one sequence's tokens,
// streamed once: a sliding window with sinks, the whole context, or the
// pages of a selection (instances: span_bf16.cu, span_e4m3.cu, span_q4.cu).
//
//   a[row] = sum_t p_t z_t,  p = softmax over the row's tokens of
//   (q . K_t) / sqrt(d)
//
// Rows: query token j and head h of KV head g make row j * G + h; up to 16
// rows (the M of mma.m16n8k16) share every Key and latent that is read.
// Bound by HBM: 2 (d + r_v) multiply-adds a row and (d + r_v) cached columns
// a token.
//
// Split: the unit of work is 16 tokens.  All units of all (sequence, KV head)
// items form one line in (b, g, unit) order, cut into equal contiguous runs,
// one a CTA, so that ragged lengths load every SM alike; each CTA finds its
// run from a scan of the sequences' lengths.  A CTA's 8 warps take every 8th
// unit of an item, keep their own running maximum, sum and accumulators, and
// meet in shared memory when the item's part of the run ends.  An item that
// lies in one CTA is written there; the others leave one partial a CTA, which
// span_merge_kernel joins (the second launch, scheduled early).
//
// Data path: each warp copies its units (cp.async, 16 bytes a lane) into its
// own ring of shared memory, kStages - 1 units ahead, and no other warp waits
// for it.  The Keys are the B operand of QK (columns = tokens, as stored), so
// the scores arrive with a row's tokens in the layout of the A operand of PV
// and need no transposition; the latents are PV's B operand.  With at most 8
// rows the upper half of PV's A operand holds the rounding remainders of the
// weights, so they count with 16 (bf16) or 22 (f16) significant bits at no
// cost.
//
// The running maximum moves only when a score passes it by 8 (a factor of
// 256 in the weights, far inside the range of f16): then the warp takes the
// rows' maxima over their lanes and rescales; all other units cost one vote.
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
constexpr float kSpSlack = 8.f;

// What one sequence contributes: its live length, and the units of one KV
// head (n_sink units of sink tokens, then the window's from lo_unit on).
struct SpanSeq {
  int T, n_sink, lo_unit, n;
};
__device__ __forceinline__ SpanSeq span_seq(const SpanArgs& a, int len) {
  SpanSeq s;
  s.T = len;
  const int last = len - a.n_tot + a.j0 + a.n_q - 1;  // position of the last row
  if (len <= 0 || len > a.max_seq_len || last < 0) {
    s.T = 0;
    s.n_sink = s.lo_unit = s.n = 0;
  } else if (a.sel) {
    s.n_sink = s.lo_unit = 0;
    s.n = a.top_k << (a.logS - 4);
  } else {
    const int p0 = max(0, last - a.n_q + 1);
    const int lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
    s.lo_unit = lo >> 4;
    s.n_sink = min((a.sink + 15) >> 4, s.lo_unit);
    s.n = s.n_sink + (last >> 4) - s.lo_unit + 1;
  }
  return s;
}

// pre[b] = units of one KV head of the sequences before b; pre[B] = all.
__device__ __forceinline__ void span_scan(const SpanArgs& a, long long* pre, bool report) {
  line_scan(a.B, pre, [&](int b) -> long long {
    const int len = a.seq_lens[b];
    if (report && (len < 0 || len > a.max_seq_len)) raise_status(a.status, BASISKV_DEV_BAD_LENGTH);
    return span_seq(a, len).n;
  });
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

// Bytes of one unit (16 tokens) in a warp's ring.
template <int FMT, int D, int RV>
constexpr int sp_unit_bytes() {
  return FMT == kSpanBf16 ? 32 * (D + RV) : (FMT == kSpanE4m3 ? 16 * (D + RV) : 9 * (D + RV));
}
// Ring depth: bf16 units are 3-8 KB and one CTA of 8 warps fills an SM's
// shared memory; the narrower formats run two CTAs.
template <int FMT>
constexpr int sp_stages() {
  return FMT == kSpanBf16 ? 3 : 4;
}
template <int FMT, int D, int RV, int NR>
constexpr size_t sp_smem() {
  const size_t ring = (size_t)kSpWarps * sp_stages<FMT>() * sp_unit_bytes<FMT, D, RV>();
  const size_t meet = (size_t)kSpWarps * 8 * NR * (RV + 2) * 4;
  return ring > meet ? ring : meet;
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

template <int FMT, int D, int RV, int NR>
__global__ void __launch_bounds__(kSpThreads, FMT == kSpanBf16 || NR == 2 ? 1 : 2)
    span_kernel(SpanArgs a) {
  constexpr int NT = RV / 8, KS = D / 16, NST = sp_stages<FMT>();
  constexpr int UB = sp_unit_bytes<FMT, D, RV>();
  constexpr int RS = RV + 2;
  extern __shared__ __align__(16) uint8_t sp_smem_raw[];
  __shared__ long long pre[257];
  __shared__ uint32_t ring_t0[kSpWarps][NST];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(sp_smem_raw) + warp * NST * UB;
  float* meet = reinterpret_cast<float*>(sp_smem_raw);  // [warp][row][RV + 2] after an item
  const int R = a.n_q * a.G;

  pdl_wait();
  pdl_launch_dependents();
  span_scan(a, pre, blockIdx.x == 0);
  const long long total = pre[a.B] * a.Hkv;
  const int C = span_ctas(total, gridDim.x);
  if ((int)blockIdx.x >= C) return;
  const long long c_end = total * (blockIdx.x + 1) / C;
  long long seg = total * blockIdx.x / C;
  int b = seg < c_end ? line_find(a.B, pre, a.Hkv, seg) : 0;
  while (seg < c_end) {
    while (pre[b + 1] * a.Hkv <= seg) ++b;
    const SpanSeq sq = span_seq(a, a.seq_lens[b]);
    const int g = (int)((seg - pre[b] * a.Hkv) / sq.n);
    const long long x0 = pre[b] * a.Hkv + (long long)g * sq.n;
    const int u_begin = (int)(seg - x0);
    const int u_end = (int)min((long long)sq.n, c_end - x0);
    const int bg = b * a.Hkv + g;
    const int T = sq.T;
    // row positions: query token j sits at pos0 + j
    const int pos0 = T - a.n_tot + a.j0;
    const int p_last = pos0 + a.n_q - 1;
    const int lo_first = a.window > 0 ? max(0, max(pos0, 0) - a.window + 1) : 0;
    const int lo_last = a.window > 0 ? max(0, p_last - a.window + 1) : 0;
    const int live_end = p_last + 1;  // no row sees a token from here on

    // ---- queries: rows n and n + 8
    int pos[NR], lo[NR];
    uint32_t qa[KS][NR][2];
    float sl[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = n + 8 * i;
      const int j = r / a.G, h = r - j * a.G;
      const bool ok = r < R;
      pos[i] = ok ? pos0 + j : -1;
      lo[i] = a.window > 0 ? max(0, pos[i] - a.window + 1) : 0;
      const uint16_t* qr =
          a.q + (((size_t)b * a.n_tot + a.j0 + (ok ? j : 0)) * a.Hq + g * a.G + (ok ? h : 0)) * D;
      sl[i] = a.scale_log2;
      if constexpr (FMT == kSpanBf16) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qa[k][i][e] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * k + 8 * e + 2 * c))
                             : 0u;
      } else {
        // k-step k of the lane's columns: 4 consecutive ones (2 pairs)
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int col = FMT == kSpanE4m3 ? 64 * (k >> 2) + 16 * c + 4 * (k & 3)
                                           : (D / 4) * c + 4 * k;
          const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(qr + col)) : make_uint2(0u, 0u);
          qa[k][i][0] = w.x;
          qa[k][i][1] = w.y;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = bf16x2_to_f2(qa[k][i][e]);
            m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int ex = m > 0.f ? (int)((__float_as_uint(m) >> 23) & 0xffu) - 126 : 15;
        const int sh = max(-126, min(126, 15 - ex));
        const float sc = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = bf16x2_to_f2(qa[k][i][e]);
            const __half2 hh = __floats2half2_rn(f.x * sc, f.y * sc);
            qa[k][i][e] = *reinterpret_cast<const uint32_t*>(&hh);
          }
        sl[i] *= __uint_as_float((uint32_t)(127 - sh) << 23);
      }
    }

    float m[NR], l[NR], acc[NT][4];
#pragma unroll
    for (int i = 0; i < NR; ++i) m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;

    // ---- the warp's units: u_begin + warp + 8 i
    const int u_first = u_begin + warp;
    const int count = u_first < u_end ? (u_end - u_first + kSpWarps - 1) / kSpWarps : 0;
    // Ids of 32 units ahead, one a lane: the first token, and the tile row of
    // tokens 0-7 and 8-15 of the unit (-1: nothing to read there).
    int id_t0 = 0, id_ra = -1, id_rb = -1, id_base = 0;
    auto tile_row = [&](int t) -> int {
      if (t >= live_end) return -1;
      const int p = t >> a.logS;
      const int pp = p < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + p) : -1;
      if (pp < 0 || pp >= a.num_phys) {
        raise_status(a.status, BASISKV_DEV_BAD_PAGE);
        return -1;
      }
      return ((pp * a.Hkv + g) << a.logS) + (t & (a.S - 1));
    };
    auto fetch_ids = [&](int base) {
      id_base = base;
      const int i = base + lane;
      id_ra = id_rb = -1;
      id_t0 = 0;
      if (i >= count) return;
      const int u = u_first + kSpWarps * i;
      if (a.sel) {
        const int lp = __ldg(a.sel + (size_t)bg * a.top_k + (u >> (a.logS - 4)));
        if (lp < 0) return;
        if (lp >= a.max_pages) {
          raise_status(a.status, BASISKV_DEV_BAD_PAGE);
          return;
        }
        id_t0 = (lp << a.logS) + 16 * (u & ((a.S >> 4) - 1));
      } else {
        id_t0 = 16 * (u < sq.n_sink ? u : sq.lo_unit + u - sq.n_sink);
      }
      id_ra = tile_row(id_t0);
      if (a.S >= 16)
        id_rb = id_ra < 0 || id_t0 + 8 >= live_end ? -1 : id_ra + 8;
      else
        id_rb = tile_row(id_t0 + 8);
    };
    // Whether some row of this launch sees token t.
    auto seen = [&](int t) { return t < live_end && (t >= lo_first || t < a.sink); };

    auto issue = [&](int i) {
      if (i < count) {
        if (i - id_base >= 32) fetch_ids(i);
        const int src = i - id_base;
        const int t0 = __shfl_sync(0xffffffffu, id_t0, src);
        const int ra = __shfl_sync(0xffffffffu, id_ra, src);
        const int rb = __shfl_sync(0xffffffffu, id_rb, src);
        const int slot = i % NST;
        const uint32_t st = ring + slot * UB;
        // positions have 30 bits; above them, which halves are there
        if (lane == 0)
          ring_t0[warp][slot] =
              (uint32_t)t0 | (ra >= 0 ? 1u << 30 : 0u) | (rb >= 0 ? 1u << 31 : 0u);
        if (ra >= 0 || rb >= 0) {
          if constexpr (FMT == kSpanQ4) {
            // codes and scales of 16 rows, contiguous each
            const int tile = ra >> a.logS, row = ra & (a.S - 1);
            const uint8_t* kt = a.K + (size_t)tile * q4_tile_bytes(a.S, D);
            const uint8_t* zt = a.Z + (size_t)tile * q4_tile_bytes(a.S, RV);
#pragma unroll
            for (int x = 0; x < D / 2; x += 32)
              cp_async16_or_zero(st + 16 * (x + lane), kt + row * (D / 2) + 16 * (x + lane), true);
#pragma unroll
            for (int x = 0; x < RV / 2; x += 32)
              if (RV / 2 - x >= 32 || lane < RV / 2 - x)
                cp_async16_or_zero(st + 9 * D + 16 * (x + lane),
                                   zt + row * (RV / 2) + 16 * (x + lane), true);
            if (lane < D / 16)
              cp_async16_or_zero(st + 8 * D + 16 * lane,
                                 kt + a.S * (D / 2) + row * (D / 16) + 16 * lane, true);
            else if (lane < D / 16 + RV / 16)
              cp_async16_or_zero(st + 9 * D + 8 * RV + 16 * (lane - D / 16),
                                 zt + a.S * (RV / 2) + row * (RV / 16) + 16 * (lane - D / 16),
                                 true);
          } else {
            constexpr int EB = FMT == kSpanBf16 ? 2 : 1;  // bytes a column
            constexpr int KC = D * EB / 16, ZC = RV * EB / 16;
            const bool whole = t0 + 15 < live_end && (t0 >= lo_first || t0 + 15 < a.sink);
#pragma unroll
            for (int x = 0; x < 16 * KC; x += 32) {
              const int i2 = x + lane, r = i2 / KC, ch = i2 % KC;
              const int tr = r < 8 ? ra + r : rb + r - 8;
              const bool ok = (r < 8 ? ra >= 0 : rb >= 0) && (whole || seen(t0 + r));
              // chunks of a row are rotated within shared memory so that the
              // lanes' reads fall into different banks
              const int sw = FMT == kSpanBf16 ? ch ^ (r & 7) : (D == 128 ? ch ^ ((r & 1) << 2) : ch);
              cp_async16_or_zero(st + (r * KC + sw) * 16,
                                 a.K + (ok ? ((size_t)tr * D * EB + ch * 16) : 0), ok);
            }
#pragma unroll
            for (int x = 0; x < 16 * ZC; x += 32) {
              const int i2 = x + lane, r = i2 / ZC, ch = i2 % ZC;
              const int tr = r < 8 ? ra + r : rb + r - 8;
              const bool ok = (r < 8 ? ra >= 0 : rb >= 0) && (whole || seen(t0 + r));
              size_t off = 0;
              if (ok) {
                const int tile = tr >> a.logS, row = tr & (a.S - 1);
                off = ((size_t)tile * a.S * RV +
                       split_off(row, ch * (16 / EB), a.S, RV, a.zsplit)) * EB;
              }
              const int sw = FMT == kSpanBf16 ? (RV == 32 ? ch ^ ((r >> 1) & 3) :
                                                 RV == 96 ? (ch < 8 ? ch ^ (r & 7)
                                                                    : 8 + ((ch ^ (r >> 1)) & 3))
                                                          : ch ^ (r & 7))
                                              : ch;
              cp_async16_or_zero(st + 16 * D * EB + (r * ZC + sw) * 16, a.Z + off, ok);
            }
          }
        }
      }
      cp_async_commit();
    };

    if (count > 0) fetch_ids(0);
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(i);
    for (int it = 0; it < count; ++it) {
      __syncwarp();  // every lane is done with the slot that is filled next
      issue(it + NST - 1);
      cp_async_wait_group<NST - 1>();
      __syncwarp();  // the unit's copies by all lanes have landed
      const int slot = it % NST;
      const uint32_t tag = ring_t0[warp][slot];
      if (tag < 1u << 30) continue;  // nothing to read there
      const int t0 = (int)(tag & 0x3fffffffu);
      const uint32_t ks = ring + slot * UB;
      constexpr int ZB = FMT == kSpanBf16 ? 32 * D : (FMT == kSpanE4m3 ? 16 * D : 9 * D);
      const uint32_t zs = ks + ZB;
      // ---- scores: s[e] of rows n (and n + 8), tokens 2c, 2c + 1 (tile 0), + 8 (tile 1)
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (FMT == kSpanBf16) {
        const int mi = lane >> 3, row = (lane & 7) + 8 * (mi >> 1);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int ch = (2 * k + (mi & 1)) ^ (row & 7);
          uint32_t b0, b1, b2, b3;
          ldmatrix_x4(ks + row * (2 * D) + ch * 16, b0, b1, b2, b3);
          mma_bf16_16816(s0, qa[k][0][0], NR == 2 ? qa[k][NR - 1][0] : 0u, qa[k][0][1],
                         NR == 2 ? qa[k][NR - 1][1] : 0u, b0, b1);
          mma_bf16_16816(s1, qa[k][0][0], NR == 2 ? qa[k][NR - 1][0] : 0u, qa[k][0][1],
                         NR == 2 ? qa[k][NR - 1][1] : 0u, b2, b3);
        }
      } else if constexpr (FMT == kSpanE4m3) {
#pragma unroll
        for (int k4 = 0; k4 < KS / 4; ++k4) {
          // 16 columns of tokens n and n + 8
          const int ch = c + 4 * k4;
          const uint4 x = lds128(ks + n * D + (D == 128 ? ch ^ ((n & 1) << 2) : ch) * 16);
          const uint4 y = lds128(ks + (n + 8) * D + (D == 128 ? ch ^ ((n & 1) << 2) : ch) * 16);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t b0, b1, b2, b3;
            e4m3x4_to_f16(xw[w], b0, b1);
            e4m3x4_to_f16(yw[w], b2, b3);
            const int k = 4 * k4 + w;
            mma_f16_16816(s0, qa[k][0][0], NR == 2 ? qa[k][NR - 1][0] : 0u, qa[k][0][1],
                          NR == 2 ? qa[k][NR - 1][1] : 0u, b0, b1);
            mma_f16_16816(s1, qa[k][0][0], NR == 2 ? qa[k][NR - 1][0] : 0u, qa[k][0][1],
                          NR == 2 ? qa[k][NR - 1][1] : 0u, b2, b3);
          }
        }
      } else {
        // D / 4 columns of tokens n and n + 8: D / 8 bytes, one scale per 16
        uint32_t xw[D / 32], yw[D / 32], sx[D / 64], sy[D / 64];
        if constexpr (D == 128) {
          const uint4 x = lds128(ks + n * 64 + 16 * c), y = lds128(ks + (n + 8) * 64 + 16 * c);
          xw[0] = x.x, xw[1] = x.y, xw[2] = x.z, xw[3] = x.w;
          yw[0] = y.x, yw[1] = y.y, yw[2] = y.z, yw[3] = y.w;
          const uint32_t u = lds16(ks + 8 * D + n * 8 + 2 * c);
          const uint32_t v = lds16(ks + 8 * D + (n + 8) * 8 + 2 * c);
          sx[0] = q4_scale_x2(u & 255u), sx[D / 64 - 1] = q4_scale_x2(u >> 8);
          sy[0] = q4_scale_x2(v & 255u), sy[D / 64 - 1] = q4_scale_x2(v >> 8);
        } else {
          const uint2 x = lds64(ks + n * 32 + 8 * c), y = lds64(ks + (n + 8) * 32 + 8 * c);
          xw[0] = x.x, xw[1] = x.y;
          yw[0] = y.x, yw[1] = y.y;
          sx[0] = q4_scale_x2(lds8(ks + 8 * D + n * 4 + c));
          sy[0] = q4_scale_x2(lds8(ks + 8 * D + (n + 8) * 4 + c));
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t x[4], y[4];
          q4_unpack8(xw[w], x);
          q4_unpack8(yw[w], y);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 2 * w + e;
            mma_f16_16816(s0, qa[k][0][0], NR == 2 ? qa[k][NR - 1][0] : 0u, qa[k][0][1],
                          NR == 2 ? qa[k][NR - 1][1] : 0u, hmul2(x[2 * e], sx[w / 2]),
                          hmul2(x[2 * e + 1], sx[w / 2]));
            mma_f16_16816(s1, qa[k][0][0], NR == 2 ? qa[k][NR - 1][0] : 0u, qa[k][0][1],
                          NR == 2 ? qa[k][NR - 1][1] : 0u, hmul2(y[2 * e], sy[w / 2]),
                          hmul2(y[2 * e + 1], sy[w / 2]));
          }
        }
      }
      // ---- softmax weights
      const bool half[2] = {(tag >> 30 & 1u) != 0, (tag >> 31) != 0};
      const bool all_seen = tag >> 30 == 3u && t0 + 15 <= pos0 && (t0 >= lo_last || t0 + 15 < a.sink);
      const int ta = t0 + 2 * c, tb = ta + 1, tc = ta + 8, td = ta + 9;
      float x[NR][4];
      bool grow = false;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        x[i][0] = s0[2 * i] * sl[i];
        x[i][1] = s0[2 * i + 1] * sl[i];
        x[i][2] = s1[2 * i] * sl[i];
        x[i][3] = s1[2 * i + 1] * sl[i];
        if (!all_seen) {
          const int tt[4] = {ta, tb, tc, td};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(half[e >> 1] && tt[e] <= pos[i] && (tt[e] >= lo[i] || tt[e] < a.sink))) x[i][e] = -INFINITY;
        }
        grow |= fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])) > m[i] + kSpSlack;
      }
      if (__any_sync(0xffffffffu, grow)) {
        float f[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          float mx = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[i], mx);
          f[i] = mn == -INFINITY ? 1.f : ex2(m[i] - mn);
          m[i] = mn;
          l[i] *= f[i];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[t][0] *= f[0];
          acc[t][1] *= f[0];
          acc[t][2] *= f[NR - 1];
          acc[t][3] *= f[NR - 1];
        }
      }
      uint32_t pa[4];  // A operand of PV: rows n | n + 8, tokens 2c.. | + 8
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float base = m[i] == -INFINITY ? 0.f : m[i];
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ex2(x[i][e] - base);
        l[i] += (p[0] + p[1]) + (p[2] + p[3]);
        uint32_t h0, h1, e0, e1;
        if constexpr (FMT == kSpanBf16) {
          split_bf16x2(p[0], p[1], h0, e0);
          split_bf16x2(p[2], p[3], h1, e1);
        } else {
          split_f16x2(p[0], p[1], h0, e0);
          split_f16x2(p[2], p[3], h1, e1);
        }
        pa[i] = h0;
        pa[2 + i] = h1;
        if (NR == 1) {
          pa[1] = e0;
          pa[3] = e1;
        }
      }
      // ---- latents: tokens 2c, 2c + 1 (+ 8) of the lane's columns
      if constexpr (FMT == kSpanBf16) {
        const int mi = lane >> 3, row = (lane & 7) + 8 * (mi & 1);
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          const int ch = t + (mi >> 1);
          const int sw = RV == 32 ? ch ^ ((row >> 1) & 3)
                         : RV == 96 ? (ch < 8 ? ch ^ (row & 7) : 8 + ((ch ^ (row >> 1)) & 3))
                                    : ch ^ (row & 7);
          uint32_t b0, b1, b2, b3;
          ldmatrix_x4_trans(zs + row * (2 * RV) + sw * 16, b0, b1, b2, b3);
          mma_bf16_16816(acc[t], pa[0], pa[1], pa[2], pa[3], b0, b1);
          mma_bf16_16816(acc[t + 1], pa[0], pa[1], pa[2], pa[3], b2, b3);
        }
      } else if constexpr (FMT == kSpanE4m3) {
#pragma unroll
        for (int w = 0; w < RV / 32; ++w) {
          uint32_t v[4], f[2][4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = lds32(zs + (2 * c + (e & 1) + 8 * (e >> 1)) * RV + 32 * w + 4 * n);
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // token pairs of each column
            e4m3x4_to_f16(__byte_perm(v[2 * e], v[2 * e + 1], 0x5140), f[e][0], f[e][1]);
            e4m3x4_to_f16(__byte_perm(v[2 * e], v[2 * e + 1], 0x7362), f[e][2], f[e][3]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16_16816(acc[4 * w + j], pa[0], pa[1], pa[2], pa[3], f[0][j], f[1][j]);
        }
      } else {
        const uint32_t zsc = zs + 8 * RV;
        const bool live[4] = {all_seen || seen(ta), all_seen || seen(tb), all_seen || seen(tc),
                              all_seen || seen(td)};
        // scale pairs of block k for tokens (2c, 2c + 1) and (+ 8); 0 for a
        // token that no row sees, whose scale byte may be anything
        auto scales = [&](int k, uint32_t& s01, uint32_t& s89) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = lds8(zsc + (2 * c + (e & 1) + 8 * (e >> 1)) * (RV / 16) + k);
            if (!live[e]) v[e] = 0;
          }
          s01 = (v[0] << 7) | (v[1] << 23);
          s89 = (v[2] << 7) | (v[3] << 23);
        };
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
          uint32_t v[4], f0[8], f1[8], s01, s89;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = lds32(zs + (2 * c + (e & 1) + 8 * (e >> 1)) * (RV / 2) + 32 * w + 4 * n);
          pairs(v[0], v[1], f0);
          pairs(v[2], v[3], f1);
          scales(4 * w + (n >> 1), s01, s89);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_f16_16816(acc[8 * w + j], pa[0], pa[1], pa[2], pa[3], hmul2(f0[j], s01),
                          hmul2(f1[j], s89));
        }
        if constexpr (RV % 64 != 0) {
          constexpr int W0 = RV / 64;
          uint32_t v[4], f0[8], f1[8], s01, s89;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = lds16(zs + (2 * c + (e & 1) + 8 * (e >> 1)) * (RV / 2) + 32 * W0 + 2 * n);
          pairs(v[0], v[1], f0);
          pairs(v[2], v[3], f1);
          scales(4 * W0 + (n >> 2), s01, s89);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16_16816(acc[8 * W0 + j], pa[0], pa[1], pa[2], pa[3], hmul2(f0[j], s01),
                          hmul2(f1[j], s89));
        }
      }
    }
    cp_async_wait_all();
    __syncthreads();  // the rings become the meeting place

    // ---- the warps meet
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      float* row = meet + (size_t)(warp * 8 * NR + n + 8 * i) * RS;
      if (c == 0) {
        row[0] = m[i];
        row[1] = l[i];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          row[2 + sp_col<FMT, RV>(t, 2 * c + e)] =
              NR == 1 ? acc[t][e] + acc[t][2 + e] : acc[t][2 * i + e];
    }
    __syncthreads();
    const bool alone = u_begin == 0 && u_end == sq.n;  // the whole item is here
    float* slot = a.partial + (size_t)(blockIdx.x + bg) * R * RS;
    for (int o = tid; o < R * RV; o += kSpThreads) {
      const int r = o / RV, col = o - r * RV;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kSpWarps; ++w) M = fmaxf(M, meet[(size_t)(w * 8 * NR + r) * RS]);
      float L = 0.f, A = 0.f;
#pragma unroll
      for (int w = 0; w < kSpWarps; ++w) {
        const float* row = meet + (size_t)(w * 8 * NR + r) * RS;
        const float f = row[0] == -INFINITY ? 0.f : ex2(row[0] - M);
        L = fmaf(row[1], f, L);
        A = fmaf(row[2 + col], f, A);
      }
      if (alone) {
        const int j = r / a.G, h = r - j * a.G;
        a.out[(((size_t)b * a.n_tot + a.j0 + j) * a.Hq + g * a.G + h) * RV + col] =
            f_to_bf16(L > 0.f ? A / L : 0.f);
      } else {
        slot[r * RS + 2 + col] = A;
        if (col == 0) {
          slot[r * RS] = M;
          slot[r * RS + 1] = L;
        }
      }
    }
    __syncthreads();  // the meeting place becomes rings again
    seg = x0 + u_end;
  }
}

// Joins the partials of the items that several CTAs share; rows of items
// without units are zero.  One CTA per (sequence, KV head).
template <int RV>
__global__ void __launch_bounds__(kSpThreads) span_merge_kernel(SpanArgs a, int grid) {
  constexpr int RS = RV + 2;
  __shared__ long long pre[257];
  pdl_wait();
  pdl_launch_dependents();
  span_scan(a, pre, false);
  const int bg = blockIdx.x, b = bg / a.Hkv, g = bg - b * a.Hkv, R = a.n_q * a.G;
  const long long total = pre[a.B] * a.Hkv, u = pre[b + 1] - pre[b];
  const long long x0 = pre[b] * a.Hkv + g * u;
  int c0 = 0, c1 = -1;
  if (u > 0) {
    const int C = span_ctas(total, grid);
    c0 = span_cta_of(x0, total, C);
    c1 = span_cta_of(x0 + u - 1, total, C);
    if (c0 == c1) return;  // written by its one CTA
  }
  for (int o = threadIdx.x; o < R * RV; o += kSpThreads) {
    const int r = o / RV, col = o - r * RV;
    float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll 8
    for (int c = c0; c <= c1; ++c) {
      const float* s = a.partial + ((size_t)(c + bg) * R + r) * RS;
      const float mc = __ldcg(s), lc = __ldcg(s + 1), ac = __ldcg(s + 2 + col);
      if (mc == -INFINITY) continue;
      const float mn = fmaxf(M, mc);
      const float f0 = M == -INFINITY ? 0.f : ex2(M - mn), f1 = ex2(mc - mn);
      L = fmaf(L, f0, lc * f1);
      A = fmaf(A, f0, ac * f1);
      M = mn;
    }
    const int j = r / a.G, h = r - j * a.G;
    a.out[(((size_t)b * a.n_tot + a.j0 + j) * a.Hq + g * a.G + h) * RV + col] =
        f_to_bf16(L > 0.f ? A / L : 0.f);
  }
}

template <int FMT, int D, int RV, int NR>
cudaError_t launch_span_t(const SpanArgs& a, cudaStream_t st, bool pdl) {
  // Units of the longest context this call may meet; fewer CTAs when they do
  // not suffice for kSpMinUnits each.
  const long long span = a.sel ? (long long)a.top_k * a.S
                         : a.window > 0 ? (long long)a.window + a.n_q + a.sink + 48
                                        : (long long)a.max_seq_len + 16;
  const long long most = span < (long long)a.max_seq_len + 16 || a.sel
                             ? span : (long long)a.max_seq_len + 16;
  const long long units = (most + 15) / 16 * a.B * a.Hkv;
  long long grid = (long long)num_sms() * (FMT == kSpanBf16 || NR == 2 ? 1 : 2);
  if (grid > kSpanMaxCtas) grid = kSpanMaxCtas;
  if (grid > units / kSpMinUnits) grid = units / kSpMinUnits > 0 ? units / kSpMinUnits : 1;
  constexpr size_t smem = sp_smem<FMT, D, RV, NR>();
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(span_kernel<FMT, D, RV, NR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch_k(span_kernel<FMT, D, RV, NR>, dim3((unsigned)grid), dim3(kSpThreads),
                           smem, st, pdl, a);
  if (e != cudaSuccess) return e;
  return launch_k(span_merge_kernel<RV>, dim3(a.B * a.Hkv), dim3(kSpThreads), 0, st, pdl, a,
                  (int)grid);
}

template <int FMT>
cudaError_t launch_span_fmt(const SpanArgs& a, cudaStream_t st, bool pdl) {
  const bool two = a.n_q * a.G > 8;
#define BKV_SPAN_RV(DD)                                                       \
  switch (a.r_v) {                                                            \
    case 32:                                                                  \
      return two ? launch_span_t<FMT, DD, 32, 2>(a, st, pdl)                  \
                 : launch_span_t<FMT, DD, 32, 1>(a, st, pdl);                 \
    case 64:                                                                  \
      return two ? launch_span_t<FMT, DD, 64, 2>(a, st, pdl)                  \
                 : launch_span_t<FMT, DD, 64, 1>(a, st, pdl);                 \
    case 96:                                                                  \
      return two ? launch_span_t<FMT, DD, 96, 2>(a, st, pdl)                  \
                 : launch_span_t<FMT, DD, 96, 1>(a, st, pdl);                 \
    default:                                                                  \
      return two ? launch_span_t<FMT, DD, 128, 2>(a, st, pdl)                 \
                 : launch_span_t<FMT, DD, 128, 1>(a, st, pdl);                \
  }
  if (a.d == 64) {
    BKV_SPAN_RV(64)
  } else {
    BKV_SPAN_RV(128)
  }
#undef BKV_SPAN_RV
}

}  // namespace
}  // namespace basiskv
