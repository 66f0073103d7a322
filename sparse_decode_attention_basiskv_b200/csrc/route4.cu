// Page scores over 4-bit caches.
//
//   score(page) = max over its live tokens t and the group's heads h of
//                 z_t . (P_K q_h) + e_t . (U_K^T q_h)
//
// with the folded queries in fp32 (fold_query_kernel).  One pass over the z
// and e pages: (r_v + r_k) * 9 / 16 bytes a token and KV head, so HBM bounds
// it, closely followed by the instructions that widen the codes (one
// conversion and one multiplication for two columns).
//
// The pages of all (sequence, KV head) items form one line, cut into equal
// contiguous runs, one a warp (a scan of the lengths finds them, so ragged
// batches load every SM alike).  A warp copies its 16-token units (cp.async)
// into its own ring kStages - 1 units ahead.  Tokens are the columns of
// mma.m16n8k16's B operand, as stored; the rows of A are the group's heads:
// rows 0-7 hold the f16 roundings of the folded queries, rows 8-15 their
// remainders, so one product gives fp32-accurate scores (22 significant
// bits; each head is first scaled by a power of two that puts its largest
// magnitude into [2^14, 2^15), divided out of the scores again).
#include "cache4.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "line_scan.cuh"

namespace basiskv {
namespace {

constexpr int kR4Threads = kLineMaxSeqs;  // a thread scans a sequence's length
constexpr int kR4Warps = kR4Threads / 32;
constexpr int kR4Stages = 4;
constexpr int kR4CtasPerSm = 2;

// Adds the products of one part (W columns at `codes`, its scales behind
// them) to the scores of tokens n (s0) and n + 8 (s1).  Lane c holds columns
// W / 4 * c .., 4 of them a k-step.
template <int W, int K0, int KS>
__device__ __forceinline__ void r4_part(uint32_t codes, int n, int c, const uint32_t (&qh)[KS][2],
                                        const uint32_t (&ql)[KS][2], float (&s0)[4],
                                        float (&s1)[4]) {
  const uint32_t sc = codes + 8 * W;
  if constexpr (W == 16) {
    // the lane's half of a 32-bit word
    uint32_t x[4], y[4];
    const int sh = 16 * (c & 1);
    q4_unpack8(lds32(codes + n * 8 + 4 * (c >> 1)) >> sh, x);
    q4_unpack8(lds32(codes + (n + 8) * 8 + 4 * (c >> 1)) >> sh, y);
    const uint32_t sx = q4_scale_x2(lds8(sc + n)), sy = q4_scale_x2(lds8(sc + n + 8));
    mma_f16_16816(s0, qh[K0][0], ql[K0][0], qh[K0][1], ql[K0][1], hmul2(x[0], sx), hmul2(x[1], sx));
    mma_f16_16816(s1, qh[K0][0], ql[K0][0], qh[K0][1], ql[K0][1], hmul2(y[0], sy), hmul2(y[1], sy));
  } else {
    uint32_t sx = 0, sy = 0;
#pragma unroll
    for (int w = 0; w < W / 32; ++w) {  // 8 columns
      uint32_t x[4], y[4];
      q4_unpack8(lds32(codes + n * (W / 2) + (W / 8) * c + 4 * w), x);
      q4_unpack8(lds32(codes + (n + 8) * (W / 2) + (W / 8) * c + 4 * w), y);
      if (W % 64 != 0 || w % 2 == 0) {
        const int blk = ((W / 4) * c + 8 * w) >> 4;
        sx = q4_scale_x2(lds8(sc + n * (W / 16) + blk));
        sy = q4_scale_x2(lds8(sc + (n + 8) * (W / 16) + blk));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = K0 + 2 * w + e;
        mma_f16_16816(s0, qh[k][0], ql[k][0], qh[k][1], ql[k][1], hmul2(x[2 * e], sx),
                      hmul2(x[2 * e + 1], sx));
        mma_f16_16816(s1, qh[k][0], ql[k][0], qh[k][1], ql[k][1], hmul2(y[2 * e], sy),
                      hmul2(y[2 * e + 1], sy));
      }
    }
  }
}

template <int RV, int RK>
__global__ void __launch_bounds__(kR4Threads, kR4CtasPerSm) route4_kernel(Route4Args a) {
  constexpr int W = RV + RK, KS = W / 16, UB = 9 * W, NST = kR4Stages;
  extern __shared__ __align__(16) uint8_t r4_smem[];
  __shared__ long long pre[257];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(r4_smem) + warp * NST * UB;
  const int logS = 31 - __clz(a.S), upp = a.S >> 4;  // units a page: 1 or 2

  pdl_wait();
  pdl_launch_dependents();
  line_scan(a.B, pre, [&](int b) -> long long {  // pages
    const int len = a.seq_lens[b];
    if (len >= 0 && len <= a.max_seq_len) return (len + a.S - 1) >> logS;
    if (blockIdx.x == 0) raise_status(a.status, BASISKV_DEV_BAD_LENGTH);
    return 0;
  });
  const long long total = pre[a.B] * a.Hkv;
  const long long W_all = (long long)gridDim.x * kR4Warps;
  const long long w_id = (long long)blockIdx.x * kR4Warps + warp;
  const long long end = total * (w_id + 1) / W_all;
  long long seg = total * w_id / W_all;
  int b = seg < end ? line_find(a.B, pre, a.Hkv, seg) : 0;
  while (seg < end) {
    while (pre[b + 1] * a.Hkv <= seg) ++b;
    const int P = (int)(pre[b + 1] - pre[b]);
    const int g = (int)((seg - pre[b] * a.Hkv) / P);
    const long long x0 = pre[b] * a.Hkv + (long long)g * P;
    const int p0 = (int)(seg - x0), p1 = (int)min((long long)P, end - x0);
    const int T = a.seq_lens[b];
    // ---- folded queries of head n: f16 hi and lo
    uint32_t qh[KS][2], ql[KS][2];
    float inv;
    {
      const float* qr = a.qt + ((size_t)b * a.Hq + g * a.G + (n < a.G ? n : 0)) * W;
      float f[KS][4], m = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int col = k < RV / 16 ? (RV / 4) * c + 4 * k : RV + (RK / 4) * c + 4 * (k - RV / 16);
        const float4 v = __ldg(reinterpret_cast<const float4*>(qr + col));
        f[k][0] = v.x, f[k][1] = v.y, f[k][2] = v.z, f[k][3] = v.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n >= a.G) f[k][e] = 0.f;
          m = fmaxf(m, fabsf(f[k][e]));
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int ex = m > 0.f ? (int)((__float_as_uint(m) >> 23) & 0xffu) - 126 : 15;
      const int sh = max(-126, min(126, 15 - ex));
      const float sc = __uint_as_float((uint32_t)(127 + sh) << 23);
      inv = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          split_f16x2(f[k][2 * e] * sc, f[k][2 * e + 1] * sc, qh[k][e], ql[k][e]);
    }
    // ---- pages p0 .. p1 - 1, unit u = page * upp + half
    const int count = (p1 - p0) * upp;
    int id = -1, id_base = 0;  // physical pages of 32 pages, one a lane
    auto fetch_ids = [&](int base) {
      id_base = base;
      id = -1;
      if (p0 + base + lane < p1) {
        id = __ldg(a.block_table + (size_t)b * a.max_pages + p0 + base + lane);
        if (id < 0 || id >= a.num_phys) {
          raise_status(a.status, BASISKV_DEV_BAD_PAGE);
          id = -1;
        }
      }
    };
    auto issue = [&](int u) {
      if (u < count) {
        const int p = u >> (upp - 1);
        if (p - id_base >= 32) fetch_ids(p);
        const int pp = __shfl_sync(0xffffffffu, id, p - id_base);
        if (pp >= 0) {
          const int row = upp == 2 && (u & 1) ? 16 : 0;
          const size_t tile = (size_t)pp * a.Hkv + g;
          const uint8_t* zt = a.Z + tile * q4_tile_bytes(a.S, RV);
          const uint8_t* et = a.E + tile * q4_tile_bytes(a.S, RK);
          const uint32_t st = ring + (u % NST) * UB;
#pragma unroll
          for (int x = 0; x < 9 * W / 16; x += 32) {
            const int i = x + lane;
            const uint8_t* src;
            if (i < RV / 2)
              src = zt + row * (RV / 2) + 16 * i;
            else if (i < RV / 16 * 9)
              src = zt + a.S * (RV / 2) + row * (RV / 16) + 16 * (i - RV / 2);
            else if (i < RV / 16 * 9 + RK / 2)
              src = et + row * (RK / 2) + 16 * (i - RV / 16 * 9);
            else
              src = et + a.S * (RK / 2) + row * (RK / 16) + 16 * (i - RV / 16 * 9 - RK / 2);
            if (i < 9 * W / 16) cp_async16_or_zero(st + 16 * i, src);
          }
        }
      }
      cp_async_commit();
    };
    fetch_ids(0);
    // a page's physical id is looked up again when it is scored
    int sid = id, sid_base = 0;
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(i);
    float best = -INFINITY;
    for (int u = 0; u < count; ++u) {
      __syncwarp();
      issue(u + NST - 1);
      cp_async_wait_group<NST - 1>();
      __syncwarp();
      const int p = u >> (upp - 1);
      if (p - sid_base >= 32) {
        sid_base = p;
        sid = -1;
        if (p0 + p + lane < p1) {
          sid = __ldg(a.block_table + (size_t)b * a.max_pages + p0 + p + lane);
          if (sid >= a.num_phys) sid = -1;
        }
      }
      const bool there = __shfl_sync(0xffffffffu, sid, p - sid_base) >= 0;
      const uint32_t st = ring + (u % NST) * UB;
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      r4_part<RV, 0, KS>(st, n, c, qh, ql, s0, s1);
      r4_part<RK, RV / 16, KS>(st + 9 * RV, n, c, qh, ql, s0, s1);
      const int t0 = ((p0 + p) << logS) + 16 * (u & (upp - 1));
      float v[4] = {s0[0] + s0[2], s0[1] + s0[3], s1[0] + s1[2], s1[1] + s1[3]};
      if (t0 + 16 > T) {  // the last page's tail
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t0 + 2 * c + (e & 1) + 8 * (e >> 1) >= T) v[e] = -INFINITY;
      }
      if (there && n < a.G)
        best = fmaxf(best, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) * inv);
      if ((u & (upp - 1)) == upp - 1) {
        best = warp_max(best);
        if (lane == 0) a.scores[((size_t)b * a.Hkv + g) * a.max_pages + p0 + p] = best;
        best = -INFINITY;
      }
    }
    cp_async_wait_all();
    __syncwarp();
    seg = x0 + p1;
  }
}

template <int RV, int RK>
cudaError_t launch_route4_t(const Route4Args& a, cudaStream_t st, bool pdl) {
  constexpr size_t smem = (size_t)kR4Warps * kR4Stages * 9 * (RV + RK);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(route4_kernel<RV, RK>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const long long pages = (long long)((a.max_seq_len + a.S - 1) / a.S) * a.B * a.Hkv;
  long long grid = (long long)num_sms() * kR4CtasPerSm;
  if (grid > pages / kR4Warps) grid = pages / kR4Warps > 0 ? pages / kR4Warps : 1;
  return launch_k(route4_kernel<RV, RK>, dim3((unsigned)grid), dim3(kR4Threads), smem, st, pdl, a);
}

template <int RV>
cudaError_t launch_route4_rk(const Route4Args& a, cudaStream_t st, bool pdl) {
  switch (a.r_k) {
    case 16: return launch_route4_t<RV, 16>(a, st, pdl);
    case 32: return launch_route4_t<RV, 32>(a, st, pdl);
    default: return launch_route4_t<RV, 64>(a, st, pdl);
  }
}

}  // namespace

cudaError_t launch_route4(const Route4Args& a, cudaStream_t st, bool pdl) {
  switch (a.r_v) {
    case 32: return launch_route4_rk<32>(a, st, pdl);
    case 64: return launch_route4_rk<64>(a, st, pdl);
    case 96: return launch_route4_rk<96>(a, st, pdl);
    default: return launch_route4_rk<128>(a, st, pdl);
  }
}

}  // namespace basiskv
