// Page scores over 4-bit caches.
//
//   score(page) = max over its live tokens t and the group's heads h of
//                 z_t . (P_K q_h) + e_t . (U_K^T q_h)
//
// with the folded queries in fp32 (fold_query_kernel).  One pass over the z
// and e pages: (r_v + r_k) * 9 / 16 bytes a token and KV head, and a conversion
// and a multiplication for two columns to widen the codes.
//
// The units (32 tokens: one page of 32 or two of 16) of all (sequence, KV
// head) items form one line, cut into equal contiguous runs, one a warp (a
// scan of the lengths finds them, so ragged batches load every SM alike).  A
// warp brings its units into its own ring: a tile is one contiguous piece for the
// copy engine, and the lanes that looked up the next units hand over half a ring
// of them at a time, side by side.  Tokens are the
// rows of mma.m16n8k16's A operand, as stored; B holds four heads, the f16
// roundings of their folded queries in the even columns and the remainders in
// the odd ones, so a lane's two sums give one fp32-accurate score (22
// significant bits; each head is first scaled by a power of two that puts its
// largest magnitude into [2^14, 2^15), divided out of the scores again).
//
// Measured: 16 x 32K tokens, 8 KV heads, r_v 64, r_k 32 (228 MB): 64 us with the
// folding of the queries, 3.6 TB/s (69 with the selection behind it).  Neither HBM
// nor the issue slots (68%) are full: with the conversions taken out it takes 62
// us, with the multiplications 57, with both 55, so what is left is the latency of
// a unit's chain of loads and products.  Rings with one unit requested at a time
// took 70 us, a fourth of the warps as loaders for the others 101 us, two CTAs an SM
// instead of three 65 us.
#include "cache4.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "line_scan.cuh"

namespace basiskv {
namespace {

constexpr int kR4Threads = kLineMaxSeqs;  // a thread scans a sequence's length
constexpr int kR4Warps = kR4Threads / 32;
constexpr int kR4Unit = 32;
// CTAs an SM: three where the registers (one group of heads, at most 96 columns)
// and the ring allow.
template <int W, int NJ>
constexpr int r4_ctas() {
  return NJ == 1 && W <= 96 ? 3 : 2;
}

// Ring depth: 8 units where shared memory holds them, else 4.
template <int W, int NJ>
constexpr int r4_stages() {
  const int n = (226 / r4_ctas<W, NJ>() - 5) * 1024 / (kR4Warps * 18 * W);
  return n >= 8 ? 8 : (n >= 4 ? 4 : 2);
}

// The warp's maximum.
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Adds the products of one part (W columns, 16 tokens whose codes start at
// `codes` and scales at `sc`) to the scores of tokens n and n + 8.  Lane c
// holds columns W / 4 * c .., 4 of them a k-step.
template <int W, int K0, int KS, int NJ>
__device__ __forceinline__ void r4_part(uint32_t codes, uint32_t sc, int n, int c,
                                        const uint32_t (&qb)[KS][NJ][2], float (&s)[NJ][4]) {
  auto step = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) mma_f16_16816(s[j], a0, a1, a2, a3, qb[k][j][0], qb[k][j][1]);
  };
  const uint32_t row = codes + n * (W / 2) + (W / 8) * c;
  if constexpr (W == 16) {
    // the lane's half of a 32-bit word
    uint32_t x[4], y[4];
    const uint32_t at = codes + n * 8 + 4 * (c >> 1);
    const int sh = 16 * (c & 1);
    q4_unpack8(lds32(at) >> sh, x);
    q4_unpack8(lds32(at + 64) >> sh, y);
    const uint32_t sx = q4_scale_x2(lds8(sc + n)), sy = q4_scale_x2(lds8(sc + n + 8));
    step(K0, hmul2(x[0], sx), hmul2(y[0], sy), hmul2(x[1], sx), hmul2(y[1], sy));
  } else {
    uint32_t xw[W / 32], yw[W / 32], sx = 0, sy = 0;
    if constexpr (W == 128) {
      const uint4 x = lds128(row), y = lds128(row + 8 * (W / 2));
      xw[0] = x.x, xw[1] = x.y, xw[2] = x.z, xw[3] = x.w;
      yw[0] = y.x, yw[1] = y.y, yw[2] = y.z, yw[3] = y.w;
    } else if constexpr (W == 64) {
      const uint2 x = lds64(row), y = lds64(row + 8 * (W / 2));
      xw[0] = x.x, xw[1] = x.y;
      yw[0] = y.x, yw[1] = y.y;
    } else {
#pragma unroll
      for (int w = 0; w < W / 32; ++w) {
        xw[w] = lds32(row + 4 * w);
        yw[w] = lds32(row + 8 * (W / 2) + 4 * w);
      }
    }
#pragma unroll
    for (int w = 0; w < W / 32; ++w) {  // 8 columns
      uint32_t x[4], y[4];
      q4_unpack8(xw[w], x);
      q4_unpack8(yw[w], y);
      if (W % 64 != 0 || w % 2 == 0) {
        const int blk = ((W / 4) * c + 8 * w) >> 4;
        sx = q4_scale_x2(lds8(sc + n * (W / 16) + blk));
        sy = q4_scale_x2(lds8(sc + (n + 8) * (W / 16) + blk));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        step(K0 + 2 * w + e, hmul2(x[2 * e], sx), hmul2(y[2 * e], sy), hmul2(x[2 * e + 1], sx),
             hmul2(y[2 * e + 1], sy));
    }
  }
}

// NJ: groups of four heads (1 for G <= 4, 2 for G = 8).  ONE: pages of 32.
template <int RV, int RK, int NJ, bool ONE>
__global__ void __launch_bounds__(kR4Threads, r4_ctas<RV + RK, NJ>())
    route4_kernel(Route4Args a) {
  constexpr int W = RV + RK, KS = W / 16, UB = 18 * W, NST = r4_stages<W, NJ>(), NB = NST / 2;
  constexpr int PP = ONE ? 1 : 2;  // pages a unit
  extern __shared__ __align__(128) uint8_t r4_smem[];
  __shared__ long long pre[257];
  __shared__ int lens[kLineMaxSeqs];
  __shared__ uint64_t bars[kR4Warps * NST];
  __shared__ uint2 tags[kR4Warps][NST];  // the unit's pages: 1 there, 0 missing
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(r4_smem) + warp * NST * UB;
  const uint32_t bar = smem_u32(bars + warp * NST);

  if (tid < kR4Warps * NST) mbar_init(bars + tid, 1);
  fence_barrier_init();
  pdl_wait();
  pdl_launch_dependents();
  auto units_of = [&](int len) {
    return len >= 0 && len <= a.max_seq_len ? (len + kR4Unit - 1) / kR4Unit : 0;
  };
  line_scan(a.B, pre, [&](int b) -> long long {
    const int len = lens[b] = a.seq_lens[b];
    if (blockIdx.x == 0 && (len < 0 || len > a.max_seq_len))
      raise_status(a.status, BASISKV_DEV_BAD_LENGTH);
    return units_of(len);
  });
  const long long total = pre[a.B] * a.Hkv;
  const long long n_warps = (long long)gridDim.x * kR4Warps;
  const long long w_id = (long long)blockIdx.x * kR4Warps + warp;
  const long long start = total * w_id / n_warps;
  const int run = (int)(total * (w_id + 1) / n_warps - start);

  // Physical pages of 32 units ahead, one a lane (-1: not there).
  int id_a = -1, id_b = -1, id_g = 0, id_base = 0;
  auto fetch_ids = [&](int base) {
    id_base = base;
    id_a = id_b = -1;
    if (base + lane >= run) return;
    const long long x = start + base + lane;
    const int b = line_find(a.B, pre, a.Hkv, x);
    const int U = (int)(pre[b + 1] - pre[b]);
    const unsigned y = (unsigned)(x - pre[b] * a.Hkv);  // below Hkv * U
    id_g = (int)(y / (unsigned)U);
    const int p = (int)(y - (unsigned)id_g * U) * PP;
    const int P = (lens[b] + a.S - 1) / a.S;
    auto look = [&](int q) {
      int id = q < P ? __ldg(a.block_table + (size_t)b * a.max_pages + q) : -1;
      if (q < P && (id < 0 || id >= a.num_phys)) {
        raise_status(a.status, BASISKV_DEV_BAD_PAGE);
        id = -1;
      }
      return id;
    };
    id_a = look(p);
    if (PP == 2) id_b = look(p + 1);
  };
  // Requests units k .. k + NB - 1 into slots `slot` ..: a lane each.
  auto issue = [&](int k, int slot) {
    if (k >= run) return;
    if (k - id_base >= 32) fetch_ids(k);
    const int i = lane - (k - id_base);
    if (i < 0 || i >= NB || k + i >= run) return;
    slot += i;
    const uint32_t st = ring + slot * UB, b = bar + 8 * slot;
    auto copy = [&](uint32_t dst, const uint8_t* src, uint32_t bytes) {
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
          "[%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(b)
          : "memory");
    };
    constexpr int TZ = (ONE ? 18 : 9) * RV, TE = (ONE ? 18 : 9) * RK;  // tile bytes
    tags[warp][slot] = make_uint2(id_a >= 0, id_b >= 0);
    mbar_arrive_expect_tx(bars + warp * NST + slot, ((id_a >= 0) + (id_b >= 0)) * (TZ + TE));
    if (id_a >= 0) {
      const size_t t = (size_t)id_a * a.Hkv + id_g;
      copy(st, a.Z + t * TZ, TZ);
      copy(st + 18 * RV, a.E + t * TE, TE);
    }
    if (id_b >= 0) {
      const size_t t = (size_t)id_b * a.Hkv + id_g;
      copy(st + 9 * RV, a.Z + t * TZ, TZ);
      copy(st + 18 * RV + 9 * RK, a.E + t * TE, TE);
    }
  };
  if (run > 0) fetch_ids(0);
  issue(0, 0);
  issue(NB, NB);
  int k_next = 2 * NB;
  int slot = 0;
  uint32_t phase = 0;
  bool landing = true;  // no wait has run out yet (the others would, too)

  for (int seg = 0; seg < run;) {
    int b, g, u0, item_end;
    {
      const long long x = start + seg;
      b = line_find(a.B, pre, a.Hkv, x);
      const int U = (int)(pre[b + 1] - pre[b]);
      const unsigned y = (unsigned)(x - pre[b] * a.Hkv);  // below Hkv * U
      g = (int)(y / (unsigned)U);
      u0 = (int)(y - (unsigned)g * U);
      item_end = min(run, seg + U - u0);
    }
    const int T = lens[b];
    float* out = a.scores + ((size_t)b * a.Hkv + g) * a.max_pages;
    // ---- folded queries: column n of group j is head 4 j + n / 2, part n % 2
    uint32_t qb[KS][NJ][2];
    float inv[NJ];  // of head 4 j + c, whose scores the lane gets
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int h = 4 * j + (n >> 1);
      const float* qr = a.qt + ((size_t)b * a.Hq + g * a.G + (h < a.G ? h : 0)) * W;
      float f[KS][4], m = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int col = k < RV / 16 ? (RV / 4) * c + 4 * k : RV + (RK / 4) * c + 4 * (k - RV / 16);
        const float4 v = __ldg(reinterpret_cast<const float4*>(qr + col));
        f[k][0] = v.x, f[k][1] = v.y, f[k][2] = v.z, f[k][3] = v.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (h >= a.G) f[k][e] = 0.f;
          m = fmaxf(m, fabsf(f[k][e]));
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int ex = m > 0.f ? (int)((__float_as_uint(m) >> 23) & 0xffu) - 126 : 15;
      const int sh = max(-126, min(126, 15 - ex));
      const float sc = __uint_as_float((uint32_t)(127 + sh) << 23);
      const int shc = __shfl_sync(0xffffffffu, sh, 8 * c);
      inv[j] = __uint_as_float((uint32_t)(127 - shc) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t hi, lo;
          split_f16x2(f[k][2 * e] * sc, f[k][2 * e + 1] * sc, hi, lo);
          qb[k][j][e] = n & 1 ? lo : hi;
        }
    }
    for (; seg < item_end; ++seg, ++u0) {
      landing = landing && mbar_poll(bars + warp * NST + slot, phase, a.status);
      const uint2 tag = tags[warp][slot];
      const uint32_t st = ring + slot * UB;
      const int t0 = u0 * kR4Unit;
      float best[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        float s[NJ][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        constexpr int H1 = ONE ? 8 : 9, S0 = ONE ? 16 : 8, S1 = 17;
        r4_part<RV, 0, KS, NJ>(st + v * H1 * RV, st + (v ? S1 : S0) * RV, n, c, qb, s);
        r4_part<RK, RV / 16, KS, NJ>(st + 18 * RV + v * H1 * RK,
                                     st + 18 * RV + (v ? S1 : S0) * RK, n, c, qb, s);
        float x = -INFINITY, y = -INFINITY;  // tokens n and n + 8
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (4 * j + c < a.G) {
            x = fmaxf(x, (s[j][0] + s[j][1]) * inv[j]);
            y = fmaxf(y, (s[j][2] + s[j][3]) * inv[j]);
          }
        if (t0 + kR4Unit > T) {  // the last unit's tail
          if (t0 + 16 * v + n >= T) x = -INFINITY;
          if (t0 + 16 * v + n + 8 >= T) y = -INFINITY;
        }
        best[v] = fmaxf(x, y);
      }
      if (ONE) {
        const float r = redux_max(fmaxf(best[0], best[1]));
        if (lane == 0) out[u0] = tag.x ? r : -INFINITY;
      } else {
        const float r0 = redux_max(best[0]), r1 = redux_max(best[1]);
        // the second page exists when the unit's first token past it does
        if (lane < 2 && (lane == 0 || t0 + 16 < T))
          out[2 * u0 + lane] = (lane ? tag.y : tag.x) ? (lane ? r1 : r0) : -INFINITY;
      }
      ++slot;
      if (slot == NB || slot == NST) {  // half the ring has been read by every lane
        __syncwarp();
        if (landing) {
          issue(k_next, slot - NB);
          k_next += NB;
        }
        if (slot == NST) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  }
  // a wait has run out: no copy may still be on its way into this block's memory
  if (!landing)
    for (int k = k_next - NST; k < min(k_next, run); ++k)
      mbar_wait(bars + warp * NST + k % NST, (k / NST) & 1, a.status, kDrainNs);
}

template <int RV, int RK, int NJ, bool ONE>
cudaError_t launch_route4_t(const Route4Args& a, cudaStream_t st, bool pdl) {
  constexpr size_t smem = (size_t)kR4Warps * r4_stages<RV + RK, NJ>() * 18 * (RV + RK);
  cudaError_t e = cudaFuncSetAttribute(route4_kernel<RV, RK, NJ, ONE>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long units = (long long)((a.max_seq_len + kR4Unit - 1) / kR4Unit) * a.B * a.Hkv;
  long long grid = (long long)num_sms() * r4_ctas<RV + RK, NJ>();
  if (grid > units / kR4Warps) grid = units / kR4Warps > 0 ? units / kR4Warps : 1;
  return launch_k(route4_kernel<RV, RK, NJ, ONE>, dim3((unsigned)grid), dim3(kR4Threads), smem,
                  st, pdl, a);
}

template <int RV, int RK>
cudaError_t launch_route4_p(const Route4Args& a, cudaStream_t st, bool pdl) {
  if (a.S == 32)
    return a.G == 8 ? launch_route4_t<RV, RK, 2, true>(a, st, pdl)
                    : launch_route4_t<RV, RK, 1, true>(a, st, pdl);
  return a.G == 8 ? launch_route4_t<RV, RK, 2, false>(a, st, pdl)
                  : launch_route4_t<RV, RK, 1, false>(a, st, pdl);
}

template <int RV>
cudaError_t launch_route4_rk(const Route4Args& a, cudaStream_t st, bool pdl) {
  switch (a.r_k) {
    case 16: return launch_route4_p<RV, 16>(a, st, pdl);
    case 32: return launch_route4_p<RV, 32>(a, st, pdl);
    default: return launch_route4_p<RV, 64>(a, st, pdl);
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
