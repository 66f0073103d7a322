// Writing rows into a 4-bit cache, and reading them back.
//
// Both are one pass over the data: 2 bytes a column in and 9/16 out, or the
// other way round, with some five operations a column, so HBM bounds them as
// long as the bookkeeping stays small.  A thread keeps one block of 16 columns
// of one head (of the k, z or e row) and walks tokens: 32 contiguous bytes on
// the dense side (one 256-bit access), 8 bytes of codes and the scale's byte
// on the cache side, and nothing to share with its neighbours.  The blocks of
// one token are spread over a CTA's threads, several tokens side by side
// where a token has few.  One row at a time a thread, at 48 resident warps:
// more rows in flight cost registers, and so warps.
//
// Measured (8 x 4096 tokens, 8 KV heads, 128 + 96 + 64 columns, 193 MB each way):
// write 37 us, read 41, together 81, 4.8 TB/s where a copy reaches 6.5: the warps wait
// for their loads, so it is bytes in flight that lack.  With two rows a thread 86 us,
// with four 94, at 32 resident warps 92; blocks of four rows on CTAs of 256 threads,
// of which a token of 144 blocks left 112 idle, 106.
#include "cache4.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace basiskv {
namespace {

constexpr int kC4Threads = 512;  // of a CTA, at most
constexpr int kC4Warps = 48;      // resident on an SM

struct Block16 {
  uint32_t w[8];
};
// A block of a dense row: one access where the rows are 32-byte aligned, else two.
__device__ __forceinline__ Block16 ld_block(const uint16_t* p, bool wide) {
  Block16 v;
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]),
                   "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p));
  } else {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    const uint4 y = __ldg(reinterpret_cast<const uint4*>(p + 8));
    v = {{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}};
  }
  return v;
}
__device__ __forceinline__ void st_block(uint16_t* p, const Block16& v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]),
                 "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
                 "r"(v.w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    *reinterpret_cast<uint4*>(p + 8) = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
  }
}

// The thread's block: part (k, z, e), head, block within the head's row.
struct C4Block {
  int part, g, c, w;
};
__device__ __forceinline__ C4Block c4_block(const Cache4Args& a, int i) {
  C4Block t;
  t.part = 0;
#pragma unroll
  for (int p = 0; p < 2; ++p)
    if (t.part == p && i >= a.blocks[p]) {
      i -= a.blocks[p];
      ++t.part;
    }
  t.w = t.part == 0 ? a.width[0] : (t.part == 1 ? a.width[1] : a.width[2]);
  t.g = i / (t.w >> 4);
  t.c = i - t.g * (t.w >> 4);
  return t;
}

// Physical page of token t of sequence b, or -1 (out of range: reported).
__device__ __forceinline__ int c4_page(const Cache4Args& a, int b, int t) {
  const int p = t >> a.logS;
  const int pp = p < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + p) : -1;
  if (pp >= 0 && pp < a.num_phys) return pp;
  raise_status(a.status, BASISKV_DEV_BAD_PAGE);
  return -1;
}

template <bool WRITE>
__global__ void __launch_bounds__(kC4Threads, kC4Warps * 32 / kC4Threads)
    cache4_kernel(Cache4Args a, int per, int side) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.z;
  const int len = __ldg(a.seq_lens + b);
  int t0;  // token of row 0
  if constexpr (WRITE) {
    const bool fits = len >= 0 && (long long)len + a.n <= (long long)a.max_pages * a.S;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
      if (!fits) raise_status(a.status, BASISKV_DEV_OVERFLOW);
      if (a.lens_out) a.lens_out[b] = fits ? len + a.n : len;
    }
    if (!fits) return;
    t0 = len;
  } else {
    t0 = __ldg(a.first + b);
  }
  const int s = threadIdx.x / per, i = blockIdx.x * per + threadIdx.x - s * per;
  if (s >= side || i >= a.blocks[0] + a.blocks[1] + a.blocks[2]) return;
  const C4Block t = c4_block(a, i);
  // dense rows, and the block's place in a tile
  const size_t pitch = (size_t)a.Hkv * t.w;
  const size_t dense = (size_t)b * a.n * pitch + t.g * t.w + 16 * t.c;
  const uint16_t* src =
      WRITE ? (t.part == 0 ? a.rows[0] : t.part == 1 ? a.rows[1] : a.rows[2]) + dense : nullptr;
  uint16_t* dst =
      WRITE ? nullptr : (t.part == 0 ? a.out[0] : t.part == 1 ? a.out[1] : a.out[2]) + dense;
  const bool wide = (reinterpret_cast<uintptr_t>(WRITE ? src : dst) & 31) == 0;
  const uint32_t tile_bytes = q4_tile_bytes(a.S, t.w);
  uint8_t* cache = (t.part == 0 ? a.cache[0] : t.part == 1 ? a.cache[1] : a.cache[2]) +
                   (size_t)t.g * tile_bytes;
  const size_t page_bytes = (size_t)a.Hkv * tile_bytes;
  const uint32_t code_at = 8 * t.c, scale_at = (a.S * t.w >> 1) + t.c;

  const int step = side * gridDim.y;
  int j = blockIdx.y * side + s;
  // page of row j (-1: the row is left as it was), looked up a row ahead
  auto page_of = [&](int j) {
    const long long tok = (long long)t0 + j;
    if (j >= a.n || (!WRITE && (tok < 0 || tok >= len))) return -1;
    return c4_page(a, b, (int)tok);
  };
  for (int next = page_of(j); j < a.n; j += step) {
    const int pp = next;
    if constexpr (WRITE) {
      const Block16 v = ld_block(src + (size_t)j * pitch, wide);
      next = page_of(j + step);
      if (pp < 0) continue;
      // largest magnitude on pairs of bf16 without their signs (integer order)
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = __vmaxu2(m, v.w[e] & 0x7fff7fffu);
      const float amax = __uint_as_float(max(m & 0xffff0000u, m << 16));
      const uint32_t sb = q4_scale_byte(amax);
      uint2 codes = make_uint2(0u, 0u);
      if (sb) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(q4_scale_value(sb)));
        const float2 inv = make_float2(r, r);
        float2 x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = q4_quotient2(bf16x2_to_f2(v.w[e]), inv);
          y[e] = q4_quotient2(bf16x2_to_f2(v.w[4 + e]), inv);
        }
        codes = make_uint2(q4_pack8(x), q4_pack8(y));
      }
      const int r = (int)(((uint32_t)t0 + (uint32_t)j) & (uint32_t)(a.S - 1));
      uint8_t* tile = cache + pp * page_bytes;
      *reinterpret_cast<uint2*>(tile + r * (t.w >> 1) + code_at) = codes;
      tile[r * (t.w >> 4) + scale_at] = (uint8_t)sb;
    } else {
      const int r = (int)(((uint32_t)t0 + (uint32_t)j) & (uint32_t)(a.S - 1));
      const uint8_t* tile = cache + (pp < 0 ? 0 : pp) * page_bytes;
      uint2 w = make_uint2(0u, 0u);
      uint32_t sb = 0;
      if (pp >= 0) {
        w = __ldg(reinterpret_cast<const uint2*>(tile + r * (t.w >> 1) + code_at));
        sb = __ldg(tile + r * (t.w >> 4) + scale_at);
      }
      next = page_of(j + step);
      if (pp < 0) continue;
      const uint32_t s2 = q4_scale_x2(sb);
      uint32_t h[8];
      q4_unpack8(w.x, *reinterpret_cast<uint32_t(*)[4]>(h));
      q4_unpack8(w.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
      Block16 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // exact in f16 and in bf16
        const uint32_t p = hmul2(h[e], s2);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
        const __nv_bfloat162 u = __floats2bfloat162_rn(f.x, f.y);
        o.w[e] = *reinterpret_cast<const uint32_t*>(&u);
      }
      st_block(dst + (size_t)j * pitch, o, wide);
    }
  }
}

// CTAs of `side` tokens of all their blocks (of half of them or less where a
// token has more than 320), the number of tokens that leaves the fewest lanes of
// the last warp without a block; one wave of them, which walks the tokens.
template <bool WRITE>
cudaError_t launch_cache4(const Cache4Args& a, cudaStream_t st, bool pdl) {
  constexpr int kMost = 320;
  const int all = a.blocks[0] + a.blocks[1] + a.blocks[2];
  const int gx = (all + kMost - 1) / kMost;
  const int per = gx == 1 ? all : ((all + gx - 1) / gx + 31) / 32 * 32;  // threads a token
  auto warps = [&](int tokens) { return (tokens * per + 31) / 32; };
  int side = 1;
  for (int x = 2; x * per <= kMost; ++x)
    if (warps(x) * side <= warps(side) * x) side = x;
  long long gy = (long long)num_sms() * (kC4Warps / warps(side)) / ((long long)gx * a.B);
  const long long most = (a.n + side - 1) / side;
  if (gy > most) gy = most;
  if (gy < 1) gy = 1;
  return launch_k(cache4_kernel<WRITE>, dim3(gx, (unsigned)gy, a.B), dim3(32 * warps(side)), 0, st,
                  pdl, a, per, side);
}

}  // namespace

cudaError_t launch_cache4_write(const Cache4Args& a, cudaStream_t st, bool pdl) {
  return launch_cache4<true>(a, st, pdl);
}

cudaError_t launch_cache4_read(const Cache4Args& a, cudaStream_t st, bool pdl) {
  return launch_cache4<false>(a, st, pdl);
}

}  // namespace basiskv
