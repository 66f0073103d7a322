// Writing rows into a 4-bit cache, and reading them back.
//
// Both are one pass over the data: 2 bytes a column in and 9/16 out, or the
// other way round, with a few operations a column, so HBM bounds them.  A
// lane handles 8 columns of one row (a 16-byte access on the dense side and a
// 4-byte one on the cache side); two neighbouring lanes share a block of 16
// columns and meet in one shuffle for its largest magnitude.  The columns of
// all heads of one token's row are contiguous, so a CTA walks tokens with its
// lanes along that row.
#include "cache4.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace basiskv {
namespace {

constexpr int kC4Threads = 256;

// Where token t of sequence b lives: the tile row index (physical page *
// S + row), or -1 (no such page).
__device__ __forceinline__ int c4_row(const Cache4Args& a, int b, int t) {
  const int p = t / a.S;
  if (p >= a.max_pages) return -1;
  const int pp = __ldg(a.block_table + (size_t)b * a.max_pages + p);
  if (pp < 0 || pp >= a.num_phys) {
    raise_status(a.status, BASISKV_DEV_BAD_PAGE);
    return -1;
  }
  return pp * a.S + (t - p * a.S);
}

// Part and chunk of task i of one token: the rows of k, z and e one after
// the other, Hkv * w / 8 chunks each.
struct C4Task {
  int part, g, c, w;
};
__device__ __forceinline__ C4Task c4_task(const Cache4Args& a, int i) {
  C4Task t;
  t.part = 0;
#pragma unroll
  for (int p = 0; p < 2; ++p)
    if (t.part == p && i >= a.chunks[p]) {
      i -= a.chunks[p];
      ++t.part;
    }
  t.w = a.width[t.part];
  t.g = i / (t.w >> 3);
  t.c = i - t.g * (t.w >> 3);
  return t;
}

__global__ void __launch_bounds__(kC4Threads) cache4_write_kernel(Cache4Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int per = a.chunks[0] + a.chunks[1] + a.chunks[2];  // even: w / 8 is even
  const int b = blockIdx.z;
  const int len = __ldg(a.seq_lens + b);
  const bool fits = len >= 0 && (long long)len + a.n <= (long long)a.max_pages * a.S;
  if (a.lens_out && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (!fits) raise_status(a.status, BASISKV_DEV_OVERFLOW);
    a.lens_out[b] = fits ? len + a.n : len;
  }
  if (!fits) return;
  for (int j = blockIdx.y; j < a.n; j += gridDim.y) {
    const int row = c4_row(a, b, len + j);
    if (row < 0) continue;
    const int pp = row / a.S, r = row - pp * a.S;
    for (int i = blockIdx.x * kC4Threads + threadIdx.x; i < per; i += gridDim.x * kC4Threads) {
      const C4Task t = c4_task(a, i);
      const uint16_t* src = a.rows[t.part];
      const uint4 v = ldg_stream(src + (((size_t)b * a.n + j) * a.Hkv + t.g) * t.w + 8 * t.c);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      float f[8], m = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = bf16lo(u[k]);
        f[2 * k + 1] = bf16hi(u[k]);
        m = fmaxf(m, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
      }
      // lanes 2i and 2i + 1 hold one block and leave the loop together
      const unsigned pair = 3u << (threadIdx.x & 30);
      m = fmaxf(m, __shfl_xor_sync(pair, m, 1));
      const uint32_t sb = q4_scale_byte(m);
      const float s = q4_scale_value(sb);
      uint32_t codes = 0;
      if (sb) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          codes |= q4_pack2(__fdiv_rn(f[2 * k], s), __fdiv_rn(f[2 * k + 1], s)) << (8 * k);
      }
      uint8_t* tile = a.cache[t.part] + (size_t)(pp * a.Hkv + t.g) * q4_tile_bytes(a.S, t.w);
      *reinterpret_cast<uint32_t*>(tile + (r * t.w >> 1) + 4 * t.c) = codes;
      if (!(t.c & 1)) tile[(a.S * t.w >> 1) + (r * t.w >> 4) + (t.c >> 1)] = (uint8_t)sb;
    }
  }
}

__global__ void __launch_bounds__(kC4Threads) cache4_read_kernel(Cache4Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int per = a.chunks[0] + a.chunks[1] + a.chunks[2];
  const int b = blockIdx.z;
  const int first = __ldg(a.first + b);
  const int len = __ldg(a.seq_lens + b);
  for (int j = blockIdx.y; j < a.n; j += gridDim.y) {
    const long long t64 = (long long)first + j;
    if (t64 < 0 || t64 >= len) continue;  // not a live token: its row is left as it was
    const int row = c4_row(a, b, (int)t64);
    if (row < 0) continue;
    const int pp = row / a.S, r = row - pp * a.S;
    for (int i = blockIdx.x * kC4Threads + threadIdx.x; i < per; i += gridDim.x * kC4Threads) {
      const C4Task t = c4_task(a, i);
      const uint8_t* tile =
          a.cache[t.part] + (size_t)(pp * a.Hkv + t.g) * q4_tile_bytes(a.S, t.w);
      const uint32_t w =
          __ldg(reinterpret_cast<const uint32_t*>(tile + (r * t.w >> 1) + 4 * t.c));
      const float s = q4_scale_value(__ldg(tile + (a.S * t.w >> 1) + (r * t.w >> 4) + (t.c >> 1)));
      uint32_t h[4], o[4];
      q4_unpack8(w, h);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
        o[k] = (uint32_t)f_to_bf16(f.x * s) | ((uint32_t)f_to_bf16(f.y * s) << 16);
      }
      *reinterpret_cast<uint4*>(a.out[t.part] + (((size_t)b * a.n + j) * a.Hkv + t.g) * t.w +
                                8 * t.c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

dim3 c4_grid(const Cache4Args& a) {
  const int per = a.chunks[0] + a.chunks[1] + a.chunks[2];
  const int gx = (per + kC4Threads - 1) / kC4Threads;
  long gy = (long)num_sms() * 16 / ((long)gx * a.B);
  if (gy < 1) gy = 1;
  if (gy > a.n) gy = a.n;
  return dim3(gx, (unsigned)gy, a.B);
}

}  // namespace

cudaError_t launch_cache4_write(const Cache4Args& a, cudaStream_t st, bool pdl) {
  return launch_k(cache4_write_kernel, c4_grid(a), dim3(kC4Threads), 0, st, pdl, a);
}

cudaError_t launch_cache4_read(const Cache4Args& a, cudaStream_t st, bool pdl) {
  return launch_k(cache4_read_kernel, c4_grid(a), dim3(kC4Threads), 0, st, pdl, a);
}

}  // namespace basiskv
