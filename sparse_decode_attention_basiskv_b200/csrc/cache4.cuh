// The 4-bit cache format (device side).
//
// A row of w columns is cut into blocks of 16.  Each block has one scale
// byte, 5 exponent bits (bias 15) over 3 mantissa bits: the upper bits of an
// IEEE half without its sign, so (byte << 7) are the scale's half bits.  Each
// column is an E2M1 code (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6), two codes a byte, the even column in the low nibble.
//
//   scale = round(amax / 6)  to 4 significant bits, nearest even, <= 10240
//   code  = round(x / scale) to E2M1, nearest even, magnitude <= 6
//   value = code * scale
//
// value has at most 6 significant bits and lies in [2^-18, 61440], so it is
// exact in f16 and in bf16: the attention and the scoring widen codes to f16,
// multiply by the scale in f16, and lose nothing.  10240 = 61440 / 6 is the
// largest scale whose products stay finite in f16.
//
// One (page, KV head) tile of S rows: codes [S][w / 2], then scales
// [S][w / 16]; S * w * 9 / 16 bytes, a multiple of 16.
#pragma once

#include "common.cuh"

namespace basiskv {

__host__ __device__ constexpr int q4_tile_bytes(int S, int w) { return S * w / 16 * 9; }

constexpr float kQ4MaxScale = 10240.f;

// Scale byte of a block whose largest magnitude is amax (>= 0, finite).
// Below 2^-14 the byte counts steps of 2^-17 (a half's subnormals).
__device__ __forceinline__ uint32_t q4_scale_byte(float amax) {
  const float s = fminf(__fdiv_rn(amax, 6.f), kQ4MaxScale);
  if (s < 6.103515625e-05f) return (uint32_t)__float2int_rn(s * 131072.f);
  const uint32_t u = __float_as_uint(s);
  return ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
}
__device__ __forceinline__ float q4_scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}
// The scale twice, as an f16 pair.
__device__ __forceinline__ uint32_t q4_scale_x2(uint32_t byte) { return byte * 0x00800080u; }

// One byte of codes (low nibble x0, high nibble x1), nearest even, saturated.
__device__ __forceinline__ uint32_t q4_pack2(float x0, float x1) {
  uint32_t r;
  asm("{ .reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
      "cvt.u32.u8 %0, t; }"
      : "=r"(r)
      : "f"(x0), "f"(x1));
  return r;
}

// Four bytes of codes -> four f16 pairs (pair i = byte i: low nibble first).
__device__ __forceinline__ void q4_unpack8(uint32_t w, uint32_t (&o)[4]) {
  asm("{ .reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace basiskv
