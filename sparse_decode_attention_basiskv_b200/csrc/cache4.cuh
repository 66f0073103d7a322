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

// Scale byte of a block whose largest magnitude is amax (a bf16 value >= 0).
// Below 2^-14 the byte counts steps of 2^-17 (a half's subnormals).
//
// The quotient is taken as a product with fp32(1 / 6), off by less than 2^-22
// of it, and then rounded to 13 significant bits: a quotient of an 8-bit
// number by 6 either is a tie of the 4-bit rounding, which 13 bits hold
// exactly, or lies at least 2^-9 of itself from every tie, so the byte is that
// of the exact quotient.
__device__ __forceinline__ uint32_t q4_scale_byte(float amax) {
  const float s = fminf(amax * (1.f / 6.f), kQ4MaxScale);
  const uint32_t u = (__float_as_uint(s) + 0x200u) & ~0x3ffu;
  if (s < 6.1035e-05f)  // below 2^-14 less the rounding (where both forms agree)
    return (uint32_t)__float2int_rn(__uint_as_float(u) * 131072.f);
  return ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
}
__device__ __forceinline__ float q4_scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}
// The scale twice, as an f16 pair.
__device__ __forceinline__ uint32_t q4_scale_x2(uint32_t byte) { return byte * 0x00800080u; }

// x / scale for two columns, ready for the rounding to E2M1.  inv is 1 / scale
// to fp32: adding and taking off 1.5 * 2^11 rounds the product to multiples of
// 2^-12.  A quotient of an 8-bit number by a 4-bit one either is a tie between
// two codes, which that keeps exactly, or lies at least 2^-8 of itself (2^-10)
// from every tie, so the codes are those of the exact quotient.
__device__ __forceinline__ float2 q4_quotient2(float2 x, float2 inv) {
  constexpr float C = 0x1.8p11f;
  float2 t = make_float2(C, C);
  ffma2(t, x, inv);
  return make_float2(t.x - C, t.y - C);
}

// Eight columns -> four bytes of codes (even columns in the low nibbles),
// nearest even, saturated.
__device__ __forceinline__ uint32_t q4_pack8(const float2 (&x)[4]) {
  uint32_t r;
  asm("{ .reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d}; }"
      : "=r"(r)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y),
        "f"(x[3].x), "f"(x[3].y));
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
