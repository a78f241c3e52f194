// A row of a 4-bit pool: one token of one kv head, 128 columns in 72 bytes -- 64 of e2m1
// codes (1 sign, 2 exponent bits, 1 fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6; column 2 i in
// the low half of byte i), then a scale for each 16 columns.  A scale is the upper bits of
// a positive half: 5 exponent and 3 fraction bits, byte b standing for the half with the
// bits b << 7.  So a scale is decoded by a shift, NaN included, and code times scale (2 and
// 4 significant bits) is exact as a half up to 6 * 10240 and as a bf16.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "pa_device.cuh"

namespace pa {

constexpr int kRow4Bytes = 72;                    // a row: codes, then scales
constexpr int kRow4Codes = 64;
constexpr float kMostScale4 = 10240.f;            // 6 * 10240 is below the largest half
constexpr uint32_t kNanScale4 = 0xffu;

// The scale byte of 16 columns whose largest magnitude has the bits `amax` (of a float; the
// bits of a NaN are the largest): the nearest to amax / 6, ties to even, steps of 2^-17 at
// the least; NaN if one of them is.
__device__ __forceinline__ uint32_t scale4_of(uint32_t amax) {
  if (amax > 0x7f800000u) return kNanScale4;
  const float y = fminf(__fdiv_rn(__uint_as_float(amax), 6.f), kMostScale4);
  if (y < 6.103515625e-5f) return static_cast<uint32_t>(__float2int_rn(y * 131072.f));   // below 2^-14
  const uint32_t u = __float_as_uint(y);
  return ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
}

__device__ __forceinline__ float scale4_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// x / s, correctly rounded, from r = 1 / s correctly rounded: the product with r, corrected
// by its exact remainder (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990).  A product alone would take some of the many bf16
// elements that lie on the border of two codes to the wrong one.
__device__ __forceinline__ float quotient4(float x, float s, float r) {
  const float z = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-z, s, x), r, z);
}

// Eight floats over s as codes: nearest, ties to even, magnitudes above 6 s saturate.  Zeros have no
// sign (the remainder's sum is +0), and under a scale of 0 nothing has.
__device__ __forceinline__ uint32_t codes4_of(const float* x, float s) {
  const float r = s > 0.f ? __frcp_rn(s) : 0.f;
  // (beyond 8 s a code saturates, and an infinity has no remainder: only the largest scale
  // has such elements)
  const bool over = s == kMostScale4;
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = quotient4(over ? fminf(fmaxf(x[i], -8.f * s), 8.f * s) : x[i], s, r);
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
  return s == 0.f ? 0u : w;
}

// The eight codes of a word as four pairs of halves, unscaled (the lower column in the
// lower half).
__device__ __forceinline__ void halves4_of(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace pa
