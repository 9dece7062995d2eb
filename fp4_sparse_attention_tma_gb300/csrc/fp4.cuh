// Device code for the 4-bit form: E2M1 codes (sign, two bits of exponent, one of mantissa: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6), two a byte with the even element in the low half, and a UE8M0 scale byte e for
// every 32 elements, which stand for code * 2^(e - 127).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "pairs.cuh"

namespace idxk {

constexpr int kFp4Block = 32;

// 2^(e - 127) (subnormal for e = 0, NaN for e = 255).
__device__ __forceinline__ float scale_of(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}

// The scale byte of a block whose largest magnitude has the bits `top`: the smallest e with
// |x| <= 6 * 2^(e - 127), so that nothing is cut off; 255 where a NaN or an infinity is among them.
// 6 * 2^n is 1.5 * 2^(n + 2): the exponent less 2, and 1 more where the mantissa exceeds 1.5.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const uint32_t e = (top + 0x003FFFFFu) >> 23;
  return e < 2 ? 0u : e - 2;
}

// 8 elements over their block's scale as codes, element 0 in the lowest bits: the multiplication by a
// power of two is exact, the conversion rounds to the nearest code, ties to the even one.
__device__ __forceinline__ uint32_t to_codes(const float (&x)[8], uint32_t e) {
  const float inv = __uint_as_float((254u - e) << 23);   // 2^(127 - e)
  uint32_t r;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 z = both(mul2(two(x[i], x[i + 1]), two(inv, inv)));
    y[i] = z.x, y[i + 1] = z.y;
  }
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return e == 255 ? 0u : r;   // not finite: codes 0
}

// The 8 codes of a word as pairs of fp16 numbers (exact).
__device__ __forceinline__ void from_codes(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "mov.b32 {t0, t1, t2, t3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, t2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

}  // namespace idxk
