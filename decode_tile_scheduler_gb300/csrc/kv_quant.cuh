// kv_quant.cuh -- the codes of quantised cache rows: E4M3 with an fp32 scale per 64
// elements, E2M1 with an E8M0 scale per 32 (fia.h gives both rules).
#pragma once

#include "common.cuh"

namespace fia {

constexpr float kFp8Max = 448.f;
constexpr float kBf16Max = 3.38953139e38f;  // largest finite bf16 value

// Four values over `scale` as E4M3 codes, the first in the lowest byte.  (The division
// as IEEE rounds it is the format's definition.)
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3, float scale) {
  uint32_t r;  // (the first source of a pair lands in its upper byte)
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(__fdiv_rn(x0, scale)), "f"(__fdiv_rn(x1, scale)), "f"(__fdiv_rn(x2, scale)),
        "f"(__fdiv_rn(x3, scale)));
  return r;
}

// The E8M0 code of the smallest 2^e, e >= -127, with amax <= 6 * 2^e (amax finite, not
// negative; 127, a scale of 1, for 0).  With amax = 1.f * 2^x, 6 = 1.5 * 2^2: e = x - 2
// where 1.f <= 1.5, else x - 1; below the normal numbers 2^-127 is enough.
__device__ __forceinline__ int mx_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  if (bits == 0u) return 127;
  return max((int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0), 0);
}
// 2^-(e - 127), for codes up to 253 (every finite amax's).
__device__ __forceinline__ float mx_inverse(int e) { return __int_as_float((254 - e) << 23); }

// Eight values times `inv` as E2M1 codes, to nearest, ties to even, saturated at 6; the
// first in the lowest half byte.  (Powers of two: the products are exact, or so small
// that the code is 0.)
__device__ __forceinline__ uint32_t e2m1x8(float x0, float x1, float x2, float x3, float x4,
                                           float x5, float x6, float x7, float inv) {
  uint32_t r;  // (the first source of a pair lands in the upper half)
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x0 * inv), "f"(x1 * inv), "f"(x2 * inv), "f"(x3 * inv), "f"(x4 * inv), "f"(x5 * inv),
        "f"(x6 * inv), "f"(x7 * inv));
  return r;
}

}  // namespace fia
