// moe_fp4.cuh - MXFP4 arithmetic shared by the conversion kernels and the
// gate/up product: blocks of 32 consecutive elements, one power-of-two scale
// per block (UE8M0: its biased exponent byte), E2M1 elements, two to a byte,
// the even element in the low half.
//
// Scale (OCP MX): 2^(floor(log2 amax) - 2), 2 being the exponent of E2M1's
// largest number 6 = 1.5 * 2^2.  floor(log2 amax) is amax's exponent field, so
// the scale byte is max(field - 2, 0) (a block below 2^-125 takes 2^-127).
// Elements are x / scale (exact: a power of two), rounded to nearest even and
// saturated to 6.  A block that holds a NaN or an infinity takes the NaN scale
// byte 255 and zero codes: it reads back as NaN everywhere.
#pragma once

#include <cstdint>

namespace moe {

constexpr uint32_t kFp4NanScale = 255u;

// Scale byte of a block whose largest |x| has the bits `amax_bits`.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax_bits) {
  const uint32_t field = amax_bits >> 23;
  return field == 255u ? kFp4NanScale : (field > 2u ? field - 2u : 0u);
}

// 1 / scale = 2^(127 - byte), 0 for the NaN scale.  Bytes run from 0 to 252
// otherwise, so the exponent field 254 - byte is a normal number's.
__device__ __forceinline__ float fp4_inv_scale(uint32_t byte) {
  return byte == kFp4NanScale ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// The scale itself: 2^(byte - 127); 2^-127 is subnormal.
__device__ __forceinline__ float fp4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : (byte == kFp4NanScale ? 0x7FC00000u : byte << 23));
}

// Eight floats (already divided by their scale) to eight E2M1 codes (round to
// nearest even, saturating), the first in the lowest bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// A byte of two codes to two halves (exact), the low code in the low half.
__device__ __forceinline__ uint32_t e2m1x2_to_half2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}

}  // namespace moe
