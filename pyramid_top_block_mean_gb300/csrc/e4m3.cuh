// e4m3.cuh -- rows of an 8-bit cache: e4m3 codes and a power of two each.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pisa {

// e4m3 rows.  A code c of a row with the scale s stands for c 2^(s - 127): the
// bits of c, its sign apart, placed 4 bits up are the bf16 number c 2^-120 (for
// subnormal codes too), and a product with 2^(s - 7) makes it the row's number,
// exactly.  That power is a bf16 number up to s = 134; beyond (rows with values
// over 57344) a second product does the rest.  A scale of 255 gives NaN.
__device__ __forceinline__ uint32_t row_factor(uint32_t scale) {  // in both halves of a pair
  const uint32_t f = scale == 255u ? 0x7fc0u : (scale < 134u ? scale + 120u : 254u) << 7;
  return f * 0x10001u;
}
__device__ __forceinline__ bool row_is_large(uint32_t scale) { return scale > 134u && scale != 255u; }
__device__ __forceinline__ uint32_t row_factor_large(uint32_t scale) {
  return (row_is_large(scale) ? scale - 134u + 127u : 127u) * 0x800080u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two codes, each with its sign in all bits of the byte above it (prmt's
// replicating selectors), as bf16 numbers times 2^-120.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x) { return (x << 4) & 0x87f087f0u; }
// The codes of bytes 0 and 1, and of bytes 2 and 3, of a word.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t x;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(x) : "r"(w));
  return codes_to_bf16(x);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t x;
  asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(x) : "r"(w));
  return codes_to_bf16(x);
}
// The codes of bytes 0 and 1, and of bytes 2 and 3, in fp16, of which every
// code is a number (NaN's codes stay NaN).
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Two numbers, already over their row's power, to the nearest codes.
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Four pairs times a factor; eight codes as pairs of bf16 numbers times a factor
// (row_factor), and as those of a row with any scale.
__device__ __forceinline__ uint4 mul_pairs(uint4 x, uint32_t f) {
  return make_uint4(mul_bf16x2(x.x, f), mul_bf16x2(x.y, f), mul_bf16x2(x.z, f), mul_bf16x2(x.w, f));
}
__device__ __forceinline__ uint4 code_pairs(uint2 w, uint32_t f) {
  return mul_pairs(make_uint4(codes_lo(w.x), codes_hi(w.x), codes_lo(w.y), codes_hi(w.y)), f);
}
__device__ __forceinline__ uint4 row_pairs(uint2 w, uint32_t scale) {
  const uint4 x = code_pairs(w, row_factor(scale));
  return row_is_large(scale) ? mul_pairs(x, row_factor_large(scale)) : x;
}
// The number of one code of a row with the scale s, in fp32.
__device__ __forceinline__ float code_number(uint32_t c, uint32_t scale) {
  const float x = __uint_as_float((c & 0x80u) << 24 | (c & 0x7fu) << 20) * 0x1p120f;
  return scale == 255u ? __uint_as_float(0x7fc00000u) : x * __uint_as_float(scale << 23);
}

}  // namespace pisa
