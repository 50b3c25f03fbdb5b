// fp4.cuh -- the 4-bit cache's format and its conversions.
//
// The K (or V) of a head in a page is page_size / 16 blocks of 9 D bytes, one
// after the other.  A block holds 16 positions: [16][D / 2] bytes of e2m1 codes
// (the even element in the low four bits), then [16][D / 16] e4m3 scales, one
// for 16 elements.  Any run of whole blocks is so one contiguous piece that
// a single bulk copy moves, whatever the page size, and a page is plain
// bytes to the page operations.
//
// A code has two significant bits and a scale four, so code x scale is exact
// in fp16 (2^-10 .. 2688) as in bf16: products with it lose nothing that the
// cache held.
#pragma once

#include <stdint.h>

#include "f32x2.cuh"

namespace dspark {

constexpr int kFp4Block = 16;  // positions of a block, and elements of a scale
__host__ __device__ constexpr int fp4_block_bytes(int D) { return 9 * D; }

// Byte offsets of a position's codes and scales within a head's part of a page.
__device__ __forceinline__ long long fp4_codes_at(int slot, int D) {
  return (long long)(slot >> 4) * (9 * D) + (slot & 15) * (D / 2);
}
__device__ __forceinline__ long long fp4_scales_at(int slot, int D) {
  return (long long)(slot >> 4) * (9 * D) + 8 * D + (slot & 15) * (D / 16);
}

// Eight codes as four pairs of fp16, elements in order.
__device__ __forceinline__ void fp4x8_to_half(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ void fp4x4_to_half(uint32_t w, uint32_t* h) {  // the low four codes
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
}

// Two e4m3 scales (the low 16 bits of s) as a pair of fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_half(uint32_t s) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(s));
  return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float half_lo(uint32_t h) {
  float f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float half_hi(uint32_t h) {
  float f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, b;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t s) { return half_lo(e4m3x2_to_half(s & 0xffu)); }

// The e4m3 nearest to x >= 0, at most 448.
__device__ __forceinline__ uint32_t float_to_e4m3(float x) {
  uint32_t r;
  asm("{\n\t.reg .b16 a;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.u32.u16 %0, a;\n\t}"
      : "=r"(r)
      : "f"(x), "f"(0.0f));
  return r;
}

// The e2m1 codes nearest to (lo, hi), ties to even, at most 6: lo in the low four bits.
__device__ __forceinline__ uint32_t floats_to_fp4x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.u32.u8 %0, a;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// The scale of a group from its largest magnitude (as bits, so that what is not
// finite counts as the largest): its byte, and what its elements are divided by.
// A group with an element that is not finite gets the scale NaN, and reads as NaN.
struct Fp4Scale {  // (inverse: of value, nearly)
  uint32_t byte;
  float value, inverse;  // scale x factor; 0 where the scale is 0 or NaN: all codes are 0
};
__device__ __forceinline__ float reciprocal(float x) {  // within a step or so; x is normal
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The e4m3 nearest to a / (6 factor).  (The sixth is refined by its exact remainder like fp4_quotient's.)
__device__ __forceinline__ uint32_t fp4_scale_byte(float a, float inv_factor) {
  a = fminf(a * inv_factor, 3e38f);
  const float sixth = 1.0f / 6.0f, q = a * sixth;
  return float_to_e4m3(__fmaf_rn(__fmaf_rn(-q, 6.0f, a), sixth, q));
}
__device__ __forceinline__ Fp4Scale fp4_scale(uint32_t amax_bits, float factor, float inv_factor) {
  Fp4Scale s;
  if (amax_bits >= 0x7f800000u) return Fp4Scale{0x7fu, 0.0f, 0.0f};
  s.byte = fp4_scale_byte(__uint_as_float(amax_bits), inv_factor);
  s.value = e4m3_to_float(s.byte) * factor;
  s.inverse = s.byte == 0u ? 0.0f : reciprocal(s.value);
  return s;
}

// x / s.value, so exactly rounded that a code's border is met if and only if x
// lies on it: the quotient by the rounded inverse, refined once by its exact
// remainder.  (A border times the scale has at most seven bits, so an x beside it
// is at least 2^-24 away relatively, more than half a step of the quotient.)
// Under any scale but the largest the quotient is at most 9 (for a subnormal scale).  Under that one it may
// leave fp32's range, and the remainder would be inf - inf: what is past 8 counts as 8, whose
// code is that of 6.
constexpr uint32_t kFp4LargestScale = 0x7eu;  // 448
__device__ __forceinline__ float at_most_8(float x, const Fp4Scale& s) {
  float y;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(8.0f * s.value));
  return y;
}
__device__ __forceinline__ float fp4_quotient(float x, const Fp4Scale& s) {
  x = at_most_8(x, s);
  const float q = x * s.inverse;
  return __fmaf_rn(__fmaf_rn(-q, s.value, x), s.inverse, q);
}

// h rounded to nearest and what it leaves, l, to one number: h with its last bit set
// wherever l is not 0 ("rounding to odd": Boldo and Melquiond, "Emulation of FMA and
// correctly rounded sums", 2008), so that a later rounding to fewer bits, or a comparison
// with a number of fewer, is that of h + l.
__device__ __forceinline__ float to_odd(float h, float l) {
  uint32_t bits = __float_as_uint(h);
  // (l is NaN where h is not finite)
  if (fabsf(l) > 0.0f && !(bits & 1u)) bits += (__float_as_uint(l) ^ bits) >> 31 ? -1 : 1;
  return __uint_as_float(bits);
}

// a c + b s, rounded to odd at 24 bits.  Products and sums as unevaluated pairs
// (Dekker 1971, Knuth's two-sum).  Not in packed arithmetic: there the compiler joins a
// product and a sum to one operation, also where they are written as roundings of their own.
__device__ __forceinline__ float rotated_odd(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
  const float ep = __fmaf_rn(a, c, -p), eq = __fmaf_rn(b, s, -q);
  const float r = __fadd_rn(p, q), t = __fsub_rn(r, p);
  const float er = __fadd_rn(__fsub_rn(p, __fsub_rn(r, t)), __fsub_rn(q, t));
  const float lo = __fadd_rn(er, __fadd_rn(ep, eq));
  const float h = __fadd_rn(r, lo), u = __fsub_rn(h, r);
  return to_odd(h, __fadd_rn(__fsub_rn(r, __fsub_rn(h, u)), __fsub_rn(lo, u)));
}

}  // namespace dspark
