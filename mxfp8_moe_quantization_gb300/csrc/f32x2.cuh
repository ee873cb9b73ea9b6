// Packed fp32 arithmetic on pairs of neighbouring columns, and mixed-precision
// products of bf16 pairs, for the kernels that are bound by HBM only while
// they spend few instructions per element.
#pragma once
#include "common.cuh"

namespace fp8moe {

FP8MOE_DEV uint64_t pk(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
FP8MOE_DEV void unpk(uint64_t p, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
FP8MOE_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
FP8MOE_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
FP8MOE_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
FP8MOE_DEV float sum_of(uint64_t p) {
  float a, b;
  unpk(p, a, b);
  return a + b;
}
FP8MOE_DEV uint64_t unpk_bf16(uint32_t w) { return pk(bf16_lo(w), bf16_hi(w)); }
FP8MOE_DEV uint32_t pack_bf16x2(uint64_t p) {
  float a, b;
  unpk(p, a, b);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// the products of two bf16 pairs, exact in fp32 (mixed-precision fma on the
// halves: no unpacking)
FP8MOE_DEV uint64_t mulx(uint32_t a, uint32_t b) {
  float x, y;
  asm("{\n .reg .b16 a, b, c, d;\n mov.b32 {a, b}, %2;\n mov.b32 {c, d}, %3;\n fma.rn.f32.bf16 %0, a, c, %4;\n"
      " fma.rn.f32.bf16 %1, b, d, %4;\n}"
      : "=f"(x), "=f"(y)
      : "r"(a), "r"(b), "f"(-0.0f));
  return pk(x, y);
}
// max(|a|, |b|, |c|), NaN above every number
FP8MOE_DEV float amax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
FP8MOE_DEV float amax3(float m, uint64_t p) {
  float a, b;
  unpk(p, a, b);
  return amax3(m, a, b);
}
// max(a, b), NaN above every number
FP8MOE_DEV float nanmax(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// MXFP8 back to values: an e8m0 byte's power of two (255 is NaN), and eight e4m3
// codes times it, as pairs; exact.
FP8MOE_DEV float mx_power(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : max(byte << 23, 0x00400000u));
}
FP8MOE_DEV uint64_t e4m3x2_f32(uint32_t c) {   // of the low 16 bits
  float x, y;
  asm("{\n .reg .b16 s, l, u;\n .reg .b32 h;\n cvt.u16.u32 s, %2;\n cvt.rn.f16x2.e4m3x2 h, s;\n mov.b32 {l, u}, h;\n"
      " cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}"
      : "=f"(x), "=f"(y)
      : "r"(c));
  return pk(x, y);
}
FP8MOE_DEV void mx_unpack8(uint2 c, float power, uint64_t (&p)[4]) {
  const uint64_t s = pk(power, power);
  p[0] = mul2(e4m3x2_f32(c.x), s), p[1] = mul2(e4m3x2_f32(c.x >> 16), s);
  p[2] = mul2(e4m3x2_f32(c.y), s), p[3] = mul2(e4m3x2_f32(c.y >> 16), s);
}
// e8m0 byte of a block maximum (the dim0 quantizer's rule on an fp32 maximum)
// and the multiplier 2^-e; infinity and NaN give a byte that no number gives
constexpr uint32_t MX_NOT_FINITE = 247;
FP8MOE_DEV uint32_t mx_byte(float amax, float& mul) {
  const uint32_t b = max(__float_as_uint(amax) >> 23, 8u) - 8u;
  mul = __uint_as_float((254u - b) << 23);
  return b;
}

}  // namespace fp8moe
