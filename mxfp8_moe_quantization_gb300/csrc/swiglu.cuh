// What the gated activation's kernels share: its arithmetic on packed pairs, the
// same for any inputs, and where rows go in layouts grouped by offsets.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"

namespace fp8moe {

// sigmoid of a pair g: 1 / D with D = 1 + 2^-t (1 - r), t = g / ln 2 rounded and
// r the rest g - t ln 2, whose exponential is 1 + r (Cody and Waite's two-part
// ln 2; |r| < 2^-17).  The reciprocal is that of D / 4, which is normal for
// every finite D, with one step of Newton's iteration.  Where e^-g is not finite
// (g below -88.72) the step's 0 * inf, and for g far up to the other side the
// infinite t, leave NaN.  Mean relative error over all bf16 |g| in (2^-10, 80)
// 3.36e-8; 1 / (1 + expf(-g)) with every step rounded 3.2e-8.
FP8MOE_DEV uint64_t sigmoid2(uint64_t g2) {
  constexpr float L = 1.44269504f, LN2_HI = 0.693147182f, LN2_LO = -1.90465421e-9f;
  const uint64_t t2 = mul2(g2, pk(L, L));
  const uint64_t r2 = fma2(t2, pk(-LN2_LO, -LN2_LO), fma2(t2, pk(-LN2_HI, -LN2_HI), g2));
  float t, u, x, y;
  unpk(t2, t, u);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(-t));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-u));
  const uint64_t d2 = fma2(pk(x, y), fma2(r2, pk(0.25f, 0.25f), pk(-0.25f, -0.25f)), pk(-0.25f, -0.25f));   // -D / 4
  unpk(d2, t, u);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(-t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-u));
  const uint64_t q2 = pk(x, y), s2 = mul2(q2, pk(0.25f, 0.25f));
  return fma2(s2, fma2(d2, q2, pk(1.0f, 1.0f)), s2);
}

// A pair of results: v, and backward the gradient of gate in v, of up in v2.
// Where sigmoid2 has no number, or a product of two inputs is beyond fp32, the
// result is not finite, by which far_tiles knows it.
template <bool BWD>
FP8MOE_DEV void act_pair(uint32_t g, uint32_t u, uint32_t d, uint64_t& v, uint64_t& v2) {
  const uint64_t g2 = unpk_bf16(g), s2 = sigmoid2(g2);
  if constexpr (BWD) {
    // 1 + g (1 - sig)
    const uint64_t f2 = fma2(g2, fma2(s2, pk(-1.0f, -1.0f), pk(1.0f, 1.0f)), pk(1.0f, 1.0f));
    v = mul2(mul2(mulx(d, u), s2), f2);
    v2 = mul2(mulx(d, g), s2);
  } else {
    v = mul2(mulx(g, u), s2);
  }
}

// act_pair on unpacked pairs, forward and backward: the activation's value returned.
FP8MOE_DEV uint64_t ckpt_pair(uint64_t g2, uint64_t u2, uint64_t d2, uint64_t& v, uint64_t& v2) {
  const uint64_t s2 = sigmoid2(g2);
  const uint64_t f2 = fma2(g2, fma2(s2, pk(-1.0f, -1.0f), pk(1.0f, 1.0f)), pk(1.0f, 1.0f));
  v = mul2(mul2(mul2(d2, u2), s2), f2);
  v2 = mul2(mul2(d2, g2), s2);
  return mul2(mul2(g2, u2), s2);
}

// The same for any inputs, from the sigmoid on in 64 bits.  Below -80 the
// sigmoid is (e^(g/4))^4, whose factors are normal as long as a result can
// differ from 0, and 0 where 64 bits have no number for it either.
FP8MOE_DEV double far_sigmoid(float g) {
  if (g < -745.0f) return 0.0;
  if (!(g < -80.0f)) return (double)__frcp_rn(1.0f + expf(-g));
  const double e = (double)expf(0.25f * fmaxf(g, -300.0f)), e2 = e * e;
  return e2 * e2;
}
template <bool BWD>
FP8MOE_DEV float far_one(float gate, float u, float d, float& du) {
  const double s = far_sigmoid(gate), g = gate;
  if constexpr (!BWD) return (float)(g * s * (double)u);
  du = (float)((double)d * g * s);
  return (float)((double)d * (double)u * s * (1.0 + g * (1.0 - s)));
}
FP8MOE_DEV bool finite2(uint64_t p) {
  float a, b;
  unpk(p, a, b);
  return amax3(0.0f, a, b) <= 3.402823466e38f;
}
template <bool BWD>
FP8MOE_DEV void far_pair(uint32_t g, uint32_t u, uint32_t d, uint64_t& v, uint64_t& v2) {
  act_pair<BWD>(g, u, d, v, v2);
  if (finite2(v) && (!BWD || finite2(v2))) return;
  float x = 0.0f, y = 0.0f;
  const float lo = far_one<BWD>(bf16_lo(g), bf16_lo(u), bf16_lo(d), x);
  const float hi = far_one<BWD>(bf16_hi(g), bf16_hi(u), bf16_hi(d), y);
  v = pk(lo, hi);
  if constexpr (BWD) v2 = pk(x, y);
}

// The padded row (in a layout whose groups start at multiples of 128 rows) of
// row `row0`, a multiple of 32; -1 if the offsets are invalid.  A warp calls
// it; each of its lanes takes every 32nd group, U of them with their loads in
// flight together.
template <int U>
FP8MOE_DEV uint32_t rows_before(const int32_t* __restrict__ offs, int E, int m, int r, int e0, bool& bad) {
  int end[U], start[U];
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int e = e0 + 32 * i;
    end[i] = e < E ? __ldg(offs + e) : 0;
    start[i] = e < E && e > 0 ? __ldg(offs + e - 1) : 0;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int e = e0 + 32 * i;
    if (e >= E) break;
    bad |= start[i] < 0 || end[i] < start[i] || end[i] > m || (end[i] & 31) || (e == E - 1 && end[i] != m);
    if (end[i] <= r) {
      sum += ((uint32_t)(end[i] - start[i]) + 127u) & ~127u;
    } else if (start[i] <= r) {
      sum += (uint32_t)(r - start[i]);
    }
  }
  return sum;
}
FP8MOE_DEV int64_t padded_row(const int32_t* __restrict__ offs, int E, int64_t M, int64_t row0, int lane) {
  const int m = (int)M, r = (int)row0;   // both at most 2^30
  uint32_t sum = 0;
  bool bad = false;
  if (E <= 32) {
    sum = rows_before<1>(offs, E, m, r, lane, bad);
  } else {
    for (int e0 = lane; e0 < E; e0 += 256) sum += rows_before<8>(offs, E, m, r, e0, bad);
  }
  if (__any_sync(0xffffffffu, bad)) return -1;
  return (int64_t)__reduce_add_sync(0xffffffffu, sum);
}

// One step of a maximum over lanes that differ in `mask`: the lower lane goes
// on with the first half of m, the upper one with the second.
template <int N>
FP8MOE_DEV void halve(const float (&m)[N], float (&out)[N / 2], int lane, int mask) {
  const bool up = lane & mask;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float other = __shfl_xor_sync(0xffffffffu, up ? m[i] : m[i + N / 2], mask);
    out[i] = nanmax(up ? m[i + N / 2] : m[i], other);
  }
}

}  // namespace fp8moe
