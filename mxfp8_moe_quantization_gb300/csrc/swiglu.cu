// Gated activation between the two expert products, with MXFP8 output along
// both dimensions, and its backward.
//
//   forward:  a = g * sig(g) * u                     (h = [g | u], fp32)
//   backward: dg = d * u * sig(g) * (1 + g (1 - sig(g))),  du = d * g * sig(g)
// Each result is written as bf16 and / or as MXFP8 blocks along its rows (the
// next product's operand) and along its columns, transposed (the operand of
// the product that contracts over the tokens), with the scales in the layouts
// the grouped GEMM reads.  The codes come from the fp32 results: one rounding.
//
// A warp holds a tile of 32 rows x 64 columns, a lane 8 rows x 8 columns
// as pairs of neighbouring columns, on which the packed fp32 instructions
// work.  A block's maximum is reduced and scattered in one go (each step
// halves the rows, or columns, a lane still looks after), so a lane derives
// one or two scales instead of every lane every one; the multipliers come
// back by shuffles.  The conversions along a column take neighbouring rows
// from the lane's registers, so the transposed codes need no byte transposes.
//
// Bound by HBM: 6.06 bytes per element forward, 10.1 backward.  Measured: 36448
// x 2048 in 256 groups forward, both directions, 72 us = 6.3 TB/s (94% of a
// copy's rate); 51136 x 1408 backward 120 us = 6.1 TB/s (91%).  The first form,
// with every lane deriving every scale, expf and a division, and 45
// instructions per element instead of about 20, took 152 and 283 us.
#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"
#include "moe_ops.h"
#include "mxcvt.cuh"
#include "scales.cuh"
#include "tma.cuh"

namespace fp8moe {
namespace {

// A warp's tile, and a CTA's: 2 x 2 warps, 64 rows x 128 columns.  (4 x 1 warps
// read 128 bytes of a row at a time: 2 to 4% longer, 16 to 0% shorter only where
// half of the last tile of few is empty; 1 x 2 the same as 2 x 2.)
constexpr int SG_ROWS = 32, SG_COLS = 64, SG_RW = 2, SG_CW = 2, SG_WARPS = SG_RW * SG_CW;
constexpr int CW = 8;   // columns per lane

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

// Where a warp's 32 rows go.  Scale bytes: row 8 rq + i, block c of s0 is at
// s0 + i * step0 + off0(c); column c of s1 at s1 + off1(c).
struct TilePlace {
  int row0;       // first row of the tile
  int W;          // columns of the result
  uint8_t *s0, *s1;
  int64_t step0;  // row-major: W / 32; tiled: 16
  int64_t band1;  // tiled s1: bytes of 128 of its rows; row-major: 0
};

// prow0, pcol1: the tile's first row in s0's layout, its column in s1's
FP8MOE_DEV void place_scales(const SwigluArgs& a, TilePlace& tp, int64_t prow0, int64_t pcol1, int64_t cp0, int64_t cp1,
                             int rq) {
  const bool t0 = a.s0_layout != FP8MOE_SCALES_ROWMAJOR, t1 = a.s1_layout != FP8MOE_SCALES_ROWMAJOR;
  tp.step0 = t0 ? 16 : tp.W / 32;
  tp.s0 = a.s0 + (t0 ? tile_off(prow0, 0, cp0) : (int64_t)tp.row0 * (tp.W / 32)) + rq * 8 * tp.step0;
  tp.band1 = t1 ? cp1 * 128 : 0;
  tp.s1 = a.s1 + (t1 ? (pcol1 >> 2) * 512 + (pcol1 & 3) : tp.row0 / 32);
}

// One tile of results to every output.  v: rows 8 rq .. 8 rq + 7 and columns
// CW cq .. of the tile, as column pairs; col0: the tile's first column; ok:
// this lane's columns exist; top: the largest scale byte that the lane derived
// (the lanes together derive every block's).
FP8MOE_DEV void put_tile(const SwigluArgs& a, const TilePlace& tp, int64_t col0, bool ok, int lane,
                         const uint64_t (&v)[8][CW / 2], uint32_t& top) {
  const int rq = lane >> 3, cq = lane & 7;
  const int64_t W = tp.W, col = col0 + cq * CW, rbase = (int64_t)tp.row0 + rq * 8;
  const int rows = rbase + 8 <= a.M ? 8 : rbase < a.M ? (int)(a.M - rbase) : 0;
  if (a.out && ok) {
    uint16_t* o = a.out + rbase * W + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= rows) break;
      *reinterpret_cast<uint4*>(o + i * W) = make_uint4(pack_bf16x2(v[i][0]), pack_bf16x2(v[i][1]),
                                                        pack_bf16x2(v[i][2]), pack_bf16x2(v[i][3]));
    }
  }
  if (!a.q0 && !a.q1) {
    float m = 0.0f, s;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int p = 0; p < CW / 2; ++p) m = amax3(m, v[i][p]);
    top = max(top, mx_byte(m, s));
  }
  if (a.q0) {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = 0.0f;
#pragma unroll
      for (int p = 0; p < CW / 2; ++p) {
        m[i] = amax3(m[i], v[i][p]);
      }
    }
    // a row block is the four lanes that differ in cq's low bits; a lane ends
    // with rows own and own + 1
    float m4[4], mk[2], mul[2];
    halve<8>(m, m4, lane, 1);
    halve<4>(m4, mk, lane, 2);
    const int own = (lane & 1) * 4 + (lane & 2);
    const int64_t blk = col >> 5;
    const int64_t c0 = a.s0_layout != FP8MOE_SCALES_ROWMAJOR ? (blk >> 2) * 512 + (blk & 3) : blk;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t b = mx_byte(mk[s], mul[s]);
      const int i = own + s;
      top = max(top, b);
      if (ok && i < rows) tp.s0[i * tp.step0 + c0] = (uint8_t)b;
    }
    uint8_t* q = a.q0 + rbase * W + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = __shfl_sync(0xffffffffu, mul[i & 1], (lane & ~3) | (i >> 2) | (i & 2));
      const uint64_t s2 = pk(s, s);
      float f[CW];
#pragma unroll
      for (int p = 0; p < CW / 2; ++p) unpk(mul2(v[i][p], s2), f[2 * p], f[2 * p + 1]);
      if (ok && i < rows)
        *reinterpret_cast<uint2*>(q + i * W) = make_uint2(cvt4(f[0], f[1], f[2], f[3]), cvt4(f[4], f[5], f[6], f[7]));
    }
  }
  if (a.q1) {   // M % 32 == 0: every row exists
    float m[CW];
#pragma unroll
    for (int p = 0; p < CW / 2; ++p) {
      m[2 * p] = m[2 * p + 1] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float x, y, z, w;
        unpk(v[i][p], x, y);
        unpk(v[i + 1][p], z, w);
        m[2 * p] = amax3(m[2 * p], x, z);
        m[2 * p + 1] = amax3(m[2 * p + 1], y, w);
      }
    }
    // a column block is the four lanes that differ in rq; a lane ends with
    // columns own and own + 1
    float mh[4], mk[2], mul[2];
    halve<8>(m, mh, lane, 8);
    halve<4>(mh, mk, lane, 16);
    const int own = ((lane >> 3) & 1) * 4 + ((lane >> 4) & 1) * 2;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t b = mx_byte(mk[s], mul[s]);
      const int64_t c = col + own + s;
      top = max(top, b);
      if (ok)
        tp.s1[tp.band1 ? (c >> 7) * tp.band1 + (c & 31) * 16 + ((c >> 5) & 3) * 4 : c * (a.M / 32)] = (uint8_t)b;
    }
    uint8_t* q = a.q1 + col * a.M + rbase;
#pragma unroll
    for (int p = 0; p < CW / 2; ++p) {
      // columns 2 p and 2 p + 1 are the two of one lane
      const int src = (lane & 7) | (p >> 1) << 3 | (p & 1) << 4;
      const float sc0 = __shfl_sync(0xffffffffu, mul[0], src), sc1 = __shfl_sync(0xffffffffu, mul[1], src);
      const uint64_t s2 = pk(sc0, sc1);
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) unpk(mul2(v[i][p], s2), x[i], y[i]);
      if (ok) {
        *reinterpret_cast<uint2*>(q + (2 * p) * a.M) = make_uint2(cvt4(x[0], x[1], x[2], x[3]), cvt4(x[4], x[5], x[6], x[7]));
        *reinterpret_cast<uint2*>(q + (2 * p + 1) * a.M) =
            make_uint2(cvt4(y[0], y[1], y[2], y[3]), cvt4(y[4], y[5], y[6], y[7]));
      }
    }
  }
}

// Shared memory of a warp with PF: one 32 x 64 box each of gate, up and, backward,
// dout, rows of 128 bytes.
constexpr int BOX_BYTES = SG_ROWS * SG_COLS * 2;
template <bool BWD>
constexpr int warp_bytes() { return (BWD ? 3 : 2) * BOX_BYTES; }
template <bool BWD>
constexpr int cta_bytes() { return SG_WARPS * (warp_bytes<BWD>() + 8); }   // + a barrier per warp

// A warp's `n` tiles from `row`, `col` on once more, if one of them has a result
// that is not finite (gates below -88.72, NaN, infinities, products beyond
// fp32): every result by far_pair, from memory, over what stands there (from the
// same lane).  After the run, when nothing else is live: inside it, or with a
// flag of its own beside the scale bytes, 51136 x 1408 backward took 131 to 152
// us without any such tile.  With such gates in 1 column of 2048, 36448 rows
// take 127 us forward instead of 76, 248 instead of 128 backward.
template <bool BWD>
FP8MOE_DEV void far_tiles(const SwigluArgs& a, TilePlace tp, int64_t row, int64_t col, int n, int col_end, int64_t cp0,
                          int64_t cp1) {
  const int lane = threadIdx.x & 31, rq = lane >> 3, cq = lane & 7;
#pragma unroll 1
  for (; n > 0 && row < a.M; --n) {
    if (col < a.F) {
      const int64_t pr = a.E0 + a.E1 > 0 ? padded_row(a.offs, a.E0 > 0 ? a.E0 : a.E1, a.M, row, lane) : row;
      tp.row0 = (int)row;
      place_scales(a, tp, a.E0 > 0 ? pr : row, (a.E1 > 0 ? pr : row) / 32, cp0, cp1, rq);
      const int64_t c = col + cq * CW;
      const bool ok = c < a.F;
      uint64_t v[8][CW / 2], v2[BWD ? 8 : 1][CW / 2];
      uint32_t top = 0;
      // one pair at a time: 32 copies of far_pair do not stay in the instruction cache
#pragma unroll 1
      for (int k = 0; k < 8 * (CW / 2); ++k) {
        const int64_t r = row + rq * 8 + k / (CW / 2), at = c + k % (CW / 2) * 2;
        const bool on = ok && r < a.M;
        auto pair = [&](const uint16_t* p) { return on ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u; };
        uint64_t x, y;
        far_pair<BWD>(pair(a.h + r * a.ldh + at), pair(a.h + r * a.ldh + a.F + at), BWD ? pair(a.dout + r * a.F + at) : 0u, x, y);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int p = 0; p < CW / 2; ++p) {
            if (k != i * (CW / 2) + p) continue;
            v[i][p] = x;
            if constexpr (BWD) v2[i][p] = y;
          }
      }
      put_tile(a, tp, col, ok, lane, v, top);
      if constexpr (BWD) put_tile(a, tp, a.F + col, ok, lane, v2, top);
    }
    // the next tile of the run
    col += SG_CW * SG_COLS;
    if (col >= col_end) {
      col -= col_end;
      row += SG_RW * SG_ROWS;
    }
  }
}

// PF: a CTA walks a contiguous run of tiles, column tiles fastest, and each of
// its warps has the next tile's boxes loaded by TMA while it works on the
// current one from registers.  Without PF every CTA has one tile (few tiles:
// nothing to overlap), loaded straight into registers.
template <bool BWD, bool PF>
FP8MOE_DEV void swiglu_body(const CUtensorMap* th, const CUtensorMap* td, const SwigluArgs& a, int64_t cp0, int64_t cp1,
                            int col_tiles, int tiles, int per) {
  extern __shared__ __align__(128) uint8_t dsm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rq = lane >> 3, cq = lane & 7;
  uint8_t* wbuf = dsm + warp * warp_bytes<BWD>();
  uint64_t* wbar = reinterpret_cast<uint64_t*>(dsm + SG_WARPS * warp_bytes<BWD>()) + warp;
  // the CTA's run of tiles, and a tile's place stepped along it
  const int t0 = blockIdx.x * per, t1 = tiles - t0 < per ? tiles : t0 + per;
  struct Place {
    int row;
    int col;
  };
  auto first = [&](int t) {
    const int rb = t / col_tiles;
    return Place{(rb * SG_RW + warp % SG_RW) * SG_ROWS, ((t - rb * col_tiles) * SG_CW + warp / SG_RW) * SG_COLS};
  };
  const int col_end = col_tiles * SG_CW * SG_COLS;
  auto next = [&](Place p) {
    p.col += SG_CW * SG_COLS;
    if (p.col >= col_end) {
      p.col -= col_end;
      p.row += SG_RW * SG_ROWS;
    }
    return p;
  };
  // the tile's boxes (one lane); a warp whose rows lie past M loads nothing
  auto issue = [&](const Place& p) {
    const int64_t r = p.row;
    const int c = p.col;
    if (r >= a.M || c >= a.F || (a.stall && blockIdx.x == 0 && warp == 0)) return;
    mbar_expect_tx(wbar, warp_bytes<BWD>());
    tma_load_2d(wbuf, th, wbar, c, (int)r);
    tma_load_2d(wbuf + BOX_BYTES, th, wbar, (int)a.F + c, (int)r);
    if (BWD) tma_load_2d(wbuf + 2 * BOX_BYTES, td, wbar, c, (int)r);
  };
  Place cur = first(t0);
  if (PF) {
    if (lane == 0) {
      mbar_init(wbar, 1);
      mbar_fence_init();
      issue(cur);
    }
    __syncwarp();
  }
  TilePlace tp;
  tp.W = (int)(BWD ? 2 * a.F : a.F);
  tp.row0 = -1;
  uint32_t parity = 0, top = 0;
  for (int t = t0; t < t1; ++t) {
    const int row0 = cur.row;
    if (row0 >= a.M) break;   // column tiles are fastest: the later tiles' rows are not lower
    const int64_t col0 = cur.col, col = col0 + cq * CW;
    cur = next(cur);
    if (col0 >= a.F) {   // this warp's half of the last column tile is empty
      if (PF && lane == 0 && t + 1 < t1) issue(cur);
      continue;
    }
    const bool ok = col < a.F;
    const bool moved = row0 != tp.row0;
    tp.row0 = row0;
    uint4 g[PF ? 1 : 8], u[PF ? 1 : 8], d[PF || !BWD ? 1 : 8];
    if constexpr (!PF) {
      const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = (int64_t)row0 + rq * 8 + i;
        const bool on = ok && r < a.M;
        g[i] = on ? ld_nc16(a.h + r * a.ldh + col) : z;
        u[i] = on ? ld_nc16(a.h + r * a.ldh + a.F + col) : z;
        if constexpr (BWD) d[i] = on ? ld_nc16(a.dout + r * a.F + col) : z;
      }
    }
    bool fail = false;
    if (moved) {   // the loads are in flight meanwhile
      int64_t pr = row0;
      if (a.E0 + a.E1 > 0) {
        pr = padded_row(a.offs, a.E0 > 0 ? a.E0 : a.E1, a.M, row0, lane);
        if (pr < 0) {
          if (lane == 0) set_status(a.status, FP8MOE_ERR_DEVICE_OFFSETS);
          fail = true;
        }
      }
      place_scales(a, tp, a.E0 > 0 ? pr : row0, (a.E1 > 0 ? pr : row0) / 32, cp0, cp1, rq);
    }
    if (PF) {
      // (also before leaving on bad offsets: no load stays in flight)
      if (!mbar_wait(wbar, parity, nullptr)) {
        set_status(a.status, FP8MOE_ERR_TIMEOUT);
        (void)mbar_wait(wbar, parity, nullptr);   // the late copies, again with a limit
        fail = true;
      }
      parity ^= 1;
    }
    if (fail) break;
    uint64_t v[8][CW / 2], v2[BWD ? 8 : 1][CW / 2];
    const uint8_t* lp = wbuf + rq * 8 * 128 + cq * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 gq = PF ? *reinterpret_cast<const uint4*>(lp + i * 128) : g[PF ? 0 : i];
      const uint4 uq = PF ? *reinterpret_cast<const uint4*>(lp + BOX_BYTES + i * 128) : u[PF ? 0 : i];
      uint4 dq = make_uint4(0, 0, 0, 0);
      if constexpr (BWD) dq = PF ? *reinterpret_cast<const uint4*>(lp + 2 * BOX_BYTES + i * 128) : d[PF ? 0 : i];
      const uint32_t gw[4] = {gq.x, gq.y, gq.z, gq.w}, uw[4] = {uq.x, uq.y, uq.z, uq.w};
      const uint32_t dw[4] = {dq.x, dq.y, dq.z, dq.w};
#pragma unroll
      for (int p = 0; p < CW / 2; ++p) {
        act_pair<BWD>(gw[p], uw[p], dw[p], v[i][p], v2[BWD ? i : 0][p]);
      }
    }
    if (PF) {
      __syncwarp();   // the boxes are read
      if (lane == 0 && t + 1 < t1) {
        fence_proxy_async_smem();
        issue(cur);
      }
    }
    put_tile(a, tp, col0, ok, lane, v, top);
    if constexpr (BWD) put_tile(a, tp, a.F + col0, ok, lane, v2, top);
  }
  if (__any_sync(0xffffffffu, top == MX_NOT_FINITE)) {
    const Place p = first(t0);
    far_tiles<BWD>(a, tp, p.row, p.col, t1 - t0, col_end, cp0, cp1);
  }
}

template <bool BWD>
__global__ void __launch_bounds__(SG_WARPS * 32, BWD ? 3 : 4)
    k_swiglu_run(const __grid_constant__ CUtensorMap th, const __grid_constant__ CUtensorMap td, SwigluArgs a, int64_t cp0,
                 int64_t cp1, int col_tiles, int tiles, int per) {
  swiglu_body<BWD, true>(&th, &td, a, cp0, cp1, col_tiles, tiles, per);
}
template <bool BWD>
__global__ void __launch_bounds__(SG_WARPS * 32)
    k_swiglu_few(SwigluArgs a, int64_t cp0, int64_t cp1, int col_tiles, int tiles) {
  swiglu_body<BWD, false>(nullptr, nullptr, a, cp0, cp1, col_tiles, tiles, 1);
}

// Tiles per CTA, of which an SM holds occ at a time.  With many a CTA takes
// two: one exposes its first load and group lookup, longer runs wait for the
// slowest (51136 x 1408 backward: 123.5 us with one, 115.8 two, 117.3 three, 120
// four, 126.6 six).  With few it is the last round of CTAs that counts, where an
// SM may have one CTA left: what leaves the shortest sum over the rounds, a
// tile taking as long as k CTAs on an SM share it but at least 2.1 of that
// (46720 x 192 backward, 1460 tiles: 21.1 us with two, 27.5 with three; 4096 x 4096
// backward, 2048 tiles: 35.3 and, with five, 32.2; 38176 x 288 forward, 1791
// tiles: 12.2 with three, 16.0 with two).
int64_t tiles_per_cta(int64_t tiles, int64_t num_sms, int64_t occ) {
  const int64_t fit = num_sms * occ;
  if (tiles > 6 * fit) return 2;
  int64_t best = 1, least = INT64_MAX;
  for (int64_t per = 1; per <= 5; ++per) {
    const int64_t n = (tiles + per - 1) / per, rest = n % fit, k = (rest + num_sms - 1) / num_sms;
    const int64_t cost = n / fit * (per * 10 * occ + 5) + (rest ? per * (k > 2 ? 10 * k : 21) + 5 : 0);
    if (cost < least) least = cost, best = per;
  }
  return best;
}

template <bool BWD>
cudaError_t launch_dir(SwigluArgs a, cudaStream_t st) {
  const int64_t W = BWD ? 2 * a.F : a.F;
  const int64_t cp0 = (W / 32 + 3) / 4 * 4;
  const int64_t cp1 = (a.M / 32 + 3) / 4 * 4 + (int64_t)a.E1 * 4;
  const int64_t col_tiles = (a.F + SG_COLS * SG_CW - 1) / (SG_COLS * SG_CW);
  const int64_t tiles = (a.M + SG_ROWS * SG_RW - 1) / (SG_ROWS * SG_RW) * col_tiles;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  // Fewer tiles than SMs: straight into registers, without the boxes' barrier
  // and descriptors (16 tiles: 3.6 us forward and 5.5 backward against 3.8 and
  // 5.9; no difference at 256).  A box is not wider than a result row.
  if (tiles <= a.num_sms || a.F < SG_COLS) {
    k_swiglu_few<BWD><<<(unsigned)tiles, SG_WARPS * 32, 0, st>>>(a, cp0, cp1, (int)col_tiles, (int)tiles);
    return cudaGetLastError();
  }
  CUtensorMap th{}, td{};
  cudaError_t e = cudaFuncSetAttribute(k_swiglu_run<BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, cta_bytes<BWD>());
  if (e != cudaSuccess) return e;
  static std::atomic<int> occ{0};
  const int64_t per_sm = blocks_per_sm(occ, k_swiglu_run<BWD>, SG_WARPS * 32, cta_bytes<BWD>(), 1);
  a.stall = take_ring_stall_hook();
  cuuint64_t dims[2] = {(cuuint64_t)(2 * a.F), (cuuint64_t)a.M}, strides[1] = {(cuuint64_t)(a.ldh * 2)};
  const cuuint32_t box[2] = {SG_COLS, SG_ROWS};
  if (!make_tmap(&th, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.h, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  if (BWD) {
    dims[0] = (cuuint64_t)a.F;
    strides[0] = (cuuint64_t)(a.F * 2);
    if (!make_tmap(&td, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.dout, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  }
  const int64_t per = tiles_per_cta(tiles, a.num_sms, per_sm);
  k_swiglu_run<BWD><<<(unsigned)((tiles + per - 1) / per), SG_WARPS * 32, cta_bytes<BWD>(), st>>>(
      th, td, a, cp0, cp1, (int)col_tiles, (int)tiles, (int)per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t st) {
  return a.dout ? launch_dir<true>(a, st) : launch_dir<false>(a, st);
}

}  // namespace fp8moe
