// Backward of the gated activation from an MXFP8 checkpoint of its input, with
// MXFP8 output along both dimensions, and the activation of the checkpoint's values
// along its columns: the operand of the second product's weight gradient.
//
//   g, u = code * 2^e;  dg = d * u * sig(g) * (1 + g (1 - sig(g))),  du = d * g * sig(g),  a = g * sig(g) * u
// The arithmetic is the bf16 form's (swiglu.cuh), and so are the results' bits.
//
// A warp's tile is 32 x 32, a lane's 8 x 4 (the bf16 form's is twice as wide): a block
// of a row is one warp's eight lanes, so that its scale is read once a row, and three
// warps a scheduler have room for a tile's values and for the next tile, whose loads are
// on their way while this one's gradients go out.  A CTA is a warp: nothing is shared,
// and the last round is the shorter.  Its tiles follow a row, four of them, whose scales
// are then read and written as a word, as each row's lie in a sector of their own.  Maxima
// go through the lanes two in a word.  (51136 x 1408 with a cold L2: 223 us without the
// next tile's loads, 164 with single scale bytes and four warps a CTA, 159 with words, 155
// with a warp a CTA, 151 with maxima in pairs; twelve warps a CTA 177.)
//
// Nothing is saturated: three warps a scheduler, all that the registers leave, issue 0.55
// instructions a cycle, 44 an element of a (five block scalings, the unpacking and the
// sigmoid), and wait in between for loads, shuffles and an SM's memory pipe, which takes
// every 32 bytes apart that a store's lanes have in one row or column, and is 64% busy.
// HBM's 9.2 bytes an element would take 100 us; measured, among other passes: 51136 x 1408
// in 64 groups, all outputs, 147 us = 4.5 TB/s (67% of a copy's rate).  Without the
// activation 119 us, as the bf16 form (its boxes by TMA), for 8.1 bytes against 10.1.
#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"
#include "moe_ops.h"
#include "mxcvt.cuh"
#include "scales.cuh"
#include "swiglu.cuh"

namespace fp8moe {
namespace {

// Warps an SM: without the activation 128 registers do (120 us, 123 with twelve warps).
template <bool ACT>
constexpr int sc_warps() { return ACT ? 12 : 16; }
constexpr int CP = 2;                // column pairs of a lane

// i rows of `stride` elements: a product of 32-bit factors (sizes are below 2^30)
FP8MOE_DEV uint64_t wide(uint32_t stride, uint32_t i) { return (uint64_t)stride * i; }

// A lane's place in every tensor at column 0 (bases come from the arguments, so that
// few addresses stay in registers).  It has rows 8 rq .. of the warp's 32 and columns
// 4 cq .. of a tile.
struct Rows {
  uint32_t F, M;
  int rows;            // of the lane's eight, those that exist
  uint64_t at;         // in hq and q0; twice that in out, 4 cq more in dout (bytes)
  uint64_t at_h;       // scales of h: of row `lane` of the tile
  uint64_t at_s0;
  uint32_t step0;
  uint64_t at1;        // in q1 and aq1
  uint64_t at_s1;      // in s1 and as1: of the tile's block of rows
  uint32_t band1;      // 128 columns' scales, in units of 128 bytes, 0: row-major
  bool has_scale, tiled0;
  bool h_words, s0_words;   // four neighbouring scales of a row are an aligned word: of h, of q0
};

// Row scales on their way out: four of a row are written together, as each row's lie
// in a sector of their own.
struct RowScales {
  uint32_t word = 0, have = 0;   // bytes of a word, and which
};

// Bytes from s1 to the scale of lane-column j (below 32) of a tile at column `col`.
FP8MOE_DEV uint64_t column_scale(const Rows& r, uint32_t col, uint32_t j) {
  return r.at_s1 + (r.band1 ? wide(r.band1, col >> 7) * 128 + (col >> 5 & 3u) * 4 + j * 16 : wide(r.M / 32, col + j));
}

// Maxima on their way through the lanes, two in a word: a block's scale hangs on the upper
// halves of their fp32 words only (NaN is the largest, infinity next).
FP8MOE_DEV uint32_t upper2(float lo, float hi) { return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632); }
// One step over lanes that differ in `mask`, as halve()
template <int N>
FP8MOE_DEV void halve2(const uint32_t (&m)[N], uint32_t (&out)[N / 2], int lane, int mask) {
  const bool up = lane & mask;
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    out[i] = umax16x2(up ? m[i + N / 2] : m[i], __shfl_xor_sync(0xffffffffu, up ? m[i] : m[i + N / 2], mask));
}
// The last step: a lane goes on with one of the two.
FP8MOE_DEV uint32_t halve1(uint32_t m, int lane, int mask) {
  m = umax16x2(m, __shfl_xor_sync(0xffffffffu, m, mask));
  return lane & mask ? m >> 16 : m & 0xFFFFu;
}
// mx_byte of an upper half
FP8MOE_DEV uint32_t mx_byte16(uint32_t h, float& mul) { return mx_byte(__uint_as_float(h << 16), mul); }

// Codes and scales along the rows: v's columns are those from `col` of 2F.
template <bool ALL>
FP8MOE_DEV void put_rows(const SwigluArgs& a, const Rows& r, uint32_t col, int lane, const uint64_t (&v)[8][CP], RowScales& sc,
                         bool last, uint32_t& top) {
  const int cq = lane & 7;
  float m[8], mul;
  uint32_t w4[4], w2[2], w1[1];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = amax3(amax3(0.0f, v[i][0]), v[i][1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) w4[i] = upper2(m[2 * i], m[2 * i + 1]);
  // a row's block is the eight lanes of a row group; a lane ends with row `own`
  halve2<4>(w4, w2, lane, 1);
  halve2<2>(w2, w1, lane, 2);
  const int own = (cq & 1) * 4 + (cq & 2) + (cq >> 2);
  const uint32_t b = mx_byte16(halve1(w1[0], lane, 4), mul), blk = col >> 5;
  top = max(top, b);
  uint8_t* s0 = a.s0 + r.at_s0 + (uint32_t)own * r.step0 + (r.tiled0 ? (blk >> 2) * 512 : blk & ~3u);
  sc.word |= b << (blk & 3) * 8;
  sc.have |= 1u << (blk & 3);
  if (last || !r.s0_words || (blk & 3) == 3) {
    if (ALL || own < r.rows) {
      if (r.s0_words && sc.have == 15u) {
        *reinterpret_cast<uint32_t*>(s0) = sc.word;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (sc.have >> i & 1u) s0[i] = (uint8_t)(sc.word >> 8 * i);
      }
    }
    sc = RowScales{};
  }
  uint8_t* q = a.q0 + r.at + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = __shfl_sync(0xffffffffu, mul, (lane & ~7) | (i >> 2) | (i & 2) | (i & 1) << 2);
    float f[4];
    unpk(mul2(v[i][0], pk(s, s)), f[0], f[1]);
    unpk(mul2(v[i][1], pk(s, s)), f[2], f[3]);
    if (ALL || i < r.rows) *reinterpret_cast<uint32_t*>(q + wide(2 * r.F, i)) = cvt4(f[0], f[1], f[2], f[3]);
  }
}

// Codes and scales along the columns from `col` on, transposed (M % 32 == 0: every
// row exists).
FP8MOE_DEV void put_columns(const Rows& r, uint8_t* q1, uint8_t* s1, uint32_t col, int lane, const uint64_t (&v)[8][CP],
                            uint32_t& top) {
  float m[4], mul;
#pragma unroll
  for (int p = 0; p < CP; ++p) {
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
  // a column's block is the four lanes that differ in the row group; a lane ends
  // with column `own`
  const uint32_t w2[2] = {upper2(m[0], m[1]), upper2(m[2], m[3])};
  uint32_t w1[1];
  halve2<2>(w2, w1, lane, 8);
  const uint32_t own = (uint32_t)(((lane >> 3) & 1) * 2 + (lane >> 4)), b = mx_byte16(halve1(w1[0], lane, 16), mul);
  top = max(top, b);
  s1[column_scale(r, col, (lane & 7) * 4 + own)] = (uint8_t)b;
  uint8_t* q = q1 + r.at1 + wide(r.M, col);
#pragma unroll
  for (int p = 0; p < CP; ++p) {
    const int src = (lane & 7) | p << 3;   // column 2 p's lane; 2 p + 1's is 16 further
    const float k0 = __shfl_sync(0xffffffffu, mul, src), k1 = __shfl_sync(0xffffffffu, mul, src | 16);
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) unpk(v[i][p], x[i], y[i]);
    *reinterpret_cast<uint2*>(q + wide(r.M, 2 * p)) =
        make_uint2(cvt4(x[0] * k0, x[1] * k0, x[2] * k0, x[3] * k0), cvt4(x[4] * k0, x[5] * k0, x[6] * k0, x[7] * k0));
    *reinterpret_cast<uint2*>(q + wide(r.M, 2 * p + 1)) =
        make_uint2(cvt4(y[0] * k1, y[1] * k1, y[2] * k1, y[3] * k1), cvt4(y[4] * k1, y[5] * k1, y[6] * k1, y[7] * k1));
  }
}

// The same of one column pair, p: its block's four lanes each take its maximum and
// scale, and one keeps it in `mine`: that of column 4 (lane & 7) + (lane >> 3).
FP8MOE_DEV void put_pair(const Rows& r, uint8_t* q1, uint32_t col, int p, int lane, const uint64_t (&v)[8], uint32_t& mine,
                         uint32_t& top) {
  float m0 = 0.0f, m1 = 0.0f, k0, k1, x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) unpk(v[i], x[i], y[i]);
#pragma unroll
  for (int i = 0; i < 8; i += 2) m0 = amax3(m0, x[i], x[i + 1]), m1 = amax3(m1, y[i], y[i + 1]);
  uint32_t m = upper2(m0, m1);
  m = umax16x2(m, __shfl_xor_sync(0xffffffffu, m, 8));
  m = umax16x2(m, __shfl_xor_sync(0xffffffffu, m, 16));
  const uint32_t b0 = mx_byte16(m & 0xFFFFu, k0), b1 = mx_byte16(m >> 16, k1);
  top = max(top, max(b0, b1));
  uint8_t* q = q1 + r.at1 + wide(r.M, col + 2 * p);
  *reinterpret_cast<uint2*>(q) =
      make_uint2(cvt4(x[0] * k0, x[1] * k0, x[2] * k0, x[3] * k0), cvt4(x[4] * k0, x[5] * k0, x[6] * k0, x[7] * k0));
  *reinterpret_cast<uint2*>(q + r.M) =
      make_uint2(cvt4(y[0] * k1, y[1] * k1, y[2] * k1, y[3] * k1), cvt4(y[4] * k1, y[5] * k1, y[6] * k1, y[7] * k1));
  if (lane >> 4 == p) mine = lane & 8 ? b1 : b0;
}

// One of the two gradients to every output but the activation's.
template <bool ALL>
FP8MOE_DEV void put_gradient(const SwigluArgs& a, const Rows& r, uint32_t col, int lane, const uint64_t (&v)[8][CP], RowScales& sc,
                             bool last, uint32_t& top) {
  if (a.out) {
    uint16_t* o = a.out + r.at + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (ALL || i < r.rows)
        *reinterpret_cast<uint2*>(o + wide(2 * r.F, i)) = make_uint2(pack_bf16x2(v[i][0]), pack_bf16x2(v[i][1]));
  }
  if (a.q0) put_rows<ALL>(a, r, col, lane, v, sc, last, top);
  if (a.q1) put_columns(r, a.q1, a.s1, col, lane, v, top);
  if (!a.q0 && !a.q1) {
    float m = 0.0f, s;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = amax3(amax3(m, v[i][0]), v[i][1]);
    top = max(top, mx_byte(m, s));
  }
}

// A warp's tile as it is in memory; sg, su: the scales of row `lane`, of this tile or
// (h_words) of the four blocks that it is one of.
struct Tile {
  uint32_t g[8], u[8], sg, su;
  uint2 d[8];
};
FP8MOE_DEV const uint16_t* dout_at(const SwigluArgs& a, const Rows& r, uint32_t col, int lane) {
  return reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(a.dout) + r.at + (lane & 7) * 4) + col;
}
FP8MOE_DEV void load_scales(const SwigluArgs& a, const Rows& r, uint32_t col, uint32_t& sg, uint32_t& su) {
  const uint8_t* s = a.hs + r.at_h;
  sg = r.has_scale ? __ldg(s + (col >> 5)) : 0u;
  su = r.has_scale ? __ldg(s + ((r.F + col) >> 5)) : 0u;
}
template <bool ALL>
FP8MOE_DEV void load(const SwigluArgs& a, const Rows& r, uint32_t col, int lane, bool first, Tile& t) {
  const uint8_t *g = a.hq + r.at + col, *u = g + r.F;
  const uint16_t* d = dout_at(a, r, col, lane);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool on = ALL || i < r.rows;
    t.g[i] = on ? __ldg(reinterpret_cast<const uint32_t*>(g + wide(2 * r.F, i))) : 0u;
    t.u[i] = on ? __ldg(reinterpret_cast<const uint32_t*>(u + wide(2 * r.F, i))) : 0u;
    t.d[i] = on ? __ldg(reinterpret_cast<const uint2*>(d + wide(r.F, i))) : make_uint2(0, 0);
  }
  if (!r.h_words) {
    load_scales(a, r, col, t.sg, t.su);
  } else if (first || (col & 127) == 0) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(a.hs + r.at_h) + (col >> 7);
    t.sg = r.has_scale ? __ldg(s) : 0u;
    t.su = r.has_scale ? __ldg(s + (r.F >> 7)) : 0u;
  }
}
// Two scales' powers of two in a word: they are upper halves of their fp32 words.
FP8MOE_DEV uint32_t powers(uint32_t sg, uint32_t su) {
  return __float_as_uint(mx_power(sg)) >> 16 | __float_as_uint(mx_power(su));
}
FP8MOE_DEV float power_of_gate(uint32_t w) { return __uint_as_float(w << 16); }
FP8MOE_DEV float power_of_up(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The warp's tiles from column `col` up to column `end`; the next tile's loads are on
// their way while the gradients go out.
template <bool ACT, bool ALL>
FP8MOE_DEV uint32_t tiles(const SwigluArgs& a, const Rows& r, uint32_t col, uint32_t end, int lane) {
  const int rq = lane >> 3;
  uint32_t top = 0;
  Tile t;
  RowScales sc, sc2;
  if (col < end) load<ALL>(a, r, col, lane, true, t);
#pragma unroll 1
  while (col < end) {
    uint64_t v[8][CP], v2[8][CP];
    uint32_t w[8];
    const uint32_t at = r.h_words ? (col >> 5 & 3) * 8 : 0, pw = powers(t.sg >> at & 255u, t.su >> at & 255u);
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __shfl_sync(0xffffffffu, pw, rq * 8 + i);
    // column pair by column pair: the activation's values go to their codes at
    // once, only the gradients stay in registers
#pragma unroll
    for (int p = 0; p < CP; ++p) {
      uint64_t act[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gs = power_of_gate(w[i]), us = power_of_up(w[i]);
        act[i] = ckpt_pair(mul2(e4m3x2_f32(t.g[i] >> (16 * p)), pk(gs, gs)), mul2(e4m3x2_f32(t.u[i] >> (16 * p)), pk(us, us)), unpk_bf16(p ? t.d[i].y : t.d[i].x), v[i][p], v2[i][p]);
      }
      if constexpr (ACT) put_pair(r, a.aq1, col, p, lane, act, mine, top);
    }
    const bool grads = a.out || a.q0 || a.q1;
    if constexpr (ACT) a.as1[column_scale(r, col, (lane & 7) * 4 + rq)] = (uint8_t)mine;
    const uint32_t next = col + 32;
    const bool last = next >= end;
    if (!last) load<ALL>(a, r, next, lane, false, t);
    if (grads) put_gradient<ALL>(a, r, col, lane, v, sc, last, top);
    if (grads) put_gradient<ALL>(a, r, r.F + col, lane, v2, sc2, last, top);
    col = next;
  }
  return top;
}

// A tile with every value by far_pair.  A function of its own, so that the other
// tiles' registers are not its.
template <bool ACT>
__device__ __noinline__ void far_tile(const SwigluArgs& a, const Rows& r, uint32_t col) {
  const int lane = threadIdx.x, rq = lane >> 3;
  const uint8_t *hq = a.hq + r.at + col, *uq = hq + r.F;
  const uint16_t* dp = dout_at(a, r, col, lane);
  uint32_t sg, su;
  load_scales(a, r, col, sg, su);
  const uint32_t pw = powers(sg, su);
  uint64_t v[8][CP], v2[8][CP], act[8][CP];
  uint32_t top = 0;
  // one pair at a time: many copies of far_pair do not stay in the instruction cache
#pragma unroll 1
  for (int k = 0; k < 8 * CP; ++k) {
    const int i0 = k / CP, p0 = k % CP;
    const uint32_t w = __shfl_sync(0xffffffffu, pw, rq * 8 + i0);
    auto h_pair = [&](const uint8_t* q, float s) {
      return i0 < r.rows ? pack_bf16x2(mul2(e4m3x2_f32(__ldg(reinterpret_cast<const uint16_t*>(q + wide(2 * r.F, i0) + 2 * p0))), pk(s, s)))
                         : 0u;
    };
    const uint32_t g = h_pair(hq, power_of_gate(w)), u = h_pair(uq, power_of_up(w));
    const uint32_t d = i0 < r.rows ? __ldg(reinterpret_cast<const uint32_t*>(dp + wide(r.F, i0) + 2 * p0)) : 0u;
    uint64_t x, y, z, none;
    far_pair<true>(g, u, d, x, y);
    far_pair<false>(g, u, 0u, z, none);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int p = 0; p < CP; ++p)
        if (k == i * CP + p) v[i][p] = x, v2[i][p] = y, act[i][p] = z;
  }
  if constexpr (ACT) put_columns(r, a.aq1, a.as1, col, lane, act, top);
  if (a.out || a.q0 || a.q1) {
    RowScales sc, sc2;
    put_gradient<false>(a, r, col, lane, v, sc, true, top);
    put_gradient<false>(a, r, r.F + col, lane, v2, sc2, true, top);
  }
}

// A CTA: a warp, 32 rows and `per` column tiles of 32 from its place on.  ALL: M % 32 == 0,
// every row of a warp exists (as for any output along the columns).
template <bool ACT, bool ALL>
__global__ void __launch_bounds__(32, sc_warps<ACT>())
    k_swiglu_bwd_ckpt(const __grid_constant__ SwigluArgs a, uint32_t cp0, uint32_t cp1, int per) {
  const int lane = threadIdx.x, rq = lane >> 3, cq = lane & 7;
  // row tiles beyond the grid's 65535 are its z
  const int row0 = (int)(blockIdx.z * gridDim.y + blockIdx.y) * 32;
  if (row0 >= a.M) return;
  int prow = row0;
  if (a.E0 + a.E1 > 0) {
    prow = (int)padded_row(a.offs, a.E0 > 0 ? a.E0 : a.E1, a.M, row0, lane);
    if (prow < 0) {
      if (lane == 0) set_status(a.status, FP8MOE_ERR_DEVICE_OFFSETS);
      return;
    }
  }
  Rows r;
  const uint32_t F = r.F = (uint32_t)a.F, M = r.M = (uint32_t)a.M, first = row0 + rq * 8;
  r.rows = first + 8 <= M ? 8 : first < M ? (int)(M - first) : 0;
  r.at = wide(2 * F, first) + cq * 4;
  r.has_scale = ALL || row0 + lane < a.M;
  r.at_h = wide(F / 16, row0 + lane);
  r.tiled0 = a.s0_layout != FP8MOE_SCALES_ROWMAJOR;
  r.step0 = r.tiled0 ? 16 : F / 16;
  r.at_s0 = (r.tiled0 ? (uint64_t)tile_off(a.E0 > 0 ? prow : row0, 0, cp0) : wide(F / 16, row0)) + rq * 8 * r.step0;
  const bool tiled1 = a.s1_layout != FP8MOE_SCALES_ROWMAJOR;
  const uint32_t blk1 = (a.E1 > 0 ? prow : row0) / 32;
  r.at_s1 = tiled1 ? wide(512, blk1 >> 2) + (blk1 & 3) : row0 / 32;
  r.band1 = tiled1 ? cp1 : 0;
  r.at1 = wide(M, cq * 4) + first;
  r.h_words = F % 128 == 0 && ((uintptr_t)a.hs & 3) == 0;
  r.s0_words = r.tiled0 && ((uintptr_t)a.s0 & 3) == 0;
  const uint32_t col = blockIdx.x * per * 32, end = min(F, col + per * 32);
  const uint32_t top = tiles<ACT, ALL>(a, r, col, end, lane);
  // results that are not finite (see far_pair): all of the run's once more
  if (__any_sync(0xffffffffu, top == MX_NOT_FINITE)) {
    const Rows far = r;   // (in memory; r is not)
#pragma unroll 1
    for (uint32_t c = col; c < end; c += 32) far_tile<ACT>(a, far, c);
  }
}

// Column tiles of a CTA, `fit` of which are resident: what leaves the shortest sum
// over the rounds, the first tile's loads and the row's places counted as half a tile.
int64_t tiles_per_cta(int64_t col_tiles, int64_t row_tiles, int64_t fit) {
  int64_t best = 1, least = INT64_MAX;
  for (int64_t per = 1; per <= 4 && per <= col_tiles; per *= 2) {
    const int64_t n = (col_tiles + per - 1) / per * row_tiles, cost = (n + fit - 1) / fit * (2 * per + 1);
    if (cost < least) least = cost, best = per;
  }
  return best;
}

}  // namespace

cudaError_t launch_swiglu_bwd_ckpt(const SwigluArgs& a, cudaStream_t st) {
  const int64_t cp0 = (2 * a.F / 32 + 3) / 4 * 4, cp1 = (a.M / 32 + 3) / 4 * 4 + (int64_t)a.E1 * 4;
  const int64_t col_tiles = a.F / 32, row_tiles = (a.M + 31) / 32;
  const int64_t per = tiles_per_cta(col_tiles, row_tiles, (int64_t)(a.aq1 ? sc_warps<true>() : sc_warps<false>()) * a.num_sms);
  const int64_t ny = row_tiles < 32768 ? row_tiles : 32768;
  const dim3 grid((unsigned)((col_tiles + per - 1) / per), (unsigned)ny, (unsigned)((row_tiles + ny - 1) / ny));
  auto run = [&](auto kern) {
    kern<<<grid, 32, 0, st>>>(a, (uint32_t)cp0, (uint32_t)cp1, (int)per);
    return cudaGetLastError();
  };
  return a.aq1          ? run(k_swiglu_bwd_ckpt<true, true>)
         : a.M % 32 == 0 ? run(k_swiglu_bwd_ckpt<false, true>)
                         : run(k_swiglu_bwd_ckpt<false, false>);
}

}  // namespace fp8moe
