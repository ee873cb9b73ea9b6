// Backward of the gated activation from an MXFP8 checkpoint of its input, with
// MXFP8 output along both dimensions, and the activation of the checkpoint's values
// along its columns: the operand of the second product's weight gradient.
//
//   g, u = code * 2^e;  dg = d * u * sig(g) * (1 + g (1 - sig(g))),  du = d * g * sig(g),  a = g * sig(g) * u
// The arithmetic is the bf16 form's (swiglu.cuh), and so are the results' bits.
//
// Bound by HBM in bytes (9.2 an element of a), but with some 40 instructions an
// element by issue: five block scalings, the unpacking and the sigmoid.  So a warp's
// tile is 32 x 32, a lane's 8 x 4 (the bf16 form's is twice as wide): half the
// registers, and five CTAs an SM instead of three.  A block of a row is then one
// warp's eight lanes, so that its scale is read once a row; loads go straight to
// registers, hidden by the other warps.
#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"
#include "moe_ops.h"
#include "mxcvt.cuh"
#include "scales.cuh"
#include "swiglu.cuh"

namespace fp8moe {
namespace {

constexpr int SC_WARPS = 4;          // 2 x 2: 64 rows x 64 columns
constexpr int SC_CTAS = 4;           // of them an SM
constexpr int CP = 2;                // column pairs of a lane

// Where a warp's tile goes: bytes of its first row and column in each layout.
struct Place {
  int row0;
  int64_t col;            // this lane's first column
  bool ok;                // it exists
  int rows;               // rows of this lane that exist
};

// Codes and scales along the rows: v's columns start at column `col` of W.
FP8MOE_DEV void put_rows(const SwigluArgs& a, const Place& pl, int64_t W, int64_t col, uint8_t* s0, int64_t step0, int lane,
                         const uint64_t (&v)[8][CP], uint32_t& top) {
  const int cq = lane & 7;
  float m[8], m4[4], m2[2], mk[1], mul;
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = amax3(amax3(0.0f, v[i][0]), v[i][1]);
  // a row's block is the eight lanes of a row group; a lane ends with row `own`
  halve<8>(m, m4, lane, 1);
  halve<4>(m4, m2, lane, 2);
  halve<2>(m2, mk, lane, 4);
  const int own = (cq & 1) * 4 + (cq & 2) + (cq >> 2);
  const uint32_t b = mx_byte(mk[0], mul);
  top = max(top, b);
  const int64_t blk = col >> 5;
  if (pl.ok && own < pl.rows)
    s0[own * step0 + (a.s0_layout != FP8MOE_SCALES_ROWMAJOR ? (blk >> 2) * 512 + (blk & 3) : blk)] = (uint8_t)b;
  uint8_t* q = a.q0 + ((int64_t)pl.row0 + (lane >> 3) * 8) * W + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = __shfl_sync(0xffffffffu, mul, (lane & ~7) | (i >> 2) | (i & 2) | (i & 1) << 2);
    const uint64_t s2 = pk(s, s);
    float f[4];
    unpk(mul2(v[i][0], s2), f[0], f[1]);
    unpk(mul2(v[i][1], s2), f[2], f[3]);
    if (pl.ok && i < pl.rows) *reinterpret_cast<uint32_t*>(q + i * W) = cvt4(f[0], f[1], f[2], f[3]);
  }
}

// Codes and scales along the columns, transposed (M % 32 == 0: every row exists).
FP8MOE_DEV void put_columns(const SwigluArgs& a, const Place& pl, int64_t col, uint8_t* q1, uint8_t* s1, int64_t band1, int lane,
                            const uint64_t (&v)[8][CP], uint32_t& top) {
  float m[4], m2[2], mk[1], mul;
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
  halve<4>(m, m2, lane, 8);
  halve<2>(m2, mk, lane, 16);
  const int own = ((lane >> 3) & 1) * 2 + (lane >> 4);
  const uint32_t b = mx_byte(mk[0], mul);
  top = max(top, b);
  const int64_t c = col + own;
  if (pl.ok) s1[band1 ? (c >> 7) * band1 + (c & 31) * 16 + ((c >> 5) & 3) * 4 : c * (a.M / 32)] = (uint8_t)b;
  uint8_t* q = q1 + col * a.M + pl.row0 + (lane >> 3) * 8;
#pragma unroll
  for (int p = 0; p < CP; ++p) {
    const int src = (lane & 7) | p << 3;   // column 2 p's lane; 2 p + 1's is 16 further
    const float sc0 = __shfl_sync(0xffffffffu, mul, src), sc1 = __shfl_sync(0xffffffffu, mul, src | 16);
    const uint64_t s2 = pk(sc0, sc1);
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) unpk(mul2(v[i][p], s2), x[i], y[i]);
    if (pl.ok) {
      *reinterpret_cast<uint2*>(q + (2 * p) * a.M) = make_uint2(cvt4(x[0], x[1], x[2], x[3]), cvt4(x[4], x[5], x[6], x[7]));
      *reinterpret_cast<uint2*>(q + (2 * p + 1) * a.M) = make_uint2(cvt4(y[0], y[1], y[2], y[3]), cvt4(y[4], y[5], y[6], y[7]));
    }
  }
}

// The same of one column pair: its block's four lanes each take its maximum and
// scale.
FP8MOE_DEV void put_pair(const SwigluArgs& a, const Place& pl, int64_t col, uint8_t* q1, uint8_t* s1, int64_t band1, int lane,
                         const uint64_t (&v)[8], uint32_t& top) {
  float m0 = 0.0f, m1 = 0.0f, k0, k1, x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) unpk(v[i], x[i], y[i]);
#pragma unroll
  for (int i = 0; i < 8; i += 2) m0 = amax3(m0, x[i], x[i + 1]), m1 = amax3(m1, y[i], y[i + 1]);
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    m0 = nanmax(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = nanmax(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
  const uint32_t b0 = mx_byte(m0, k0), b1 = mx_byte(m1, k1);
  top = max(top, max(b0, b1));
  const uint64_t k2 = pk(k0, k1);
#pragma unroll
  for (int i = 0; i < 8; ++i) unpk(mul2(v[i], k2), x[i], y[i]);
  uint8_t* q = q1 + col * a.M + pl.row0 + (lane >> 3) * 8;
  *reinterpret_cast<uint2*>(q) = make_uint2(cvt4(x[0], x[1], x[2], x[3]), cvt4(x[4], x[5], x[6], x[7]));
  *reinterpret_cast<uint2*>(q + a.M) = make_uint2(cvt4(y[0], y[1], y[2], y[3]), cvt4(y[4], y[5], y[6], y[7]));
  if (lane < 8) {
    auto at = [&](int64_t c) { return band1 ? (c >> 7) * band1 + (c & 31) * 16 + ((c >> 5) & 3) * 4 : c * (a.M / 32); };
    s1[at(col)] = (uint8_t)b0;
    s1[at(col + 1)] = (uint8_t)b1;
  }
}

// One of the two gradients to every output but the activation's.
FP8MOE_DEV void put_gradient(const SwigluArgs& a, const Place& pl, int64_t col, uint8_t* s0, int64_t step0, uint8_t* s1,
                             int64_t band1, int lane, const uint64_t (&v)[8][CP], uint32_t& top) {
  const int64_t W = 2 * a.F;
  if (a.out && pl.ok) {
    uint16_t* o = a.out + ((int64_t)pl.row0 + (lane >> 3) * 8) * W + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < pl.rows) *reinterpret_cast<uint2*>(o + i * W) = make_uint2(pack_bf16x2(v[i][0]), pack_bf16x2(v[i][1]));
  }
  if (a.q0) put_rows(a, pl, W, col, s0, step0, lane, v, top);
  if (a.q1) put_columns(a, pl, col, a.q1, s1, band1, lane, v, top);
  if (!a.q0 && !a.q1) {
    float m = 0.0f, s;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = amax3(amax3(m, v[i][0]), v[i][1]);
    top = max(top, mx_byte(m, s));
  }
}

// A warp's tile.  FAR: every value by far_pair.
template <bool FAR>
FP8MOE_DEV void tile(const SwigluArgs& a, int row0, int col0, int64_t prow, int64_t cp0, int64_t cp1, int lane, uint32_t& top) {
  const int rq = lane >> 3;
  Place pl;
  pl.row0 = row0;
  pl.col = col0 + (lane & 7) * 4;
  pl.ok = true;                        // F % 32 == 0: a tile's columns exist together
  const int64_t r = (int64_t)row0 + rq * 8;
  pl.rows = r + 8 <= a.M ? 8 : r < a.M ? (int)(a.M - r) : 0;
  // this lane's row's powers of two
  float pg = 0.0f, pu = 0.0f;
  if (row0 + lane < a.M) {
    const uint8_t* s = a.hs + (int64_t)(row0 + lane) * (a.F / 16) + (col0 >> 5);
    pg = mx_power(__ldg(s)), pu = mx_power(__ldg(s + (a.F >> 5)));
  }
  const bool t0 = a.s0_layout != FP8MOE_SCALES_ROWMAJOR, t1 = a.s1_layout != FP8MOE_SCALES_ROWMAJOR;
  const int64_t p0 = a.E0 > 0 ? prow : row0, p1 = (a.E1 > 0 ? prow : row0) / 32, step0 = t0 ? 16 : a.F / 16;
  uint8_t* s0 = a.s0 + (t0 ? tile_off(p0, 0, cp0) : (int64_t)row0 * (a.F / 16)) + rq * 8 * step0;
  const int64_t at1 = t1 ? (p1 >> 2) * 512 + (p1 & 3) : row0 / 32, band1 = t1 ? cp1 * 128 : 0;
  const uint8_t* hq = a.hq + r * 2 * a.F + pl.col;
  const uint16_t* dp = a.dout + r * a.F + pl.col;
  uint64_t v[8][CP], v2[8][CP];
  if constexpr (!FAR) {
    uint32_t cg[8], cu[8];
    uint2 d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool on = i < pl.rows;
      cg[i] = on ? __ldg(reinterpret_cast<const uint32_t*>(hq + i * 2 * a.F)) : 0u;
      cu[i] = on ? __ldg(reinterpret_cast<const uint32_t*>(hq + i * 2 * a.F + a.F)) : 0u;
      d[i] = on ? __ldg(reinterpret_cast<const uint2*>(dp + i * a.F)) : make_uint2(0, 0);
    }
    // column pair by column pair: the activation's values go to their codes at
    // once, only the gradients stay in registers
#pragma unroll
    for (int p = 0; p < CP; ++p) {
      uint64_t act[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gs = __shfl_sync(0xffffffffu, pg, rq * 8 + i), us = __shfl_sync(0xffffffffu, pu, rq * 8 + i);
        const uint64_t g2 = mul2(e4m3x2_f32(cg[i] >> (16 * p)), pk(gs, gs)), u2 = mul2(e4m3x2_f32(cu[i] >> (16 * p)), pk(us, us));
        act[i] = ckpt_pair(g2, u2, unpk_bf16(p ? d[i].y : d[i].x), v[i][p], v2[i][p]);
      }
      if (a.aq1) put_pair(a, pl, pl.col + 2 * p, a.aq1, a.as1 + at1, band1, lane, act, top);
    }
  } else {
    // one pair at a time: many copies of far_pair do not stay in the instruction cache
    uint64_t act[8][CP];
#pragma unroll 1
    for (int k = 0; k < 8 * CP; ++k) {
      const int i0 = k / CP, p0 = k % CP;
      const float gs = __shfl_sync(0xffffffffu, pg, rq * 8 + i0), us = __shfl_sync(0xffffffffu, pu, rq * 8 + i0);
      auto h_pair = [&](const uint8_t* q, float s) {
        return i0 < pl.rows ? pack_bf16x2(mul2(e4m3x2_f32(__ldg(reinterpret_cast<const uint16_t*>(q + i0 * 2 * a.F + 2 * p0))), pk(s, s))) : 0u;
      };
      const uint32_t g = h_pair(hq, gs), u = h_pair(hq + a.F, us);
      const uint32_t d = i0 < pl.rows ? __ldg(reinterpret_cast<const uint32_t*>(dp + i0 * a.F + 2 * p0)) : 0u;
      uint64_t x, y, z, none;
      far_pair<true>(g, u, d, x, y);
      far_pair<false>(g, u, 0u, z, none);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int p = 0; p < CP; ++p)
          if (k == i * CP + p) v[i][p] = x, v2[i][p] = y, act[i][p] = z;
    }
    if (a.aq1) put_columns(a, pl, pl.col, a.aq1, a.as1 + at1, band1, lane, act, top);
  }
  if (a.out || a.q0 || a.q1) {
    put_gradient(a, pl, pl.col, s0, step0, a.s1 + at1, band1, lane, v, top);
    put_gradient(a, pl, a.F + pl.col, s0, step0, a.s1 + at1, band1, lane, v2, top);
  }
}

// A function of its own, so that the other tiles' registers are not its
__device__ __noinline__ void far_tile(const SwigluArgs& a, int row0, int col0, int64_t prow, int64_t cp0, int64_t cp1) {
  uint32_t top = 0;
  tile<true>(a, row0, col0, prow, cp0, cp1, threadIdx.x & 31, top);
}

// A CTA: 64 rows and `per` column tiles of 64 from its place on.
__global__ void __launch_bounds__(SC_WARPS * 32, SC_CTAS)
    k_swiglu_bwd_ckpt(SwigluArgs a, int64_t cp0, int64_t cp1, int col_tiles, int per) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int runs = (col_tiles + per - 1) / per, rb = blockIdx.x / runs, c0 = (blockIdx.x - rb * runs) * per;
  const int row0 = (rb * 2 + (warp & 1)) * 32;
  if (row0 >= a.M) return;
  int64_t prow = row0;
  if (a.E0 + a.E1 > 0) {
    prow = padded_row(a.offs, a.E0 > 0 ? a.E0 : a.E1, a.M, row0, lane);
    if (prow < 0) {
      if (lane == 0) set_status(a.status, FP8MOE_ERR_DEVICE_OFFSETS);
      return;
    }
  }
  uint32_t top = 0;
  const int c1 = min(col_tiles, c0 + per);
  for (int c = c0; c < c1; ++c) {
    const int col0 = c * 64 + (warp >> 1) * 32;
    if (col0 < a.F) tile<false>(a, row0, col0, prow, cp0, cp1, lane, top);
  }
  // results that are not finite (see far_pair): all of the run's once more
  if (__any_sync(0xffffffffu, top == MX_NOT_FINITE))
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      const int col0 = c * 64 + (warp >> 1) * 32;
      if (col0 < a.F) far_tile(a, row0, col0, prow, cp0, cp1);
    }
}

}  // namespace

cudaError_t launch_swiglu_bwd_ckpt(const SwigluArgs& a, cudaStream_t st) {
  const int64_t cp0 = (2 * a.F / 32 + 3) / 4 * 4, cp1 = (a.M / 32 + 3) / 4 * 4 + (int64_t)a.E1 * 4;
  const int64_t col_tiles = (a.F + 63) / 64, row_tiles = (a.M + 63) / 64;
  const int64_t per = 1;
  const int64_t grid = row_tiles * ((col_tiles + per - 1) / per);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  k_swiglu_bwd_ckpt<<<(unsigned)grid, SC_WARPS * 32, 0, st>>>(a, cp0, cp1, (int)col_tiles, (int)per);
  return cudaGetLastError();
}

}  // namespace fp8moe
