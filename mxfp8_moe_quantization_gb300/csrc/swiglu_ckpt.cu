// Backward of the gated activation from an MXFP8 checkpoint of its input, with
// MXFP8 output along both dimensions, and the activation of the checkpoint's values
// along its columns: the operand of the second product's weight gradient.
//
//   g, u = code * 2^e;  dg = d * u * sig(g) * (1 + g (1 - sig(g))),  du = d * g * sig(g),  a = g * sig(g) * u
// The arithmetic is the bf16 form's (swiglu.cuh), and so are the results' bits.
//
// Bound by HBM in bytes (9.2 an element of a), but with some 45 instructions an
// element by issue: five block scalings, the unpacking and the sigmoid.  So a warp's
// tile is 32 x 32, a lane's 8 x 4 (the bf16 form's is twice as wide): half the
// registers, and four CTAs an SM instead of three.  A block of a row is then one
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

// i rows of `stride` elements: a product of 32-bit factors (sizes are below 2^30)
FP8MOE_DEV uint64_t wide(uint32_t stride, uint32_t i) { return (uint64_t)stride * i; }

// A warp's rows: where they are in every tensor (column 0, or this lane's in a tile
// at column 0).  The lane has rows 8 rq .. and columns 4 cq .. of a tile.
struct Rows {
  uint32_t F, M;
  int rows;                    // of the lane's eight, those that exist
  const uint8_t* h;            // codes of gate
  const uint8_t* hs;           // scales: of row `lane` of the tile
  bool has_scale;
  const uint16_t* d;
  uint16_t* out;
  uint8_t *q0, *s0;            // rows' codes and scales
  uint32_t step0;
  bool tiled0;
  uint8_t *q1, *s1, *aq1, *as1;  // columns'; s1 and as1: of the tile's block of rows
  uint32_t band1;              // 128 columns' scales, in units of 128 bytes, 0: row-major
};

// Bytes from s1 to the scale of lane-column j (below 32) of a tile at column `col`.
FP8MOE_DEV uint64_t column_scale(const Rows& r, uint32_t col, uint32_t j) {
  return r.band1 ? wide(r.band1, col >> 7) * 128 + (col >> 5 & 3u) * 4 + j * 16 : wide(r.M / 32, col + j);
}

// Codes and scales along the rows: v's columns are those from `col` of 2F.
FP8MOE_DEV void put_rows(const Rows& r, uint32_t col, int lane, const uint64_t (&v)[8][CP], uint32_t& top) {
  const int cq = lane & 7;
  float m[8], m4[4], m2[2], mk[1], mul;
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = amax3(amax3(0.0f, v[i][0]), v[i][1]);
  // a row's block is the eight lanes of a row group; a lane ends with row `own`
  halve<8>(m, m4, lane, 1);
  halve<4>(m4, m2, lane, 2);
  halve<2>(m2, mk, lane, 4);
  const int own = (cq & 1) * 4 + (cq & 2) + (cq >> 2);
  const uint32_t b = mx_byte(mk[0], mul), blk = col >> 5;
  top = max(top, b);
  if (own < r.rows) r.s0[(uint32_t)own * r.step0 + (r.tiled0 ? (blk >> 2) * 512 + (blk & 3) : blk)] = (uint8_t)b;
  uint8_t* q = r.q0 + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = __shfl_sync(0xffffffffu, mul, (lane & ~7) | (i >> 2) | (i & 2) | (i & 1) << 2);
    float f[4];
    unpk(v[i][0], f[0], f[1]);
    unpk(v[i][1], f[2], f[3]);
    if (i < r.rows) *reinterpret_cast<uint32_t*>(q + wide(2 * r.F, i)) = cvt4(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
  }
}

// Codes and scales along the columns from `col` on, transposed (M % 32 == 0: every
// row exists).
FP8MOE_DEV void put_columns(const Rows& r, uint8_t* q1, uint8_t* s1, uint32_t col, int lane, const uint64_t (&v)[8][CP],
                            uint32_t& top) {
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
  const uint32_t own = (uint32_t)(((lane >> 3) & 1) * 2 + (lane >> 4)), b = mx_byte(mk[0], mul);
  top = max(top, b);
  s1[column_scale(r, col, (lane & 7) * 4 + own)] = (uint8_t)b;
  uint8_t* q = q1 + wide(r.M, col);
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
// scale.
FP8MOE_DEV void put_pair(const Rows& r, uint8_t* q1, uint8_t* s1, uint32_t col, int p, int lane, const uint64_t (&v)[8],
                         uint32_t& top) {
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
  uint8_t* q = q1 + wide(r.M, col + 2 * p);
  *reinterpret_cast<uint2*>(q) =
      make_uint2(cvt4(x[0] * k0, x[1] * k0, x[2] * k0, x[3] * k0), cvt4(x[4] * k0, x[5] * k0, x[6] * k0, x[7] * k0));
  *reinterpret_cast<uint2*>(q + r.M) =
      make_uint2(cvt4(y[0] * k1, y[1] * k1, y[2] * k1, y[3] * k1), cvt4(y[4] * k1, y[5] * k1, y[6] * k1, y[7] * k1));
  if (lane < 8) {
    s1[column_scale(r, col, lane * 4 + 2 * p)] = (uint8_t)b0;
    s1[column_scale(r, col, lane * 4 + 2 * p + 1)] = (uint8_t)b1;
  }
}

// One of the two gradients to every output but the activation's.
FP8MOE_DEV void put_gradient(const Rows& r, uint32_t col, int lane, const uint64_t (&v)[8][CP], uint32_t& top) {
  if (r.out) {
    uint16_t* o = r.out + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < r.rows) *reinterpret_cast<uint2*>(o + wide(2 * r.F, i)) = make_uint2(pack_bf16x2(v[i][0]), pack_bf16x2(v[i][1]));
  }
  if (r.q0) put_rows(r, col, lane, v, top);
  if (r.q1) put_columns(r, r.q1, r.s1, col, lane, v, top);
  if (!r.q0 && !r.q1) {
    float m = 0.0f, s;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = amax3(amax3(m, v[i][0]), v[i][1]);
    top = max(top, mx_byte(m, s));
  }
}

// A warp's tile at column col.  FAR: every value by far_pair.
template <bool ACT, bool FAR>
FP8MOE_DEV void tile(const Rows& r, uint32_t col, int lane, uint32_t& top) {
  const int rq = lane >> 3;
  const uint32_t F = r.F;
  // row `lane`'s powers of two
  float pg = 0.0f, pu = 0.0f;
  if (r.has_scale) pg = mx_power(__ldg(r.hs + (col >> 5))), pu = mx_power(__ldg(r.hs + (F >> 5) + (col >> 5)));
  const uint8_t *hq = r.h + col, *uq = hq + F;
  const uint16_t* dp = r.d + col;
  uint64_t v[8][CP], v2[8][CP];
  if constexpr (!FAR) {
    uint32_t cg[8], cu[8];
    uint2 d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool on = i < r.rows;
      cg[i] = on ? __ldg(reinterpret_cast<const uint32_t*>(hq + wide(2 * F, i))) : 0u;
      cu[i] = on ? __ldg(reinterpret_cast<const uint32_t*>(uq + wide(2 * F, i))) : 0u;
      d[i] = on ? __ldg(reinterpret_cast<const uint2*>(dp + wide(F, i))) : make_uint2(0, 0);
    }
    // column pair by column pair: the activation's values go to their codes at
    // once, only the gradients stay in registers
#pragma unroll
    for (int p = 0; p < CP; ++p) {
      uint64_t act[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gs = __shfl_sync(0xffffffffu, pg, rq * 8 + i), us = __shfl_sync(0xffffffffu, pu, rq * 8 + i);
        float x, y, z, w;
        unpk(e4m3x2_f32(cg[i] >> (16 * p)), x, y);
        unpk(e4m3x2_f32(cu[i] >> (16 * p)), z, w);
        act[i] = ckpt_pair(pk(x * gs, y * gs), pk(z * us, w * us), unpk_bf16(p ? d[i].y : d[i].x), v[i][p], v2[i][p]);
      }
      if constexpr (ACT) put_pair(r, r.aq1, r.as1, col, p, lane, act, top);
    }
  } else {
    // one pair at a time: many copies of far_pair do not stay in the instruction cache
    uint64_t act[8][CP];
#pragma unroll 1
    for (int k = 0; k < 8 * CP; ++k) {
      const int i0 = k / CP, p0 = k % CP;
      const float gs = __shfl_sync(0xffffffffu, pg, rq * 8 + i0), us = __shfl_sync(0xffffffffu, pu, rq * 8 + i0);
      auto h_pair = [&](const uint8_t* q, float s) {
        return i0 < r.rows ? pack_bf16x2(mul2(e4m3x2_f32(__ldg(reinterpret_cast<const uint16_t*>(q + wide(2 * F, i0) + 2 * p0))), pk(s, s)))
                           : 0u;
      };
      const uint32_t g = h_pair(hq, gs), u = h_pair(uq, us);
      const uint32_t d = i0 < r.rows ? __ldg(reinterpret_cast<const uint32_t*>(dp + wide(F, i0) + 2 * p0)) : 0u;
      uint64_t x, y, z, none;
      far_pair<true>(g, u, d, x, y);
      far_pair<false>(g, u, 0u, z, none);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int p = 0; p < CP; ++p)
          if (k == i * CP + p) v[i][p] = x, v2[i][p] = y, act[i][p] = z;
    }
    if constexpr (ACT) put_columns(r, r.aq1, r.as1, col, lane, act, top);
  }
  if (r.out || r.q0 || r.q1) {
    put_gradient(r, col, lane, v, top);
    put_gradient(r, F + col, lane, v2, top);
  }
}

// A function of its own, so that the other tiles' registers are not its
template <bool ACT>
__device__ __noinline__ void far_tile(const Rows& r, uint32_t col) {
  uint32_t top = 0;
  tile<ACT, true>(r, col, threadIdx.x & 31, top);
}

// A CTA: 64 rows and `per` column tiles of 64 from its place on.
template <bool ACT>
__global__ void __launch_bounds__(SC_WARPS * 32, SC_CTAS) k_swiglu_bwd_ckpt(SwigluArgs a, uint32_t cp0, uint32_t cp1, int col_tiles, int per) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rq = lane >> 3, cq = lane & 7;
  // row tiles beyond the grid's 65535 are its z
  const int row0 = (int)((blockIdx.z * gridDim.y + blockIdx.y) * 2 + (warp & 1)) * 32, c0 = blockIdx.x * per;
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
  r.h = a.hq + wide(2 * F, first) + cq * 4;
  r.d = a.dout + wide(F, first) + cq * 4;
  r.has_scale = row0 + lane < a.M;
  r.hs = a.hs + wide(F / 16, row0 + lane);
  r.out = a.out ? a.out + wide(2 * F, first) + cq * 4 : nullptr;
  r.q0 = a.q0 ? a.q0 + wide(2 * F, first) + cq * 4 : nullptr;
  r.tiled0 = a.s0_layout != FP8MOE_SCALES_ROWMAJOR;
  r.step0 = r.tiled0 ? 16 : F / 16;
  r.s0 = a.s0 + (r.tiled0 ? tile_off(a.E0 > 0 ? prow : row0, 0, cp0) : (int64_t)wide(F / 16, row0)) + rq * 8 * r.step0;
  const bool tiled1 = a.s1_layout != FP8MOE_SCALES_ROWMAJOR;
  const uint32_t blk1 = (a.E1 > 0 ? prow : row0) / 32;
  const uint64_t at1 = tiled1 ? wide(512, blk1 >> 2) + (blk1 & 3) : row0 / 32;
  r.band1 = tiled1 ? cp1 : 0;
  const uint64_t col1 = wide(M, cq * 4) + first;
  r.q1 = a.q1 ? a.q1 + col1 : nullptr;
  r.s1 = a.s1 + at1;
  r.aq1 = a.aq1 + col1;
  r.as1 = a.as1 + at1;
  uint32_t top = 0;
  const int c1 = min(col_tiles, c0 + per);
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const uint32_t col = c * 64 + (warp >> 1) * 32;
    if (col < F) tile<ACT, false>(r, col, lane, top);
  }
  // results that are not finite (see far_pair): all of the run's once more
  if (__any_sync(0xffffffffu, top == MX_NOT_FINITE))
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      const uint32_t col = c * 64 + (warp >> 1) * 32;
      if (col < F) far_tile<ACT>(r, col);
    }
}

}  // namespace

cudaError_t launch_swiglu_bwd_ckpt(const SwigluArgs& a, cudaStream_t st) {
  const int64_t cp0 = (2 * a.F / 32 + 3) / 4 * 4, cp1 = (a.M / 32 + 3) / 4 * 4 + (int64_t)a.E1 * 4;
  const int64_t col_tiles = (a.F + 63) / 64, row_tiles = (a.M + 63) / 64;
  // Column tiles of a CTA: two where there are many
  const int64_t per = col_tiles * row_tiles > (int64_t)4 * SC_CTAS * a.num_sms ? 2 : 1;
  const int64_t ny = row_tiles < 32768 ? row_tiles : 32768;
  const dim3 grid((unsigned)((col_tiles + per - 1) / per), (unsigned)ny, (unsigned)((row_tiles + ny - 1) / ny));
  if (a.aq1) {
    k_swiglu_bwd_ckpt<true><<<grid, SC_WARPS * 32, 0, st>>>(a, (uint32_t)cp0, (uint32_t)cp1, (int)col_tiles, (int)per);
  } else {
    k_swiglu_bwd_ckpt<false><<<grid, SC_WARPS * 32, 0, st>>>(a, (uint32_t)cp0, (uint32_t)cp1, (int)col_tiles, (int)per);
  }
  return cudaGetLastError();
}

}  // namespace fp8moe
