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
// A warp holds a tile of 32 rows x 64 columns, a lane 8 rows x 8 columns: the
// 16-byte loads of eight lanes fill a 128-byte line, a row block's maximum is
// two shuffles, a column block's two more, and the conversions along a column
// take neighbouring rows from the same lane's registers, so that the
// transposed codes need no byte transposes.  Four warps of a CTA take 128
// consecutive rows: their column runs fill whole 128-byte lines of q1.
#include "common.cuh"
#include "launch.h"
#include "moe_ops.h"
#include "scales.cuh"

namespace fp8moe {
namespace {

constexpr int SG_ROWS = 32, SG_COLS = 64, SG_WARPS = 4;

FP8MOE_DEV void unpack8s(const uint4& q, float (&f)[8]) {
  f[0] = bf16_lo(q.x), f[1] = bf16_hi(q.x), f[2] = bf16_lo(q.y), f[3] = bf16_hi(q.y);
  f[4] = bf16_lo(q.z), f[5] = bf16_hi(q.z), f[6] = bf16_lo(q.w), f[7] = bf16_hi(q.w);
}
FP8MOE_DEV uint32_t pack2s(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The padded row (in a layout whose groups start at multiples of 128 rows) of
// row `row0`, a multiple of 32; -1 if the offsets are invalid.  A warp calls
// it; each of its lanes takes every 32nd group.
FP8MOE_DEV int64_t padded_row(const int32_t* offs, int E, int64_t M, int64_t row0, int lane) {
  uint32_t sum = 0;
  int bad = 0, prev = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const int end = e < E ? offs[e] : 0;
    int start = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) start = prev;
    prev = __shfl_sync(0xffffffffu, end, 31);
    if (e < E) {
      if (start < 0 || end < start || end > M || (end & 31) || (e == E - 1 && end != M)) bad = 1;
      if (end <= row0) {
        sum += ((uint32_t)(end - start) + 127u) & ~127u;
      } else if (start <= row0) {
        sum += (uint32_t)(row0 - start);
      }
    }
  }
  if (__any_sync(0xffffffffu, bad)) return -1;
  return (int64_t)__reduce_add_sync(0xffffffffu, sum);
}

FP8MOE_DEV uint32_t block_byte(float amax, float& mul) {
  const uint32_t b = max(__float_as_uint(amax) >> 23, 8u) - 8u;
  mul = __uint_as_float((254u - b) << 23);
  return b;
}

struct TilePlace {
  int64_t row0;   // first row of the tile
  int64_t prow0;  // the row in s0's layout
  int64_t pcol1;  // the scale column in s1's layout
  int64_t W;      // columns of the result
  int64_t cp0, cp1;  // padded scale columns of s0 / s1
};

// One tile of results v (lane: rows 8 rq .., columns 8 cq ..) to every output.
// col0: the tile's first column; ok: this lane's columns exist.
FP8MOE_DEV void put_tile(const SwigluArgs& a, const TilePlace& tp, int64_t col0, bool ok, int rq, int cq,
                         const float (&v)[8][8]) {
  const int64_t W = tp.W, col = col0 + cq * 8, rbase = tp.row0 + rq * 8;
  if (a.out && ok) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (rbase + i < a.M)
        *reinterpret_cast<uint4*>(a.out + (rbase + i) * W + col) =
            make_uint4(pack2s(v[i][0], v[i][1]), pack2s(v[i][2], v[i][3]), pack2s(v[i][4], v[i][5]),
                       pack2s(v[i][6], v[i][7]));
  }
  if (a.q0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = 0.0f, s;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t b = block_byte(m, s);
      if (!ok || rbase + i >= a.M) continue;
      *reinterpret_cast<uint2*>(a.q0 + (rbase + i) * W + col) =
          make_uint2(enc4<false>(v[i][0] * s, v[i][1] * s, v[i][2] * s, v[i][3] * s),
                     enc4<false>(v[i][4] * s, v[i][5] * s, v[i][6] * s, v[i][7] * s));
      if ((cq & 3) == 0)
        a.s0[a.s0_layout == FP8MOE_SCALES_ROWMAJOR ? (rbase + i) * (W / 32) + col / 32
                                                  : tile_off(tp.prow0 + rq * 8 + i, col / 32, tp.cp0)] = (uint8_t)b;
    }
  }
  if (a.q1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float m = 0.0f, s;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i][j]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      const uint32_t b = block_byte(m, s);
      if (!ok) continue;
      *reinterpret_cast<uint2*>(a.q1 + (col + j) * a.M + rbase) =
          make_uint2(enc4<false>(v[0][j] * s, v[1][j] * s, v[2][j] * s, v[3][j] * s),
                     enc4<false>(v[4][j] * s, v[5][j] * s, v[6][j] * s, v[7][j] * s));
      if (rq == 0)
        a.s1[a.s1_layout == FP8MOE_SCALES_ROWMAJOR ? (col + j) * (a.M / 32) + tp.row0 / 32
                                                  : tile_off(col + j, tp.pcol1, tp.cp1)] = (uint8_t)b;
    }
  }
}

template <bool BWD>
__global__ void __launch_bounds__(SG_WARPS * 32) k_swiglu(SwigluArgs a, int64_t cp0, int64_t cp1, int64_t col_tiles) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rq = lane >> 3, cq = lane & 7;
  TilePlace tp;
  tp.row0 = ((int64_t)blockIdx.x / col_tiles * SG_WARPS + warp) * SG_ROWS;
  if (tp.row0 >= a.M) return;
  const int64_t col0 = (int64_t)blockIdx.x % col_tiles * SG_COLS, col = col0 + cq * 8;
  const bool ok = col < a.F;
  tp.W = BWD ? 2 * a.F : a.F;
  tp.cp0 = cp0, tp.cp1 = cp1;
  const uint4 z = make_uint4(0, 0, 0, 0);
  uint4 g[8], u[8], d[BWD ? 8 : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = tp.row0 + rq * 8 + i;
    const bool on = ok && r < a.M;
    g[i] = on ? ld_nc16(a.h + r * a.ldh + col) : z;
    u[i] = on ? ld_nc16(a.h + r * a.ldh + a.F + col) : z;
    if constexpr (BWD) d[i] = on ? ld_nc16(a.dout + r * a.F + col) : z;
  }
  tp.prow0 = tp.row0;
  tp.pcol1 = tp.row0 / 32;
  if (a.E0 + a.E1 > 0) {   // after the loads, which are in flight meanwhile
    const int64_t pr = padded_row(a.offs, a.E0 > 0 ? a.E0 : a.E1, a.M, tp.row0, lane);
    if (pr < 0) {
      if (lane == 0) set_status(a.status, FP8MOE_ERR_DEVICE_OFFSETS);
      return;
    }
    if (a.E0 > 0) tp.prow0 = pr;
    if (a.E1 > 0) tp.pcol1 = pr / 32;
  }
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float gf[8], uf[8], df[8];
    unpack8s(g[i], gf);
    unpack8s(u[i], uf);
    if constexpr (BWD) unpack8s(d[i], df);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sg = __fdividef(1.0f, 1.0f + expf(-gf[j]));
      v[i][j] = BWD ? df[j] * uf[j] * sg * (1.0f + gf[j] * (1.0f - sg)) : gf[j] * sg * uf[j];
    }
  }
  put_tile(a, tp, col0, ok, rq, cq, v);
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float gf[8], df[8];
      unpack8s(g[i], gf);
      unpack8s(d[i], df);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = df[j] * gf[j] * __fdividef(1.0f, 1.0f + expf(-gf[j]));
    }
    put_tile(a, tp, a.F + col0, ok, rq, cq, v);
  }
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t st) {
  const int64_t W = a.dout ? 2 * a.F : a.F;
  const int64_t cp0 = (W / 32 + 3) / 4 * 4;
  const int64_t cp1 = (a.M / 32 + 3) / 4 * 4 + (int64_t)a.E1 * 4;
  const int64_t col_tiles = (a.F + SG_COLS - 1) / SG_COLS;
  const int64_t blocks = (a.M + SG_ROWS * SG_WARPS - 1) / (SG_ROWS * SG_WARPS) * col_tiles;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (a.dout) {
    k_swiglu<true><<<(unsigned)blocks, SG_WARPS * 32, 0, st>>>(a, cp0, cp1, col_tiles);
  } else {
    k_swiglu<false><<<(unsigned)blocks, SG_WARPS * 32, 0, st>>>(a, cp0, cp1, col_tiles);
  }
  return cudaGetLastError();
}

}  // namespace fp8moe
