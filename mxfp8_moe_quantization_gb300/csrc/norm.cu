// Residual addition + RMS norm with an 8-bit output, and its backward.
//
// Forward, per row of H elements (fp32 throughout, every output rounded once):
//   a = x + r            h = bf16(a)      (r may be absent; then h is x itself)
//   rstd = 1 / sqrt(mean(a^2) + eps)
//   y = (a * rstd) * w   as bf16, and / or as
//     MXFP8:   per 32 elements the e8m0 byte of max|y| and e4m3(y * 2^-e)
//     rowwise: s = max / max(max|y|, 1e-12), e4m3(y * s), 1 / s per row
// The codes come from the fp32 y, not from its bf16 copy: one rounding.
// Backward (xh = h * rstd, g = dy * w):
//   dx = rstd * (g - xh * mean(g * xh)) + dh,   dw = sum over rows of dy * xh
//
// Both directions move each element once and are bound by HBM; a row lives in
// the registers of its warps between its loads and its stores.
#include "common.cuh"
#include "launch.h"
#include "scales.cuh"

namespace fp8moe {
namespace {

// Threads of a CTA whose threads hold V 16-byte chunks per tensor (V = 1 in
// up to 64 registers, V = 2 and 4 in up to 128).
template <int V>
constexpr int norm_threads() { return V == 1 ? 1024 : 512; }
constexpr int NORM_MAX_CHUNKS = 4 * norm_threads<4>();   // longer rows (H > 16384) take the looping kernels

// a load that the same thread may follow with a store to the same place (the
// residual stream is updated in place), so not through the read-only path
FP8MOE_DEV uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
FP8MOE_DEV void unpack8(const uint4& q, float (&f)[8]) {
  f[0] = bf16_lo(q.x), f[1] = bf16_hi(q.x), f[2] = bf16_lo(q.y), f[3] = bf16_hi(q.y);
  f[4] = bf16_lo(q.z), f[5] = bf16_hi(q.z), f[6] = bf16_lo(q.w), f[7] = bf16_hi(q.w);
}
FP8MOE_DEV uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
FP8MOE_DEV uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
template <bool W32>
FP8MOE_DEV void load_w8(const void* w, int64_t ch, float (&f)[8]) {
  if constexpr (W32) {
    const float4 a = reinterpret_cast<const float4*>(w)[2 * ch], b = reinterpret_cast<const float4*>(w)[2 * ch + 1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8(reinterpret_cast<const uint4*>(w)[ch], f);
  }
}

enum { NORM_OUT_NONE = 0, NORM_OUT_MX = 1, NORM_OUT_ROW = 2, NORM_OUT_ROW_FNUZ = 3 };

struct NormFwdArgs {
  const uint16_t *x, *r;
  int64_t ldx, ldr, T, rows;  // rows: T, or the padded rows of the 128x4 scale layout
  int H;
  const void* w;
  float eps;
  uint16_t *h, *y;
  float* rstd;
  uint8_t* q;
  ScaleSpec sc;   // MXFP8 scales
  float* inv;     // rowwise scales
};

// Sum (or maximum) over the WPR warps of a row; slot: the row's place in `red`.
template <bool MAX>
FP8MOE_DEV float row_reduce(float v, float* red, int wpr, int group, int wrow) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if (wpr > 1) {
    if ((threadIdx.x & 31) == 0) red[group * wpr + wrow] = v;
    __syncthreads();
    v = red[group * wpr];
    for (int i = 1; i < wpr; ++i) v = MAX ? fmaxf(v, red[group * wpr + i]) : v + red[group * wpr + i];
  }
  return v;
}

// the eight codes of one chunk and, for MXFP8, its block's scale byte
template <int OUT>
FP8MOE_DEV uint2 encode8(const float (&v)[8], float s) {
  constexpr bool FZ = OUT == NORM_OUT_ROW_FNUZ;
  return make_uint2(enc4<FZ>(__fmul_rn(v[0], s), __fmul_rn(v[1], s), __fmul_rn(v[2], s), __fmul_rn(v[3], s)),
                    enc4<FZ>(__fmul_rn(v[4], s), __fmul_rn(v[5], s), __fmul_rn(v[6], s), __fmul_rn(v[7], s)));
}
FP8MOE_DEV float absmax8(const float (&v)[8]) {
  return fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))),
               fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7]))));
}
// e8m0 byte of a block maximum (the dim0 quantizer's rule on an fp32
// maximum) and the multiplier 2^-e
FP8MOE_DEV uint32_t mx_byte(float amax, float& mul) {
  const uint32_t b = max(__float_as_uint(amax) >> 23, 8u) - 8u;
  mul = __uint_as_float((254u - b) << 23);
  return b;
}

// One chunk of y: its bf16 copy, codes and scale.  Every lane of the warp
// calls it (the block maximum is a shuffle over four lanes).
template <int OUT>
FP8MOE_DEV void put_chunk(const NormFwdArgs& a, int64_t row, int ch, bool ok, const float (&v)[8], float s) {
  if (a.y && ok) *reinterpret_cast<uint4*>(a.y + row * a.H + (int64_t)ch * 8) = pack8(v);
  if constexpr (OUT == NORM_OUT_MX) {
    float m = absmax8(v);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t b = mx_byte(m, s);
    if (ok && (ch & 3) == 0) {
      const int64_t c = ch >> 2;
      a.sc.p[a.sc.layout == FP8MOE_SCALES_ROWMAJOR ? row * (a.H / 32) + c : tile_off(row, c, a.sc.Cp)] = (uint8_t)b;
    }
  }
  if constexpr (OUT != NORM_OUT_NONE) {
    if (ok) *reinterpret_cast<uint2*>(a.q + row * a.H + (int64_t)ch * 8) = encode8<OUT>(v, s);
  }
}

// the bytes of the 128x4 layout that stand for no block
FP8MOE_DEV void zero_scale_pad(const NormFwdArgs& a, int64_t row, int t, int n) {
  for (int64_t c = (row < a.T ? a.H / 32 : 0) + t; c < a.sc.Cp; c += n) a.sc.p[tile_off(row, c, a.sc.Cp)] = 0;
}

// A CTA holds `groups` rows, wpr warps each; a thread V chunks of its row.
template <int V, int OUT, bool W32>
__global__ void __launch_bounds__(norm_threads<V>()) k_norm_fwd(NormFwdArgs a, int wpr) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, group = warp / wpr, wrow = warp % wpr;
  const int tpr = wpr * 32, t = threadIdx.x - group * tpr;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + group;
  const bool active = row < a.T;
  const int nch = a.H / 8;
  uint4 xv[V], rv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ch = t + i * tpr;
    const bool ok = active && ch < nch;
    xv[i] = ok ? ld16(a.x + row * a.ldx + (int64_t)ch * 8) : make_uint4(0, 0, 0, 0);
    rv[i] = ok && a.r ? ld16(a.r + row * a.ldr + (int64_t)ch * 8) : make_uint4(0, 0, 0, 0);
  }
  float v[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    unpack8(xv[i], v[i]);
    if (a.r) {
      float f[8];
      unpack8(rv[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += f[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  ss = row_reduce<false>(ss, red[0], wpr, group, wrow);
  const float rstd = rsqrtf(__fdiv_rn(ss, (float)a.H) + a.eps);
  if (active && a.rstd && t == 0) a.rstd[row] = rstd;
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ch = t + i * tpr;
    const bool ok = active && ch < nch;
    if (a.h && ok) *reinterpret_cast<uint4*>(a.h + row * a.H + (int64_t)ch * 8) = pack8(v[i]);
    float wf[8];
    if (ok) {
      load_w8<W32>(a.w, ch, wf);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) wf[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = ok ? v[i][j] * rstd * wf[j] : 0.0f;
    if (OUT >= NORM_OUT_ROW) am = fmaxf(am, absmax8(v[i]));
  }
  float s = 1.0f;
  if constexpr (OUT >= NORM_OUT_ROW) {
    am = row_reduce<true>(am, red[1], wpr, group, wrow);
    float inv;
    rowwise_scale<OUT == NORM_OUT_ROW_FNUZ>(am, s, inv);
    if (active && t == 0) a.inv[row] = inv;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ch = t + i * tpr;
    put_chunk<OUT>(a, row, ch, active && ch < nch, v[i], s);
  }
  if (OUT == NORM_OUT_MX && a.sc.layout != FP8MOE_SCALES_ROWMAJOR && row < a.rows) zero_scale_pad(a, row, t, tpr);
}

// Rows longer than a CTA's registers hold: one CTA per row, which reads the
// row again (from L2) for each pass.
template <int OUT, bool W32>
__global__ void __launch_bounds__(1024) k_norm_fwd_long(NormFwdArgs a) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, n = blockDim.x, nch = a.H / 8;
  const bool active = row < a.T;
  auto load = [&](int ch, float (&v)[8]) {
    unpack8(ld16(a.x + row * a.ldx + (int64_t)ch * 8), v);
    if (a.r) {
      float f[8];
      unpack8(ld16(a.r + row * a.ldr + (int64_t)ch * 8), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
  };
  if (active) {
    float ss = 0.0f;
    for (int ch = t; ch < nch; ch += n) {
      float v[8];
      load(ch, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
    }
    ss = row_reduce<false>(ss, red[0], n / 32, 0, t >> 5);
    const float rstd = rsqrtf(__fdiv_rn(ss, (float)a.H) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    auto norm = [&](int ch, float (&v)[8]) {
      float wf[8];
      load_w8<W32>(a.w, ch, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * wf[j];
    };
    float s = 1.0f;
    if constexpr (OUT >= NORM_OUT_ROW) {
      float am = 0.0f, inv;
      for (int ch = t; ch < nch; ch += n) {
        float v[8];
        load(ch, v);
        norm(ch, v);
        am = fmaxf(am, absmax8(v));
      }
      am = row_reduce<true>(am, red[1], n / 32, 0, t >> 5);
      rowwise_scale<OUT == NORM_OUT_ROW_FNUZ>(am, s, inv);
      if (t == 0) a.inv[row] = inv;
    }
    for (int c0 = 0; c0 < nch; c0 += n) {   // every lane takes every trip (block maxima are shuffles)
      const int ch = c0 + t;
      const bool ok = ch < nch;
      float v[8] = {};
      if (ok) {
        load(ch, v);
        if (a.h) *reinterpret_cast<uint4*>(a.h + row * a.H + (int64_t)ch * 8) = pack8(v);
        norm(ch, v);
      }
      put_chunk<OUT>(a, row, ch, ok, v, s);
    }
  }
  if (OUT == NORM_OUT_MX && a.sc.layout != FP8MOE_SCALES_ROWMAJOR) zero_scale_pad(a, row, t, n);
}

template <int OUT, bool W32>
cudaError_t launch_fwd_t(const NormFwdArgs& a, cudaStream_t st) {
  const int nch = a.H / 8;
  if (nch > NORM_MAX_CHUNKS) {
    k_norm_fwd_long<OUT, W32><<<(unsigned)a.rows, 1024, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int v = nch <= 256 ? 1 : nch <= 512 ? 2 : 4;
  const int wpr = (nch + 32 * v - 1) / (32 * v);
  const int groups = wpr >= 8 ? 1 : 8 / wpr;
  const unsigned blocks = (unsigned)((a.rows + groups - 1) / groups), threads = (unsigned)(wpr * 32 * groups);
  if (v == 1) k_norm_fwd<1, OUT, W32><<<blocks, threads, 0, st>>>(a, wpr);
  if (v == 2) k_norm_fwd<2, OUT, W32><<<blocks, threads, 0, st>>>(a, wpr);
  if (v == 4) k_norm_fwd<4, OUT, W32><<<blocks, threads, 0, st>>>(a, wpr);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormBwdArgs {
  const uint16_t *dy, *h, *dh;
  const float* rstd;
  const void* w;
  int64_t T;
  int H;
  uint16_t* dx;
  float* part;  // [gridDim.x][H] partial weight gradients
};

// A CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ... whole; a thread
// keeps the same V chunks of every row, so its share of dw stays in registers.
template <int V, bool W32>
__global__ void __launch_bounds__(512) k_norm_bwd(NormBwdArgs a) {
  __shared__ float red[2][32];
  const int t = threadIdx.x, n = blockDim.x, nch = a.H / 8, warps = n >> 5;
  float dw[V][8] = {};
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, par ^= 1) {
    uint4 dyv[V], hv[V], sv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = t + i * n;
      const int64_t at = row * a.H + (int64_t)ch * 8;
      const uint4 z = make_uint4(0, 0, 0, 0);
      dyv[i] = ch < nch ? ld16(a.dy + at) : z;
      hv[i] = ch < nch ? ld16(a.h + at) : z;
      sv[i] = ch < nch && a.dh ? ld16(a.dh + at) : z;
    }
    const float rstd = a.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float d[8], x[8], wf[8];
      if (t + i * n >= nch) continue;
      unpack8(dyv[i], d);
      unpack8(hv[i], x);
      load_w8<W32>(a.w, t + i * n, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = x[j] * rstd;
        dot = fmaf(d[j] * wf[j], xh, dot);
        dw[i][j] = fmaf(d[j], xh, dw[i][j]);
      }
    }
    // the two halves of `red` alternate: a row's sums are read before the
    // barrier of the next row, which writes the other half
    dot = row_reduce<false>(dot, red[par], warps, 0, t >> 5);
    const float c = __fdiv_rn(dot, (float)a.H);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = t + i * n;
      if (ch >= nch) continue;
      float d[8], x[8], s[8], wf[8], o[8];
      unpack8(dyv[i], d);
      unpack8(hv[i], x);
      unpack8(sv[i], s);
      load_w8<W32>(a.w, ch, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(rstd, fmaf(-x[j] * rstd, c, d[j] * wf[j]), s[j]);
      *reinterpret_cast<uint4*>(a.dx + row * a.H + (int64_t)ch * 8) = pack8(o);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ch = t + i * n;
    if (ch >= nch) continue;
    float4* p = reinterpret_cast<float4*>(a.part + (int64_t)blockIdx.x * a.H + (int64_t)ch * 8);
    p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
    p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
  }
}

// Rows longer than that: the row is read twice (the second time from L2) and
// a thread's share of dw stays in its CTA's row of the partials.
template <bool W32>
__global__ void __launch_bounds__(512) k_norm_bwd_long(NormBwdArgs a) {
  __shared__ float red[2][32];
  const int t = threadIdx.x, n = blockDim.x, nch = a.H / 8;
  float* part = a.part + (int64_t)blockIdx.x * a.H;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, par ^= 1) {
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int ch = t; ch < nch; ch += n) {
      float d[8], x[8], wf[8];
      unpack8(ld16(a.dy + row * a.H + (int64_t)ch * 8), d);
      unpack8(ld16(a.h + row * a.H + (int64_t)ch * 8), x);
      load_w8<W32>(a.w, ch, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = fmaf(d[j] * wf[j], x[j] * rstd, dot);
    }
    dot = row_reduce<false>(dot, red[par], n >> 5, 0, t >> 5);
    const float c = __fdiv_rn(dot, (float)a.H);
    for (int ch = t; ch < nch; ch += n) {
      const int64_t at = row * a.H + (int64_t)ch * 8;
      float d[8], x[8], s[8] = {}, wf[8], o[8];
      unpack8(ld16(a.dy + at), d);
      unpack8(ld16(a.h + at), x);
      if (a.dh) unpack8(ld16(a.dh + at), s);
      load_w8<W32>(a.w, ch, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = x[j] * rstd;
        float* p = part + (int64_t)ch * 8 + j;
        *p = row == blockIdx.x ? d[j] * xh : fmaf(d[j], xh, *p);
        o[j] = fmaf(rstd, fmaf(-xh, c, d[j] * wf[j]), s[j]);
      }
      *reinterpret_cast<uint4*>(a.dx + at) = pack8(o);
    }
  }
}

// dw[c] = sum over the P partials in order: 32 columns per CTA, 32 warps that
// each take every 32nd partial, then a fixed-order sum over the warps.
__global__ void __launch_bounds__(1024) k_norm_dw(const float* __restrict__ part, int P, int H, float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < H)
#pragma unroll 4
    for (int p = warp; p < P; p += 32) v += part[(int64_t)p * H + c];
  s[warp][lane] = v;
  __syncthreads();
  v = s[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && blockIdx.x * 32 + warp < H) dw[blockIdx.x * 32 + warp] = v;
}

template <bool W32>
cudaError_t launch_bwd_t(NormBwdArgs a, float* dw, int num_sms, cudaStream_t st) {
  const int nch = a.H / 8;
  int64_t P = NORM_BWD_PARTS < a.T ? NORM_BWD_PARTS : a.T;
  auto run = [&](auto kern, std::atomic<int>& slot, int threads) {
    const int64_t fit = (int64_t)num_sms * blocks_per_sm(slot, kern, threads, 0, 1);
    if (P > fit) P = fit;
    kern<<<(unsigned)P, threads, 0, st>>>(a);
  };
  // one occupancy figure per CTA size (in warps) of each kernel
  static std::atomic<int> occ[4][17] = {};
  const int v = nch <= 256 ? 1 : nch <= 1024 ? 2 : 4;
  const int warps = nch > NORM_MAX_CHUNKS ? 16 : (nch + 32 * v - 1) / (32 * v);
  if (nch > NORM_MAX_CHUNKS) run(k_norm_bwd_long<W32>, occ[3][warps], warps * 32);
  else if (v == 1) run(k_norm_bwd<1, W32>, occ[0][warps], warps * 32);
  else if (v == 2) run(k_norm_bwd<2, W32>, occ[1][warps], warps * 32);
  else run(k_norm_bwd<4, W32>, occ[2][warps], warps * 32);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_norm_dw<<<(unsigned)((a.H + 31) / 32), 1024, 0, st>>>(a.part, (int)P, a.H, dw);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_fwd(const void* x, int64_t ldx, const void* r, int64_t ldr, const void* w, int w32, int64_t T,
                            int64_t H, float eps, void* h, void* y, float* rstd, int recipe, int kind, void* q,
                            void* scale, int scale_layout, cudaStream_t st) {
  NormFwdArgs a{};
  a.x = (const uint16_t*)x, a.r = (const uint16_t*)r;
  a.ldx = ldx, a.ldr = ldr, a.T = a.rows = T, a.H = (int)H;
  a.w = w, a.eps = eps, a.h = (uint16_t*)h, a.y = (uint16_t*)y, a.rstd = rstd, a.q = (uint8_t*)q;
  int out = NORM_OUT_NONE;
  if (q && recipe == FP8MOE_MXFP8) {
    out = NORM_OUT_MX;
    a.sc = make_spec((uint8_t*)scale, scale_layout, T, H / 32, nullptr, 0);
    if (scale_layout != FP8MOE_SCALES_ROWMAJOR) a.rows = a.sc.Rp;
  } else if (q) {
    out = kind == FP8MOE_E4M3FNUZ ? NORM_OUT_ROW_FNUZ : NORM_OUT_ROW;
    a.inv = (float*)scale;
  }
#define FP8MOE_NORM(O) \
  if (out == O) return w32 ? launch_fwd_t<O, true>(a, st) : launch_fwd_t<O, false>(a, st);
  FP8MOE_NORM(NORM_OUT_NONE)
  FP8MOE_NORM(NORM_OUT_MX)
  FP8MOE_NORM(NORM_OUT_ROW)
  FP8MOE_NORM(NORM_OUT_ROW_FNUZ)
#undef FP8MOE_NORM
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_bwd(const void* dy, const void* h, const float* rstd, const void* w, int w32, const void* dh,
                            int64_t T, int64_t H, void* dx, float* dw, void* workspace, int num_sms,
                            cudaStream_t st) {
  if (T == 0) return cudaMemsetAsync(dw, 0, (size_t)H * sizeof(float), st);
  NormBwdArgs a{};
  a.dy = (const uint16_t*)dy, a.h = (const uint16_t*)h, a.dh = (const uint16_t*)dh, a.rstd = rstd, a.w = w;
  a.T = T, a.H = (int)H, a.dx = (uint16_t*)dx, a.part = (float*)workspace;
  return w32 ? launch_bwd_t<true>(a, dw, num_sms, st) : launch_bwd_t<false>(a, dw, num_sms, st);
}

}  // namespace fp8moe
