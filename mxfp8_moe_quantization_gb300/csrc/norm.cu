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
// Both directions move each element once and are bound by HBM as long as they
// spend few instructions and keep enough loads in flight: packed fp32 pairs
// throughout; the forward holds a row in the registers of its warps and lets
// many CTAs overlap; the backward, whose share of dw has to stay with a CTA
// over many rows, streams them through a ring of bulk copies.  Measured (bytes
// that the formulas cannot do without, of a copy's 6.68 TB/s): 16384 x 5120
// with residual, bf16 and MXFP8 outputs 115 us (99%); 8191 x 4096 rowwise 41 us
// (85%: a sum and then a maximum a row); 16384 x 5120 backward 106 us (95%); one row of 7168
// 3.0 us in a graph.  The first forms took 116, 46, 118 and 3.4 us.
#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"
#include "scales.cuh"
#include "tma.cuh"

namespace fp8moe {
namespace {

// Threads of a CTA whose threads hold V 16-byte chunks per tensor (V = 1 in
// up to 64 registers, V = 2 and 4 in up to 128).
template <int V>
constexpr int norm_threads() { return V == 1 ? 1024 : 512; }
// The backward's: V = 1 and 2 in up to 96 registers, so that two CTAs of 320
// threads share an SM
template <int V>
constexpr int norm_bwd_threads() { return V == 4 ? 512 : 640; }
constexpr int NORM_BWD_STAGES = 4;   // most slots of its ring
constexpr int NORM_MAX_CHUNKS = 4 * norm_threads<4>();   // longer rows (H > 16384) take the looping kernels

constexpr int NORM_RED = 32;   // warps of a CTA

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
// eight values as four column pairs
struct Vec8 {
  uint64_t p[4];
};
FP8MOE_DEV Vec8 unpack8(const uint4& q) { return {{unpk_bf16(q.x), unpk_bf16(q.y), unpk_bf16(q.z), unpk_bf16(q.w)}}; }
FP8MOE_DEV uint4 pack8(const Vec8& v) {
  return make_uint4(pack_bf16x2(v.p[0]), pack_bf16x2(v.p[1]), pack_bf16x2(v.p[2]), pack_bf16x2(v.p[3]));
}
template <bool W32>
FP8MOE_DEV Vec8 load_w8(const void* w, int64_t ch) {
  if constexpr (W32) {
    const float4 a = reinterpret_cast<const float4*>(w)[2 * ch], b = reinterpret_cast<const float4*>(w)[2 * ch + 1];
    return {{pk(a.x, a.y), pk(a.z, a.w), pk(b.x, b.y), pk(b.z, b.w)}};
  } else {
    return unpack8(reinterpret_cast<const uint4*>(w)[ch]);
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
    v = MAX ? nanmax(v, u) : v + u;
  }
  if (wpr > 1) {
    // a row's values, every lane one of them, zero past the last (the maxima
    // are of magnitudes)
    if ((threadIdx.x & 31) == 0) red[group * wpr + wrow] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < wpr ? red[group * wpr + lane] : 0.0f;
    for (int o = wpr > 16 ? 16 : wpr > 8 ? 8 : wpr > 4 ? 4 : 2; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = MAX ? nanmax(v, u) : v + u;
    }
    v = __shfl_sync(0xffffffffu, v, 0);
  }
  return v;
}

// the eight codes of one chunk scaled by s
template <int OUT>
FP8MOE_DEV uint2 encode8(const Vec8& v, float s) {
  constexpr bool FZ = OUT == NORM_OUT_ROW_FNUZ;
  const uint64_t s2 = pk(enc_mul<FZ>(s), enc_mul<FZ>(s));
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpk(mul2(v.p[i], s2), f[2 * i], f[2 * i + 1]);
  return make_uint2(enc4_pre<FZ>(f[0], f[1], f[2], f[3]), enc4_pre<FZ>(f[4], f[5], f[6], f[7]));
}
FP8MOE_DEV float absmax8(float m, const Vec8& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = amax3(m, v.p[i]);
  return m;
}

// One chunk of y: its bf16 copy, codes and scale.  Every lane of the warp
// calls it (the block maximum is a shuffle over four lanes).
template <int OUT>
FP8MOE_DEV void put_chunk(const NormFwdArgs& a, int64_t row, int ch, bool ok, const Vec8& v, float s) {
  if (a.y && ok) *reinterpret_cast<uint4*>(a.y + row * a.H + (int64_t)ch * 8) = pack8(v);
  if constexpr (OUT == NORM_OUT_MX) {
    float m = absmax8(0.0f, v);
    m = nanmax(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = nanmax(m, __shfl_xor_sync(0xffffffffu, m, 2));
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

// The MXFP8 codes of a thread's V chunks, t, t + tpr, ...: a block's maximum is
// over four neighbouring lanes, among which the chunks' maxima are scattered as
// they are reduced, so that a lane derives one scale instead of V (20000 x 1024
// without residual: 13.4 us against 15.6 with every scale in every lane).
template <int V>
FP8MOE_DEV void put_mx(const NormFwdArgs& a, int64_t row, int t, int tpr, int nch, bool active, const Vec8 (&v)[V]) {
  const int lane = threadIdx.x & 31;
  const bool b0 = lane & 1, b1 = lane & 2;
  float m[V];
#pragma unroll
  for (int i = 0; i < V; ++i) m[i] = absmax8(0.0f, v[i]);
  float mk;
  int own = 0;
  if constexpr (V == 4) {
    float p[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      p[i] = nanmax(b0 ? m[i + 2] : m[i], __shfl_xor_sync(0xffffffffu, b0 ? m[i] : m[i + 2], 1));
    mk = nanmax(b1 ? p[1] : p[0], __shfl_xor_sync(0xffffffffu, b1 ? p[0] : p[1], 2));
    own = b0 * 2 + b1;
  } else {
    if constexpr (V == 2) {
      mk = nanmax(b0 ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, b0 ? m[0] : m[1], 1));
      own = b0;
    } else {
      mk = nanmax(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    }
    mk = nanmax(mk, __shfl_xor_sync(0xffffffffu, mk, 2));
  }
  float s;
  const uint32_t b = mx_byte(mk, s);
  const int ch = t + own * tpr;
  if (active && ch < nch && (V == 4 || !b1) && (V >= 2 || !b0)) {
    const int64_t c = ch >> 2;
    a.sc.p[a.sc.layout == FP8MOE_SCALES_ROWMAJOR ? row * (a.H / 32) + c : tile_off(row, c, a.sc.Cp)] = (uint8_t)b;
  }
  uint8_t* q = a.q + row * a.H + (int64_t)t * 8;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float si = V == 1 ? s : __shfl_sync(0xffffffffu, s, (lane & ~3) | (V == 4 ? i >> 1 | (i & 1) << 1 : i));
    if (active && t + i * tpr < nch) *reinterpret_cast<uint2*>(q + i * tpr * 8) = encode8<NORM_OUT_MX>(v[i], si);
  }
}

// the bytes of the 128x4 layout that stand for no block
FP8MOE_DEV void zero_scale_pad(const NormFwdArgs& a, int64_t row, int t, int n) {
  for (int64_t c = (row < a.T ? a.H / 32 : 0) + t; c < a.sc.Cp; c += n) a.sc.p[tile_off(row, c, a.sc.Cp)] = 0;
}

// A CTA holds `groups` rows, wpr warps each; a thread V chunks of its row.
template <int V, int OUT, bool W32>
__global__ void __launch_bounds__(norm_threads<V>()) k_norm_fwd(NormFwdArgs a, int wpr) {
  __shared__ float red[2][NORM_RED];
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
  // the weights ahead of the row's sum where registers allow
  constexpr bool EARLY_W = V <= 2;
  Vec8 we[EARLY_W ? V : 1];
  if constexpr (EARLY_W) {
#pragma unroll
    for (int i = 0; i < V; ++i) we[i] = t + i * tpr < nch ? load_w8<W32>(a.w, t + i * tpr) : Vec8{};
  }
  Vec8 v[V];
  uint64_t ss2 = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = unpack8(xv[i]);
    if (a.r) {
      const Vec8 f = unpack8(rv[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].p[j] = add2(v[i].p[j], f.p[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) ss2 = fma2(v[i].p[j], v[i].p[j], ss2);
  }
  const float ss = row_reduce<false>(sum_of(ss2), red[0], wpr, group, wrow);
  const float rstd = rsqrtf(__fdiv_rn(ss, (float)a.H) + a.eps);
  const uint64_t rstd2 = pk(rstd, rstd);
  if (active && a.rstd && t == 0) a.rstd[row] = rstd;
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ch = t + i * tpr;
    const bool ok = active && ch < nch;
    if (a.h && ok) *reinterpret_cast<uint4*>(a.h + row * a.H + (int64_t)ch * 8) = pack8(v[i]);
    const Vec8 wf = EARLY_W ? we[EARLY_W ? i : 0] : ok ? load_w8<W32>(a.w, ch) : Vec8{};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // (chunks past the row are zero, unless rstd is infinite)
      v[i].p[j] = OUT < NORM_OUT_ROW || ok ? mul2(mul2(v[i].p[j], rstd2), wf.p[j]) : 0;
    }
    if (OUT <= NORM_OUT_MX && a.y && ok) *reinterpret_cast<uint4*>(a.y + row * a.H + (int64_t)ch * 8) = pack8(v[i]);
    if (OUT >= NORM_OUT_ROW) am = absmax8(am, v[i]);
  }
  float s = 1.0f;
  if constexpr (OUT >= NORM_OUT_ROW) {
    am = row_reduce<true>(am, red[1], wpr, group, wrow);
    float inv;
    rowwise_scale<OUT == NORM_OUT_ROW_FNUZ>(am, s, inv);
    if (active && t == 0) a.inv[row] = inv;
  }
  if constexpr (OUT == NORM_OUT_MX) {
    put_mx(a, row, t, tpr, nch, active, v);
  } else if constexpr (OUT != NORM_OUT_NONE) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = t + i * tpr;
      put_chunk<OUT>(a, row, ch, active && ch < nch, v[i], s);
    }
  }
  if (OUT == NORM_OUT_MX && a.sc.layout != FP8MOE_SCALES_ROWMAJOR && row < a.rows) zero_scale_pad(a, row, t, tpr);
}

// Rows longer than a CTA's registers hold: one CTA per row, which reads the
// row again (from L2) for each pass.
template <int OUT, bool W32>
__global__ void __launch_bounds__(1024) k_norm_fwd_long(NormFwdArgs a) {
  __shared__ float red[2][NORM_RED];
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, n = blockDim.x, nch = a.H / 8;
  const bool active = row < a.T;
  auto load = [&](int ch) {
    Vec8 v = unpack8(ld16(a.x + row * a.ldx + (int64_t)ch * 8));
    if (a.r) {
      const Vec8 f = unpack8(ld16(a.r + row * a.ldr + (int64_t)ch * 8));
#pragma unroll
      for (int j = 0; j < 4; ++j) v.p[j] = add2(v.p[j], f.p[j]);
    }
    return v;
  };
  if (active) {
    uint64_t ss2 = 0;
    for (int ch = t; ch < nch; ch += n) {
      const Vec8 v = load(ch);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss2 = fma2(v.p[j], v.p[j], ss2);
    }
    const float ss = row_reduce<false>(sum_of(ss2), red[0], n / 32, 0, t >> 5);
    const float rstd = rsqrtf(__fdiv_rn(ss, (float)a.H) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    auto norm = [&](int ch, Vec8& v) {
      const Vec8 wf = load_w8<W32>(a.w, ch);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.p[j] = mul2(mul2(v.p[j], pk(rstd, rstd)), wf.p[j]);
    };
    float s = 1.0f;
    if constexpr (OUT >= NORM_OUT_ROW) {
      float am = 0.0f, inv;
      for (int ch = t; ch < nch; ch += n) {
        Vec8 v = load(ch);
        norm(ch, v);
        am = absmax8(am, v);
      }
      am = row_reduce<true>(am, red[1], n / 32, 0, t >> 5);
      rowwise_scale<OUT == NORM_OUT_ROW_FNUZ>(am, s, inv);
      if (t == 0) a.inv[row] = inv;
    }
    for (int c0 = 0; c0 < nch; c0 += n) {   // every lane takes every trip (block maxima are shuffles)
      const int ch = c0 + t;
      const bool ok = ch < nch;
      Vec8 v{};
      if (ok) {
        v = load(ch);
        if (a.h) *reinterpret_cast<uint4*>(a.h + row * a.H + (int64_t)ch * 8) = pack8(v);
        norm(ch, v);
      }
      put_chunk<OUT>(a, row, ch, ok, v, s);
    }
  }
  if (OUT == NORM_OUT_MX && a.sc.layout != FP8MOE_SCALES_ROWMAJOR) zero_scale_pad(a, row, t, n);
}

template <int OUT, bool W32>
cudaError_t launch_fwd_t(const NormFwdArgs& a, int num_sms, cudaStream_t st) {
  const int nch = a.H / 8;
  if (nch > NORM_MAX_CHUNKS) {
    k_norm_fwd_long<OUT, W32><<<(unsigned)a.rows, 1024, 0, st>>>(a);
    return cudaGetLastError();
  }
  // Chunks per thread: a row in one warp where that fits (no barriers), else
  // four, whose loads in flight carry HBM (8192 x 4096 rowwise: 41 us against
  // 47 with two and 62 with one); with fewer rows than SMs, where one row's
  // latency counts, fewer chunks and more threads (one row of 4096: 2.6 us
  // against 3.0).  CTAs of four warps or one row.
  const bool few = a.T < num_sms;
  const int v = few ? (nch <= 512 ? 1 : nch <= 1024 ? 2 : 4) : nch <= 32 ? 1 : nch <= 64 ? 2 : 4;
  const int wpr = (nch + 32 * v - 1) / (32 * v);
  const int groups = wpr >= 4 ? 1 : 4 / wpr;
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
  const uint8_t *hq, *hs;   // h in MXFP8, row-major scales (the checkpointed forms)
  const float* rstd;
  const void* w;
  int64_t T;
  int H;
  uint16_t* dx;
  float* part;  // [gridDim.x][H] partial weight gradients
  int* status;
  int stall;    // test hook: the first CTA never loads its first rows
};

// A CTA takes blocks of `groups` consecutive rows, blockIdx.x, blockIdx.x +
// gridDim.x, ..., wpr warps a row; a thread keeps the same V chunks of every
// row, so its share of dw stays in registers.  The blocks come through a ring
// of `stages` slots that thread 0 fills with bulk copies: the slot of a block
// is free at the next block's barrier (every thread has then read it).
template <int V, bool W32>
__global__ void __launch_bounds__(norm_bwd_threads<V>()) k_norm_bwd(NormBwdArgs a, int wpr, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][NORM_RED];
  __shared__ uint64_t full[NORM_BWD_STAGES];
  __shared__ int abort_s, fills[NORM_BWD_STAGES];   // fills: thread 0's count per slot
  volatile int* abort_flag = &abort_s;
  const int tpr = wpr * 32, groups = blockDim.x / tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
  const int nch = a.H / 8;
  const uint32_t row_bytes = (uint32_t)a.H * 2, ten_bytes = row_bytes * groups;
  const uint32_t slot_bytes = ten_bytes * (a.dh ? 3 : 2);
  const int blocks = (int)((a.T + groups - 1) / groups);
  // thread 0: block nblk, the next to load, goes to slot nslot
  int nblk = blockIdx.x, nslot = 0;
  auto issue = [&]() {
    uint8_t* dst = ring + nslot * slot_bytes;
    const int64_t r0 = (int64_t)nblk * groups, at = r0 * a.H;
    const uint32_t bytes = row_bytes * (uint32_t)(a.T - r0 < groups ? a.T - r0 : groups);
    if (!a.stall || nblk > 0) {
      ++fills[nslot];
      mbar_expect_tx(&full[nslot], bytes * (a.dh ? 3 : 2));
      bulk_load(dst, a.dy + at, bytes, &full[nslot]);
      bulk_load(dst + ten_bytes, a.h + at, bytes, &full[nslot]);
      if (a.dh) bulk_load(dst + 2 * ten_bytes, a.dh + at, bytes, &full[nslot]);
    }
    nblk += gridDim.x;
    if (++nslot == stages) nslot = 0;
  };
  const float rh = __frcp_rn((float)a.H);
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      fills[s] = 0;
    }
    mbar_fence_init();
    for (int s = 0; s < stages - 1 && nblk < blocks; ++s) issue();
  }
  Vec8 dw[V];
  // bf16 weights stay in registers where there is room; others come from L1
  constexpr bool KEEP_W = !W32 && V <= 2;
  uint4 w4[KEEP_W ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    dw[i] = Vec8{};
    if constexpr (KEEP_W)
      w4[i] = t + i * tpr < nch ? reinterpret_cast<const uint4*>(a.w)[t + i * tpr] : make_uint4(0, 0, 0, 0);
  }
  // a row's rstd is loaded one block ahead (rows past T: 0, and nothing stored)
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  const float* prstd = a.rstd + row;
  uint16_t* pdx = a.dx + row * a.H + t * 8;
  float rstd = row < a.T ? *prstd : 0.0f;
  __syncthreads();
  int s = 0, par = 0;
  uint32_t phase = 0;
  for (int b = blockIdx.x; b < blocks; b += gridDim.x, row += step, pdx += step * a.H) {
    const bool live = row < a.T;
    prstd += step;
    const float rstd_next = row + step < a.T ? *prstd : 0.0f;
    const uint64_t rstd2 = pk(rstd, rstd);
    if (!mbar_wait(&full[s], phase, abort_flag)) {
      set_status(a.status, FP8MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    const uint8_t* src = ring + s * slot_bytes + group * row_bytes;
    Vec8 g[V], xh[V];
    uint64_t dot2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = t + i * tpr;
      if (ch >= nch || !live) continue;
      const uint4 dq = *reinterpret_cast<const uint4*>(src + ch * 16);
      const Vec8 d = unpack8(dq), x = unpack8(*reinterpret_cast<const uint4*>(src + ten_bytes + ch * 16));
      if constexpr (!KEEP_W) {
        const Vec8 wf = load_w8<W32>(a.w, ch);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[i].p[j] = mul2(d.p[j], wf.p[j]);
      } else {
        g[i] = {{mulx(dq.x, w4[i].x), mulx(dq.y, w4[i].y), mulx(dq.z, w4[i].z), mulx(dq.w, w4[i].w)}};
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xh[i].p[j] = mul2(x.p[j], rstd2);
        dot2 = fma2(g[i].p[j], xh[i].p[j], dot2);
        dw[i].p[j] = fma2(d.p[j], xh[i].p[j], dw[i].p[j]);
      }
    }
    // the two halves of `red` alternate: a block's sums are read before the
    // barrier of the next one, which writes the other half
    const float dot = row_reduce<false>(sum_of(dot2), red[par], wpr, group, (threadIdx.x >> 5) - group * wpr);
    par ^= 1;
    if (wpr == 1) __syncthreads();
    // past this barrier every thread has read the block before
    if (threadIdx.x == 0 && nblk < blocks && !*abort_flag) {
      fence_proxy_async_smem();
      issue();
    }
    // -dot / H, rounded once: the quotient by the reciprocal and one step of
    // Markstein's correction, which an infinite sum has no use for
    const float m = dot * rh, rest = fmaf(-m, (float)a.H, dot);
    const float c = rest == rest ? -fmaf(rest, rh, m) : -m;
    const uint64_t c2 = pk(c, c);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = t + i * tpr;
      if (ch >= nch || !live) continue;
      const Vec8 sv = a.dh ? unpack8(*reinterpret_cast<const uint4*>(src + 2 * ten_bytes + ch * 16)) : Vec8{};
      Vec8 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.p[j] = fma2(rstd2, fma2(xh[i].p[j], c2, g[i].p[j]), sv.p[j]);
      *reinterpret_cast<uint4*>(pdx + i * tpr * 8) = pack8(o);
    }
    rstd = rstd_next;
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");
  // after a wait that ran out blocks may be in flight still: none may land in
  // shared memory that is no longer this CTA's
  if (threadIdx.x == 0 && *abort_flag)
    for (int i = 0; i < stages; ++i)
      if (fills[i] > 0) (void)mbar_wait(&full[i], (uint32_t)(fills[i] - 1) & 1u, nullptr);
  // the groups' shares of dw, added in order through the ring's memory
  float* sum = reinterpret_cast<float*>(ring);
  for (int q = 0; q < groups; ++q) {
    __syncthreads();
    if (group != q) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = t + i * tpr;
      if (ch >= nch) continue;
      uint64_t* p = reinterpret_cast<uint64_t*>(sum + ch * 8);
      uint64_t* out = reinterpret_cast<uint64_t*>(a.part + (int64_t)blockIdx.x * a.H + (int64_t)ch * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t v = q == 0 ? dw[i].p[j] : add2(p[j], dw[i].p[j]);
        if (q == groups - 1) {
          out[j] = v;
        } else {
          p[j] = v;
        }
      }
    }
  }
}

// Backward from a checkpoint of h: e4m3 codes through the ring, behind dy and dh,
// and row-major scale bytes by plain loads a block ahead.  As the bf16 form, but a
// thread takes R rows at a time where rows are short: what a row costs besides its
// elements (the wait, the sum over its warps, addresses) is as many instructions as
// two chunks.
//
// HBM's share is 7.03 bytes an element with dh, 5.03 without, an eighth to a sixth
// below the bf16 form's, but the codes' unpacking (a conversion to fp16 pairs, two to
// fp32, a product by the block's power of two) comes on top of its instructions, and
// from about 20 an element on it is issue and latency that bound: 16384 x 5120 with
// dh 99 us = 5.9 TB/s (89% of a copy's rate), 16384 x 7168 131 us = 6.3, 20001 x 4096
// 100 us = 5.7, 65536 x 512 49 us = 4.8.  Rows of more than 8192 elements, four chunks a
// thread, have one CTA an SM: 8192 x 12288 195 us = 3.6 TB/s, the bf16 form 164.
template <int V, int R>
constexpr int norm_ck_threads() { return R == 4 ? 256 : R == 2 || V == 4 ? 512 : 640; }
template <int V, int R>
constexpr int norm_ck_ctas() { return R == 4 ? 2 : 1; }

template <int V, int R, bool W32>
__global__ void __launch_bounds__(norm_ck_threads<V, R>(), norm_ck_ctas<V, R>()) k_norm_bwd_ckpt(NormBwdArgs a, int wpr, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][NORM_RED * R];
  __shared__ uint64_t full[NORM_BWD_STAGES];
  __shared__ int abort_s, fills[NORM_BWD_STAGES];   // fills: thread 0's count per slot
  volatile int* abort_flag = &abort_s;
  const int tpr = wpr * 32, groups = blockDim.x / tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
  const int nch = a.H / 8, ns = a.H / 32, block = groups * R;
  const uint32_t row_bytes = (uint32_t)a.H * 2, ten_bytes = row_bytes * block;
  const uint32_t slot_bytes = ten_bytes / 2 * (a.dh ? 5 : 3), at_h = a.dh ? 2 * ten_bytes : ten_bytes;
  const int blocks = (int)((a.T + block - 1) / block);
  // thread 0: block nblk, the next to load, goes to slot nslot
  int nblk = blockIdx.x, nslot = 0;
  auto issue = [&]() {
    uint8_t* dst = ring + nslot * slot_bytes;
    const int64_t r0 = (int64_t)nblk * block, at = r0 * a.H;
    const uint32_t bytes = row_bytes * (uint32_t)(a.T - r0 < block ? a.T - r0 : block);
    if (!a.stall || nblk > 0) {
      ++fills[nslot];
      mbar_expect_tx(&full[nslot], bytes / 2 * (a.dh ? 5 : 3));
      bulk_load(dst, a.dy + at, bytes, &full[nslot]);
      if (a.dh) bulk_load(dst + ten_bytes, a.dh + at, bytes, &full[nslot]);
      bulk_load(dst + at_h, a.hq + at, bytes / 2, &full[nslot]);
    }
    nblk += gridDim.x;
    if (++nslot == stages) nslot = 0;
  };
  const float rh = __frcp_rn((float)a.H);
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      fills[s] = 0;
    }
    mbar_fence_init();
    for (int s = 0; s < stages - 1 && nblk < blocks; ++s) issue();
  }
  Vec8 dw[V];
  // the weights stay in registers where there is room (fp32, 16384 x 5120 with dh: 118
  // us from L1, 111), else they come from L1 (20001 x 4096: 107 us, 117 with spills)
  constexpr bool KEEP_W = !W32 && V <= 2, KEEP_W32 = W32 && V == 2 && R == 1;
  uint4 w4[KEEP_W ? V : 1];
  Vec8 wf[KEEP_W32 ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    dw[i] = Vec8{};
    if constexpr (KEEP_W)
      w4[i] = t + i * tpr < nch ? reinterpret_cast<const uint4*>(a.w)[t + i * tpr] : make_uint4(0, 0, 0, 0);
    if constexpr (KEEP_W32) wf[i] = t + i * tpr < nch ? load_w8<W32>(a.w, t + i * tpr) : Vec8{};
  }
  // the rows' rstd and scales are loaded one block ahead (rows past T: 0, and nothing stored)
  uint32_t row = blockIdx.x * block + group * R;
  const uint32_t T = (uint32_t)a.T, step = gridDim.x * block;
  const float* prstd = a.rstd + row;
  const uint8_t* phs = a.hs + (int64_t)row * ns + (t >> 2);
  uint16_t* pdx = a.dx + (int64_t)row * a.H + t * 8;
  float rstd_next[R];
  uint32_t sc_next[R][V];
  auto ahead = [&](uint32_t r0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool on = r0 + r < T;
      rstd_next[r] = on ? __ldg(prstd + r) : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sc_next[r][i] = on && t + i * tpr < nch ? (uint32_t)__ldg(phs + r * ns + i * (tpr >> 2)) : 0u;
    }
    prstd += step;
    phs += (int64_t)step * ns;
  };
  ahead(row);
  __syncthreads();
  int s = 0, par = 0;
  uint32_t phase = 0;
  for (int b = blockIdx.x; b < blocks; b += gridDim.x, row += step, pdx += (int64_t)step * a.H) {
    // of a row's chunk: 2^e and 2^e rstd
    float rstd[R], xs[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = rstd_next[r];
#pragma unroll
      for (int i = 0; i < V; ++i) xs[r][i] = mx_power(sc_next[r][i]);
    }
    ahead(row + step);
    if (!mbar_wait(&full[s], phase, abort_flag)) {
      set_status(a.status, FP8MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    const uint8_t* src = ring + s * slot_bytes + group * R * row_bytes;
    const uint8_t* src_h = ring + s * slot_bytes + at_h + group * R * (row_bytes / 2);
    Vec8 g[R][V], xh[R][V];
    uint64_t dot2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      dot2[r] = 0;
      const uint64_t rstd2 = pk(rstd[r], rstd[r]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int ch = t + i * tpr;
        if (ch >= nch || row + r >= T) continue;
        const uint4 dq = *reinterpret_cast<const uint4*>(src + r * row_bytes + ch * 16);
        const Vec8 d = unpack8(dq);
        mx_unpack8(*reinterpret_cast<const uint2*>(src_h + r * (row_bytes / 2) + ch * 8), xs[r][i], xh[r][i].p);
        if constexpr (!KEEP_W) {
          const Vec8 w = KEEP_W32 ? wf[KEEP_W32 ? i : 0] : load_w8<W32>(a.w, ch);
#pragma unroll
          for (int j = 0; j < 4; ++j) g[r][i].p[j] = mul2(d.p[j], w.p[j]);
        } else {
          g[r][i] = {{mulx(dq.x, w4[i].x), mulx(dq.y, w4[i].y), mulx(dq.z, w4[i].z), mulx(dq.w, w4[i].w)}};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xh[r][i].p[j] = mul2(xh[r][i].p[j], rstd2);
          dot2[r] = fma2(g[r][i].p[j], xh[r][i].p[j], dot2[r]);
          dw[i].p[j] = fma2(d.p[j], xh[r][i].p[j], dw[i].p[j]);
        }
      }
    }
    float dot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = sum_of(dot2[r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], o);
    // the two halves of `red` alternate: a block's sums are read before the
    // barrier of the next one, which writes the other half
    if (wpr > 1 && (threadIdx.x & 31) == 0)
#pragma unroll
      for (int r = 0; r < R; ++r) red[par][(threadIdx.x >> 5) * R + r] = dot[r];
    __syncthreads();
    // past this barrier every thread has read the block before
    if (threadIdx.x == 0 && nblk < blocks && !*abort_flag) {
      fence_proxy_async_smem();
      issue();
    }
    if (wpr > 1) {
      const float* p = red[par] + group * wpr * R;
#pragma unroll
      for (int r = 0; r < R; ++r) dot[r] = p[r];
      for (int i = 1; i < wpr; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) dot[r] += p[i * R + r];
    }
    par ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // -dot / H, rounded once: the quotient by the reciprocal and one step of
      // Markstein's correction, which an infinite sum has no use for
      const float m = dot[r] * rh, rest = fmaf(-m, (float)a.H, dot[r]);
      const float c = rest == rest ? -fmaf(rest, rh, m) : -m;
      const uint64_t c2 = pk(c, c), rstd2 = pk(rstd[r], rstd[r]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int ch = t + i * tpr;
        if (ch >= nch || row + r >= T) continue;
        const Vec8 sv = a.dh ? unpack8(*reinterpret_cast<const uint4*>(src + ten_bytes + r * row_bytes + ch * 16)) : Vec8{};
        Vec8 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.p[j] = fma2(rstd2, fma2(xh[r][i].p[j], c2, g[r][i].p[j]), sv.p[j]);
        *reinterpret_cast<uint4*>(pdx + r * a.H + i * tpr * 8) = pack8(o);
      }
    }
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");
  // after a wait that ran out blocks may be in flight still: none may land in
  // shared memory that is no longer this CTA's
  if (threadIdx.x == 0 && *abort_flag)
    for (int i = 0; i < stages; ++i)
      if (fills[i] > 0) (void)mbar_wait(&full[i], (uint32_t)(fills[i] - 1) & 1u, nullptr);
  // the groups' shares of dw, added in order through the ring's memory
  float* sum = reinterpret_cast<float*>(ring);
  for (int q = 0; q < groups; ++q) {
    __syncthreads();
    if (group != q) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = t + i * tpr;
      if (ch >= nch) continue;
      uint64_t* p = reinterpret_cast<uint64_t*>(sum + ch * 8);
      uint64_t* out = reinterpret_cast<uint64_t*>(a.part + (int64_t)blockIdx.x * a.H + (int64_t)ch * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t v = q == 0 ? dw[i].p[j] : add2(p[j], dw[i].p[j]);
        if (q == groups - 1) {
          out[j] = v;
        } else {
          p[j] = v;
        }
      }
    }
  }
}

// Rows longer than that: the row is read twice (the second time from L2) and
// a thread's share of dw stays in its CTA's row of the partials.
template <bool W32, bool CK>
__global__ void __launch_bounds__(512) k_norm_bwd_long(NormBwdArgs a, int, int) {
  __shared__ float red[2][NORM_RED];
  const int t = threadIdx.x, n = blockDim.x, nch = a.H / 8;
  float* part = a.part + (int64_t)blockIdx.x * a.H;
  auto load_h = [&](int64_t at) {
    if constexpr (CK) {
      Vec8 x;
      mx_unpack8(__ldg(reinterpret_cast<const uint2*>(a.hq + at)), mx_power(__ldg(a.hs + (at >> 5))), x.p);
      return x;
    } else {
      return unpack8(ld16(a.h + at));
    }
  };
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, par ^= 1) {
    const float rstd = a.rstd[row];
    const uint64_t rstd2 = pk(rstd, rstd);
    uint64_t dot2 = 0;
    for (int ch = t; ch < nch; ch += n) {
      const Vec8 d = unpack8(ld16(a.dy + row * a.H + (int64_t)ch * 8));
      const Vec8 x = load_h(row * a.H + (int64_t)ch * 8), wf = load_w8<W32>(a.w, ch);
#pragma unroll
      for (int j = 0; j < 4; ++j) dot2 = fma2(mul2(d.p[j], wf.p[j]), mul2(x.p[j], rstd2), dot2);
    }
    const float dot = row_reduce<false>(sum_of(dot2), red[par], n >> 5, 0, t >> 5);
    const float c = -__fdiv_rn(dot, (float)a.H);
    for (int ch = t; ch < nch; ch += n) {
      const int64_t at = row * a.H + (int64_t)ch * 8;
      const Vec8 d = unpack8(ld16(a.dy + at)), x = load_h(at), wf = load_w8<W32>(a.w, ch);
      const Vec8 sv = a.dh ? unpack8(ld16(a.dh + at)) : Vec8{};
      uint64_t* p = reinterpret_cast<uint64_t*>(part + (int64_t)ch * 8);
      Vec8 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t xh = mul2(x.p[j], rstd2);
        p[j] = fma2(d.p[j], xh, row == blockIdx.x ? 0 : p[j]);
        o.p[j] = fma2(rstd2, fma2(xh, pk(c, c), mul2(d.p[j], wf.p[j])), sv.p[j]);
      }
      *reinterpret_cast<uint4*>(a.dx + at) = pack8(o);
    }
  }
}

// dw[c] = sum over the P partials in order: 32 columns per CTA, 32 warps that
// each take every 32nd partial, then a fixed-order sum over the warps.
__global__ void __launch_bounds__(1024) k_norm_dw(const float* part, int P, int H, float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c < H)
#pragma unroll 10
    for (int p = warp; p < P; p += 32) v += part[(int64_t)p * H + c];
  s[warp][lane] = v;
  __syncthreads();
  v = s[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && blockIdx.x * 32 + warp < H) dw[blockIdx.x * 32 + warp] = v;
}

cudaError_t launch_dw(const NormBwdArgs& a, int P, float* dw, cudaStream_t st) {
  // launched ahead of the first kernel's end, for which it waits
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.H + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_dw, (const float*)a.part, P, a.H, dw);
}

template <bool W32>
cudaError_t launch_bwd_t(NormBwdArgs a, float* dw, int num_sms, int max_smem, cudaStream_t st) {
  const int nch = a.H / 8;
  // One chunk a thread while rows are short and there is more to read for it than
  // dy and h (20000 x 1024 with dh: fp32 weights 32.6 us against 35.6 with two,
  // bf16 30.2 against 31.6; without dh and with bf16 weights 26.4 against 26.2,
  // and 31.6 against 30.3 on 12000 x 2048)
  const int v = nch <= (W32 || a.dh ? 256 : 32) ? 1 : nch <= 1024 ? 2 : 4;
  // CTAs of eight warps or one row (65536 x 512: 50 us, 114 with a row per CTA)
  int wpr = nch > NORM_MAX_CHUNKS ? 16 : (nch + 32 * v - 1) / (32 * v);
  int groups = wpr >= 8 ? 1 : 8 / wpr;
  // The ring: as deep as lets two CTAs share an SM, at least three blocks if
  // they fit one (16384 x 5120: 108 us with three, 132 with two)
  const int64_t budget = max_smem - 2048;
  const int64_t slot = (int64_t)a.H * 2 * (a.dh ? 3 : 2) * groups;
  int stages = (int)(budget / 2 / slot < NORM_BWD_STAGES ? budget / 2 / slot : NORM_BWD_STAGES);
  if (stages < 3) stages = slot * 3 <= budget ? 3 : 2;
  const bool ring = nch <= NORM_MAX_CHUNKS && slot * stages <= budget;
  if (!ring) wpr = 16, groups = 1;
  const int64_t blocks = (a.T + groups - 1) / groups;
  int64_t P = NORM_BWD_PARTS < blocks ? NORM_BWD_PARTS : blocks;
  if (ring) a.stall = take_ring_stall_hook();
  auto run = [&](auto kern) {
    const int smem = ring ? (int)(slot * stages) : 0;
    // (the limit belongs to the kernel and every host thread that launches it:
    // always the same, whatever this call's rows take of it)
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring ? (int)budget : 0);
    int per = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, wpr * 32 * groups, smem);
    if (e != cudaSuccess || per < 1) return e == cudaSuccess ? cudaErrorInvalidConfiguration : e;
    if (P > (int64_t)num_sms * per) P = (int64_t)num_sms * per;
    kern<<<(unsigned)P, wpr * 32 * groups, smem, st>>>(a, wpr, stages);
    return cudaGetLastError();
  };
  cudaError_t e = !ring    ? run(k_norm_bwd_long<W32, false>)
                  : v == 1 ? run(k_norm_bwd<1, W32>)
                  : v == 2 ? run(k_norm_bwd<2, W32>)
                           : run(k_norm_bwd<4, W32>);
  if (e != cudaSuccess) return e;
  return launch_dw(a, (int)P, dw, st);
}

template <bool W32>
cudaError_t launch_bwd_ckpt(NormBwdArgs a, float* dw, int num_sms, int max_smem, cudaStream_t st) {
  const int nch = a.H / 8;
  // Chunks and rows of a thread at a time.  Several rows where they are short
  // (65536 x 512 with dh: 54 us with one, 48 with four), and where registers leave
  // room for one CTA an SM anyway (16384 x 7168: 164 and 131 with two); in between two
  // CTAs of one row each are better (16384 x 5120: 99, 111 with two rows).
  const int v = nch <= 256 ? 1 : nch <= 1024 ? 2 : 4, rows = nch <= 256 ? 4 : nch <= 512 || (nch > 640 && nch <= 1024) ? 2 : 1;
  int wpr = nch > NORM_MAX_CHUNKS ? 16 : (nch + 32 * v - 1) / (32 * v);
  int groups = wpr >= 8 ? 1 : 8 / wpr;
  // the ring as the bf16 form's, and as deep as fits where registers leave room for
  // one CTA only (16384 x 7168 without dh: 115 us, 145 with half the memory)
  const int64_t budget = max_smem - 2048;
  const int64_t slot = (int64_t)a.H * (a.dh ? 5 : 3) * groups * rows;
  const int64_t room = budget / (wpr * groups > (rows == 1 && v == 2 ? 10 : 8) ? 1 : 2);
  int stages = (int)(room / slot < NORM_BWD_STAGES ? room / slot : NORM_BWD_STAGES);
  if (stages < (rows > 1 ? 2 : 3)) stages = slot * 3 <= budget ? 3 : 2;
  const bool ring = nch <= NORM_MAX_CHUNKS && slot * stages <= budget;
  if (!ring) wpr = 16, groups = 1;
  const int64_t blocks = ring ? (a.T + groups * rows - 1) / (groups * rows) : a.T;
  int64_t P = NORM_BWD_PARTS < blocks ? NORM_BWD_PARTS : blocks;
  if (ring) a.stall = take_ring_stall_hook();
  auto run = [&](auto kern) {
    const int smem = ring ? (int)(slot * stages) : 0;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring ? (int)budget : 0);
    int per = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, wpr * 32 * groups, smem);
    if (e != cudaSuccess || per < 1) return e == cudaSuccess ? cudaErrorInvalidConfiguration : e;
    if (P > (int64_t)num_sms * per) P = (int64_t)num_sms * per;
    kern<<<(unsigned)P, wpr * 32 * groups, smem, st>>>(a, wpr, stages);
    return cudaGetLastError();
  };
  const cudaError_t e = !ring      ? run(k_norm_bwd_long<W32, true>)
                        : v == 1    ? run(k_norm_bwd_ckpt<1, 4, W32>)
                        : rows == 2 ? run(k_norm_bwd_ckpt<2, 2, W32>)
                        : v == 2    ? run(k_norm_bwd_ckpt<2, 1, W32>)
                                    : run(k_norm_bwd_ckpt<4, 1, W32>);
  return e != cudaSuccess ? e : launch_dw(a, (int)P, dw, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const void* x, int64_t ldx, const void* r, int64_t ldr, const void* w, int w32, int64_t T,
                            int64_t H, float eps, void* h, void* y, float* rstd, int recipe, int kind, void* q,
                            void* scale, int scale_layout, int num_sms, cudaStream_t st) {
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
  if (out == O) return w32 ? launch_fwd_t<O, true>(a, num_sms, st) : launch_fwd_t<O, false>(a, num_sms, st);
  FP8MOE_NORM(NORM_OUT_NONE)
  FP8MOE_NORM(NORM_OUT_MX)
  FP8MOE_NORM(NORM_OUT_ROW)
  FP8MOE_NORM(NORM_OUT_ROW_FNUZ)
#undef FP8MOE_NORM
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_bwd(const void* dy, const void* h, const uint8_t* hs, const float* rstd, const void* w, int w32,
                            const void* dh, int64_t T, int64_t H, void* dx, float* dw, void* workspace, int num_sms, int max_smem,
                            int* status, cudaStream_t st) {
  if (T == 0) return cudaMemsetAsync(dw, 0, (size_t)H * sizeof(float), st);
  NormBwdArgs a{};
  a.dy = (const uint16_t*)dy, a.h = (const uint16_t*)h, a.hq = (const uint8_t*)h, a.hs = hs, a.dh = (const uint16_t*)dh, a.rstd = rstd, a.w = w;
  a.T = T, a.H = (int)H, a.dx = (uint16_t*)dx, a.part = (float*)workspace, a.status = status;
  if (hs) return w32 ? launch_bwd_ckpt<true>(a, dw, num_sms, max_smem, st) : launch_bwd_ckpt<false>(a, dw, num_sms, max_smem, st);
  return w32 ? launch_bwd_t<true>(a, dw, num_sms, max_smem, st) : launch_bwd_t<false>(a, dw, num_sms, max_smem, st);
}

}  // namespace fp8moe
