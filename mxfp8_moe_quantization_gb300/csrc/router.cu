// The router of an MoE layer: scores, top-k choice, weights, per-expert
// counts and the balance loss; its gradient; and the gradient of the weights
// with which the combine sums the experts' rows.
//
// Forward, per token (fp32): s = softmax(l) or sigmoid(l); the k experts with
// the largest keys (l, or s + bias), ties to the lowest id; w = s[ids],
// divided by their sum when renormalized, times a scale.  p = s (softmax) or
// s / sum(s) (sigmoid); P_e = sum of p over the tokens, n_e = how often e was
// chosen, N = tokens; loss = E / (k N^2) * sum_e n_e P_e.
// A masked token has every logit at -inf.  An expert at -inf has s = 0, is
// chosen only when no other is left, and then has weight 0 and is not counted.
// Backward: c_e = dloss * E / (k N^2) * n_e (the counts are constants),
//   r = p (c - sum(p c)),
//   u_j = scale * w'_j (dw_j - sum_i dw_i w'_i)  (w' = renormalized scores) or
//   u_j = scale * s_j dw_j,
//   softmax: dl = r + u - p sum(u);   sigmoid: dl = (1 - s)(r + u).
//
// A warp takes a token, a lane every 32nd expert; the logits are read once.
// Sums over tokens have a fixed order (registers, then warps, then CTAs), so
// results do not change from run to run.
#include "common.cuh"
#include "launch.h"
#include "moe_ops.h"

namespace fp8moe {
namespace {

constexpr int RW = 8;               // warps per CTA
constexpr int SINGLE_CTA_T = 2 * RW;  // up to so many tokens one CTA does everything

// order-preserving key: larger float, larger key; NaN sorts with -inf; every
// key is above 0, the mark of what is taken or absent
FP8MOE_DEV uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);   // -0 and 0 are equal
  if (f != f) return 0x007FFFFFu;
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

FP8MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
FP8MOE_DEV float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

constexpr float NEG_INF = -__builtin_huge_valf();

template <int V>
FP8MOE_DEV void load_row(const RouterArgs& a, int64_t t, int lane, bool on, float (&x)[V]) {
  if (a.bf16) {
    const uint16_t* p = (const uint16_t*)a.logits + t * a.ld;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      x[i] = on && e < a.E ? __uint_as_float((uint32_t)p[e] << 16) : NEG_INF;
    }
  } else {
    const float* p = (const float*)a.logits + t * a.ld;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      x[i] = on && e < a.E ? p[e] : NEG_INF;
    }
  }
}

// Scores s and probabilities p of a row; returns (for softmax) the maximum
// and the sum that turn another logit of the row into its score.
struct RowStat {
  float m, z;
};
FP8MOE_DEV float sigmoid_rn(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }
template <int V, bool SIG>
FP8MOE_DEV RowStat row_scores(const float (&x)[V], float (&s)[V], float (&p)[V]) {
  RowStat st{0.0f, 0.0f};
  float z = 0.0f;
  if constexpr (SIG) {
#pragma unroll
    for (int i = 0; i < V; ++i) z += s[i] = sigmoid_rn(x[i]);
  } else {
    float m = NEG_INF;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    st.m = m == NEG_INF ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < V; ++i) z += s[i] = expf(x[i] - st.m);
  }
  z = warp_sum(z);
  st.z = z == 0.0f ? 1.0f : z;   // a row of nothing but -inf is all zero
#pragma unroll
  for (int i = 0; i < V; ++i) {
    p[i] = __fdiv_rn(s[i], st.z);
    if constexpr (!SIG) s[i] = p[i];
  }
  return st;
}

// counts and probability sums of one CTA (acc: this warp's lanes' sums) into
// shared memory, summed over its warps in order
struct CtaSums {
  float p[RW][ROUTER_MAX_E];
  int n[ROUTER_MAX_E + 1];
};

FP8MOE_DEV void final_sums(const RouterArgs& a, int E, const float* psum, const int* n, float* red) {
  // loss from the whole sums; every thread of the CTA calls it
  float v = 0.0f;
  for (int e = threadIdx.x; e < E; e += blockDim.x) v = fmaf((float)n[e], psum[e], v);
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0.0f;
    v = warp_sum(v);
    if (threadIdx.x == 0) {
      const float N = fmaxf((float)n[E], 1.0f);
      a.loss[0] = v * __fdiv_rn((float)E, (float)a.k) / (N * N);
    }
  }
}

template <int V, bool SIG>
__global__ void __launch_bounds__(RW * 32) k_router_fwd(RouterArgs a) {
  __shared__ CtaSums cs;
  __shared__ float red[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool sums = a.counts != nullptr;
  float acc[V] = {};
  int tokens = 0;
  if (sums) {
    for (int e = threadIdx.x; e <= a.E; e += RW * 32) cs.n[e] = 0;
    __syncthreads();
  }
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = a.bias && i * 32 + lane < a.E ? a.bias[i * 32 + lane] : 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * RW + warp; t < a.T; t += (int64_t)gridDim.x * RW) {
    const bool on = !a.mask || a.mask[t] != 0;
    float x[V], s[V], p[V];
    load_row<V>(a, t, lane, on, x);
    row_scores<V, SIG>(x, s, p);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[i] += p[i];
      // dead experts stay below every other whatever their bias
      const float f = !a.bias ? x[i] : x[i] == NEG_INF ? NEG_INF : s[i] + bias[i];
      key[i] = i * 32 + lane < a.E ? order_key(f) : 0u;
    }
    tokens += on;
    // k rounds: the warp's largest key, then the lowest id that has it
    int my_e = 0;
    float my_w = 0.0f;
    bool my_live = false;
    for (int j = 0; j < a.k; ++j) {
      uint32_t bk = 0;
      int be = INT32_MAX;
      float bs = 0.0f;
      bool bl = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool up = key[i] > bk;   // ascending ids: the first of equal keys stays
        bk = up ? key[i] : bk;
        be = up ? i * 32 + lane : be;
        bs = up ? s[i] : bs;
        bl = up ? x[i] != NEG_INF : bl;
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
      const int e = (int)__reduce_min_sync(0xffffffffu, bk == top ? (uint32_t)be : (uint32_t)INT32_MAX);
      const float ws = __shfl_sync(0xffffffffu, bs, e & 31);
      const bool wl = __shfl_sync(0xffffffffu, (int)bl, e & 31) != 0;
      if (lane == j) {
        my_e = e;
        my_w = ws;
        my_live = wl;
      }
      if (lane == (e & 31)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i == (e >> 5)) key[i] = 0u;
      }
    }
    if (a.renorm) {
      const float z = warp_sum(lane < a.k ? my_w : 0.0f);
      my_w = __fdiv_rn(my_w, z == 0.0f ? 1.0f : z);
    }
    if (lane < a.k) {
      a.idx[t * a.k + lane] = my_e;
      a.w[t * a.k + lane] = my_w * a.route_scale;
      if (sums && my_live) atomicAdd(&cs.n[my_e], 1);
    }
  }
  if (!sums) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * 32 + lane < a.E) cs.p[warp][i * 32 + lane] = acc[i];
  if (lane == 0) atomicAdd(&cs.n[a.E], tokens);
  __syncthreads();
  const bool single = gridDim.x == 1;
  float* pp = single ? a.psum : (float*)a.workspace + (int64_t)blockIdx.x * a.E;
  int* pn = single ? a.counts : (int*)((float*)a.workspace + (int64_t)gridDim.x * a.E) + (int64_t)blockIdx.x * (a.E + 1);
  for (int e = threadIdx.x; e <= a.E; e += RW * 32) {
    if (e < a.E) {
      float v = cs.p[0][e];
#pragma unroll
      for (int i = 1; i < RW; ++i) v += cs.p[i][e];
      pp[e] = v;
      cs.p[0][e] = v;
    }
    pn[e] = cs.n[e];
  }
  if (single) {
    __syncthreads();
    final_sums(a, a.E, cs.p[0], cs.n, red);
  }
}

// counts, probability sums and the loss from the CTAs' partials, in order
__global__ void __launch_bounds__(1024) k_router_sums(RouterArgs a, int parts) {
  __shared__ float sp[1024], fp[ROUTER_MAX_E], red[32];
  __shared__ int sn[1024], fn[ROUTER_MAX_E + 1];
  const int ew = (a.E + 31) / 32 * 32, groups = 1024 / ew;
  const int e = threadIdx.x % ew, g = threadIdx.x / ew;
  const float* pp = (const float*)a.workspace;
  const int* pn = (const int*)(pp + (int64_t)parts * a.E);
  float v = 0.0f;
  int n = 0;
  if (e < a.E && g < groups) {
#pragma unroll 4
    for (int i = g; i < parts; i += groups) {
      v += pp[(int64_t)i * a.E + e];
      n += pn[(int64_t)i * (a.E + 1) + e];
    }
  }
  sp[threadIdx.x] = v;
  sn[threadIdx.x] = n;
  int tok = 0;
  if (threadIdx.x < 32) {
    for (int i = threadIdx.x; i < parts; i += 32) tok += pn[(int64_t)i * (a.E + 1) + a.E];
    tok = __reduce_add_sync(0xffffffffu, tok);
  }
  __syncthreads();
  if (g == 0 && e < a.E) {
    for (int i = 1; i < groups; ++i) {
      v += sp[i * ew + e];
      n += sn[i * ew + e];
    }
    fp[e] = a.psum[e] = v;
    fn[e] = a.counts[e] = n;
  }
  if (threadIdx.x == 0) fn[a.E] = a.counts[a.E] = tok;
  __syncthreads();
  final_sums(a, a.E, fp, fn, red);
}

template <int V, bool SIG>
__global__ void __launch_bounds__(RW * 32) k_router_bwd(RouterArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float c[V];
  float coef = 0.0f;
  if (a.dloss) {
    const float N = fmaxf((float)a.counts_in[a.E], 1.0f);
    coef = a.dloss[0] * __fdiv_rn((float)a.E, (float)a.k) / (N * N);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = a.dloss && i * 32 + lane < a.E ? coef * (float)a.counts_in[i * 32 + lane] : 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * RW + warp; t < a.T; t += (int64_t)gridDim.x * RW) {
    const bool on = !a.mask || a.mask[t] != 0;
    float x[V], s[V], p[V], d[V];
    load_row<V>(a, t, lane, on, x);
    const RowStat st = row_scores<V, SIG>(x, s, p);
    float pc = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) pc = fmaf(p[i], c[i], pc);
    pc = warp_sum(pc);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = p[i] * (c[i] - pc);
    // lane j: slot j's score, from the logit itself
    int e = -1;
    float u = 0.0f;
    if (a.dw) {
      float sj = 0.0f, dwj = 0.0f;
      if (lane < a.k && on) {
        e = a.idx_in[t * a.k + lane];
        if (e < 0 || e >= a.E) e = -1;
        dwj = a.dw[t * a.k + lane];
        if (e >= 0) {
          const float xj = a.bf16 ? __uint_as_float((uint32_t)((const uint16_t*)a.logits)[t * a.ld + e] << 16)
                                  : ((const float*)a.logits)[t * a.ld + e];
          sj = SIG ? sigmoid_rn(xj) : __fdiv_rn(expf(xj - st.m), st.z);
        }
      }
      if (a.renorm) {
        const float z = warp_sum(sj);
        sj = __fdiv_rn(sj, z == 0.0f ? 1.0f : z);
        u = sj * (dwj - warp_sum(dwj * sj));
      } else {
        u = sj * dwj;
      }
      u *= a.route_scale;
      if constexpr (!SIG) {
        const float us = warp_sum(u);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = fmaf(-p[i], us, d[i]);
      }
      for (int j = 0; j < a.k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j);
        const float uj = __shfl_sync(0xffffffffu, u, j);
        if (ej >= 0 && lane == (ej & 31)) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i == (ej >> 5)) d[i] += uj;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ei = i * 32 + lane;
      if (ei >= a.E) continue;
      const float o = SIG ? d[i] * (1.0f - s[i]) : d[i];
      if (a.bf16) {
        ((__nv_bfloat16*)a.dlogits)[t * a.E + ei] = __float2bfloat16_rn(o);
      } else {
        ((float*)a.dlogits)[t * a.E + ei] = o;
      }
    }
  }
}

// dw[t, j] = sum over n of dout[t, n] * y[row_of[t, j], n]: WPT warps share a
// token (each every WPT-th group of 32 chunks), UK rows of y at a time.
template <int WPT, int UK>
__global__ void __launch_bounds__(256) k_route_weight_grad(const uint16_t* __restrict__ dout,
                                                           const uint16_t* __restrict__ y,
                                                           const int32_t* __restrict__ row_of, int64_t T, int64_t N,
                                                           int k, float* __restrict__ dw) {
  __shared__ float red[8][UK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPT;
  const int64_t t = (int64_t)blockIdx.x * (8 / WPT) + warp / WPT;
  const int64_t nv = N / 8;
  for (int j0 = 0; j0 < k; j0 += UK) {
    const uint16_t* src[UK];
    float acc[UK];
#pragma unroll
    for (int j = 0; j < UK; ++j) {
      const int r = t < T && j0 + j < k ? row_of[t * k + j0 + j] : -1;
      src[j] = r < 0 ? nullptr : y + (int64_t)r * N;
      acc[j] = 0.0f;
    }
    if (t < T) {
      for (int64_t v = part * 32 + lane; v < nv; v += 32 * WPT) {
        const uint4 d = ld_nc16(dout + t * N + v * 8);
        uint4 q[UK];
#pragma unroll
        for (int j = 0; j < UK; ++j) q[j] = src[j] ? ld_nc16(src[j] + v * 8) : make_uint4(0, 0, 0, 0);
        const uint32_t dd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < UK; ++j) {
          const uint32_t qq[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
          if (!src[j]) continue;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            acc[j] = fmaf(bf16_lo(dd[h]), bf16_lo(qq[h]), acc[j]);
            acc[j] = fmaf(bf16_hi(dd[h]), bf16_hi(qq[h]), acc[j]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < UK; ++j) {
      acc[j] = warp_sum(acc[j]);
      if (WPT > 1 && lane == 0) red[warp][j] = acc[j];
    }
    if (WPT > 1) __syncthreads();
    if (t < T && part == 0 && lane == 0) {
#pragma unroll
      for (int j = 0; j < UK; ++j) {
        float v = acc[j];
        if (WPT > 1)
          for (int i = 1; i < WPT; ++i) v += red[warp + i][j];
        if (j0 + j < k) dw[t * k + j0 + j] = v;
      }
    }
    if (WPT > 1) __syncthreads();
  }
}

template <int V, bool SIG>
cudaError_t run_fwd(const RouterArgs& a, int num_sms, cudaStream_t st) {
  static std::atomic<int> occ{0};
  int64_t blocks = a.T <= SINGLE_CTA_T ? 1 : (a.T + RW - 1) / RW;
  const int64_t fit = (int64_t)num_sms * blocks_per_sm(occ, k_router_fwd<V, SIG>, RW * 32, 0, 1);
  if (blocks > fit) blocks = fit;
  if (blocks > ROUTER_MAX_PARTS) blocks = ROUTER_MAX_PARTS;
  k_router_fwd<V, SIG><<<(unsigned)blocks, RW * 32, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.counts || blocks == 1) return e;
  k_router_sums<<<1, 1024, 0, st>>>(a, (int)blocks);
  return cudaGetLastError();
}
template <int V, bool SIG>
cudaError_t run_bwd(const RouterArgs& a, int num_sms, cudaStream_t st) {
  static std::atomic<int> occ{0};
  int64_t blocks = (a.T + RW - 1) / RW;
  const int64_t fit = (int64_t)num_sms * blocks_per_sm(occ, k_router_bwd<V, SIG>, RW * 32, 0, 1);
  if (blocks > fit) blocks = fit;
  k_router_bwd<V, SIG><<<(unsigned)blocks, RW * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

#define FP8MOE_ROUTER(V, FN)                                                         \
  if (a.E <= 32 * V)                                                                 \
    return a.score == FP8MOE_SCORE_SIGMOID ? FN<V, true>(a, num_sms, st) : FN<V, false>(a, num_sms, st);

// T == 0: one CTA writes the empty sums
cudaError_t launch_router_fwd(const RouterArgs& a, int num_sms, cudaStream_t st) {
  FP8MOE_ROUTER(1, run_fwd)
  FP8MOE_ROUTER(2, run_fwd)
  FP8MOE_ROUTER(4, run_fwd)
  FP8MOE_ROUTER(8, run_fwd)
  FP8MOE_ROUTER(16, run_fwd)
  FP8MOE_ROUTER(32, run_fwd)
  return cudaErrorInvalidValue;
}
cudaError_t launch_router_bwd(const RouterArgs& a, int num_sms, cudaStream_t st) {
  FP8MOE_ROUTER(1, run_bwd)
  FP8MOE_ROUTER(2, run_bwd)
  FP8MOE_ROUTER(4, run_bwd)
  FP8MOE_ROUTER(8, run_bwd)
  FP8MOE_ROUTER(16, run_bwd)
  FP8MOE_ROUTER(32, run_bwd)
  return cudaErrorInvalidValue;
}
#undef FP8MOE_ROUTER

cudaError_t launch_route_weight_grad(const void* dout, const void* y, const int32_t* row_of, int64_t T, int64_t N,
                                     int64_t k, float* dw, int num_sms, cudaStream_t st) {
  const uint16_t *d = (const uint16_t*)dout, *yp = (const uint16_t*)y;
  // a warp per token where that fills the GPU, eight where tokens are few
  const bool many = T >= (int64_t)num_sms * 16;
#define FP8MOE_WG(UK)                                                                                            \
  many ? k_route_weight_grad<1, UK><<<(unsigned)((T + 7) / 8), 256, 0, st>>>(d, yp, row_of, T, N, (int)k, dw)    \
       : k_route_weight_grad<8, UK><<<(unsigned)T, 256, 0, st>>>(d, yp, row_of, T, N, (int)k, dw)
  if (k <= 1) {
    FP8MOE_WG(1);
  } else if (k <= 2) {
    FP8MOE_WG(2);
  } else if (k <= 4) {
    FP8MOE_WG(4);
  } else {
    FP8MOE_WG(8);
  }
#undef FP8MOE_WG
  return cudaGetLastError();
}

}  // namespace fp8moe
