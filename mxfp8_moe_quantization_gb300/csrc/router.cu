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
// A warp takes a token, or several where experts are few and tokens many; a lane
// has pieces of four neighbouring experts.  The logits are read once.
// A row's sums have an order of their own, so that a token's choice and weights
// do not depend on the batch.  Sums over tokens have a fixed order (registers,
// then warps, then CTAs), so results do not change from run to run.  The CTAs'
// partial sums are joined by a second kernel of one cluster, launched ahead of
// the first one's end.
//
// Bound by latency, then by instruction issue (a token of 256 fp32 experts, top
// 8: about 1200 warp instructions, half of them the rounds of the choice; bf16
// logits without a bias need one maximum a round instead of two reductions:
// 65536 x 128, top 8, 31.4 us against 39.4).  In a graph: 4096 x 256, top 8,
// 10.2 us forward with the sums and 6.0 without, 4.7 backward; 8192 x 64, top 6,
// 7.2 and 3.3; 3 tokens 3.8.  The first form, which carried scores through the
// rounds and joined 512 partial sums in one CTA, took 29.9 us on the first.
#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"
#include "moe_ops.h"

namespace fp8moe {
namespace {

// Most warps of a CTA whose lanes hold V experts each (its registers).
template <int V>
constexpr int most_warps() { return V <= 8 ? 32 : V == 16 ? 16 : 8; }
constexpr int SINGLE_CTA_T = 16;   // up to so many tokens one CTA does everything

// order-preserving key: larger float, larger key; NaN sorts with -inf; every
// key is above 0, the mark of what is taken or absent
FP8MOE_DEV uint32_t order_key(float f) {
  const int u = __float_as_int(fmaxf(f + 0.0f, -__builtin_huge_valf()));   // -0 and 0 are equal
  return (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u);
}

// sums and maxima over the G lanes of a token (every lane gets the result)
template <int G = 32>
FP8MOE_DEV float lane_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int G>
FP8MOE_DEV float lane_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int G>
FP8MOE_DEV uint32_t lane_umax(uint32_t v) {
  if constexpr (G == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int G>
FP8MOE_DEV uint32_t lane_umin(uint32_t v) {
  if constexpr (G == 32) {
    return __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}

constexpr float NEG_INF = -__builtin_huge_valf();

FP8MOE_DEV float logit_at(const RouterArgs& a, int64_t t, int e) {
  return a.bf16 ? __uint_as_float((uint32_t)((const uint16_t*)a.logits)[t * a.ld + e] << 16)
                : ((const float*)a.logits)[t * a.ld + e];
}

// A lane's V experts are pieces of up to four neighbours, the lanes' pieces
// side by side: wide accesses to memory, and to shared memory without a bank
// met twice.
template <int V>
constexpr int piece() { return V < 4 ? V : 4; }
template <int V, int G>
FP8MOE_DEV int expert(int l, int i) {
  constexpr int P = piece<V>();
  return (i / P * G + l) * P + i % P;
}

// the logits of token t at this lane's experts; -inf past the last one and
// everywhere in a row that is no token
template <int V, int G>
FP8MOE_DEV void load_row(const RouterArgs& a, int64_t t, int l, bool on, float (&x)[V]) {
  constexpr int P = piece<V>();
  if (P > 1 && a.wide) {   // E is a multiple of a piece
#pragma unroll
    for (int p = 0; p < V; p += P) {
      const int e = expert<V, G>(l, p);
      const bool here = on && e < a.E;
      if (a.bf16) {
        const uint16_t* at = (const uint16_t*)a.logits + t * a.ld + e;
        constexpr uint32_t NONE = 0xFF80FF80u;   // -inf, -inf
        uint2 v = make_uint2(NONE, NONE);
        if (here) {
          if constexpr (P == 4) v = *reinterpret_cast<const uint2*>(at);
          if constexpr (P == 2) v.x = *reinterpret_cast<const uint32_t*>(at);
        }
        x[p] = bf16_lo(v.x);
        if constexpr (P >= 2) x[p + 1] = bf16_hi(v.x);
        if constexpr (P == 4) x[p + 2] = bf16_lo(v.y), x[p + 3] = bf16_hi(v.y);
      } else {
        const float* at = (const float*)a.logits + t * a.ld + e;
        float4 v = make_float4(NEG_INF, NEG_INF, NEG_INF, NEG_INF);
        if (here) {
          if constexpr (P == 4) v = *reinterpret_cast<const float4*>(at);
          if constexpr (P == 2) v.x = at[0], v.y = at[1];
        }
        x[p] = v.x;
        if constexpr (P >= 2) x[p + 1] = v.y;
        if constexpr (P == 4) x[p + 2] = v.z, x[p + 3] = v.w;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert<V, G>(l, i);
    x[i] = on && e < a.E ? logit_at(a, t, e) : NEG_INF;
  }
}

// 1 / (1 + e^-x), each step rounded to nearest (the choice with a bias hangs on it)
FP8MOE_DEV float sigmoid_rn(float x) { return __frcp_rn(1.0f + expf(-x)); }

// For the gradient both the sigmoid s and 1 - s, each to a few ulp: the smaller
// of the two is t / (1 + t) with t = e^-|x|, and the other one 1 minus that.  The
// smaller one is kept, with a sign where it is 1 - s.  (1 - s from a rounded s
// is off by 5e-4 of itself at a logit of 10, and 0 from 17 on.)  The reciprocal
// of 1 + t, which lies in [1, 2], takes one step of Newton's iteration.
FP8MOE_DEV float sigmoid_side(float x) {
  const float t = expf(-fabsf(x)), d = 1.0f + t;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  r = fmaf(fmaf(-d, r, 1.0f), r, r);
  return __int_as_float(__float_as_int(t * r) | (~__float_as_int(x) & 0x80000000));
}
FP8MOE_DEV float side_score(float q) { return __float_as_int(q) < 0 ? 1.0f + q : q; }   // s
FP8MOE_DEV float side_rest(float q) { return __float_as_int(q) < 0 ? -q : 1.0f - q; }    // 1 - s

// A row's sum, in an order that hangs on the experts' numbers alone, whatever
// lanes hold them (a token gets the same bits in any batch): bits 0 and 1 of the
// number first, then from the highest bit down.  Experts past the last are 0.
template <int V, int G>
FP8MOE_DEV float row_sum(const float (&s)[V]) {
  constexpr int P = piece<V>(), N = V / P;
  float a[N];
#pragma unroll
  for (int p = 0; p < N; ++p) {
    if constexpr (P == 4) a[p] = (s[4 * p] + s[4 * p + 1]) + (s[4 * p + 2] + s[4 * p + 3]);
    if constexpr (P == 2) a[p] = s[2 * p] + s[2 * p + 1];
    if constexpr (P == 1) a[p] = s[p];
  }
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1)
#pragma unroll
    for (int p = 0; p < h; ++p) a[p] += a[p + h];
  float v = a[0];
  // the lanes that differ in bits 0 and 1 of the number, where a piece is short
#pragma unroll
  for (int o = 1; o < 4 / P; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
#pragma unroll
  for (int o = G / 2; o >= 4 / P; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// likewise over a token's slots, l, l + G, .., from the highest bit down
template <int G, int S>
FP8MOE_DEV float slot_sum(const float (&w)[S]) {
  float a[S];
#pragma unroll
  for (int q = 0; q < S; ++q) a[q] = w[q];
#pragma unroll
  for (int h = S / 2; h > 0; h >>= 1)
#pragma unroll
    for (int q = 0; q < h; ++q) a[q] += a[q + h];
  return lane_sum<G>(a[0]);
}

// What turns a logit of the row into its score: softmax s = e^(x - m) / z;
// z is also the sum of the sigmoids.
struct RowStat {
  float m, z, rz;   // rz = 1 / z, 0 for a row of nothing but -inf (or sigmoids whose sum has no reciprocal)
};
// e / z, rounded once: the quotient by the rounded reciprocal and one step of
// Markstein's correction (e <= z; 0 where the reciprocal stands at 0)
FP8MOE_DEV float over_z(float e, const RowStat& st) {
  const float q = e * st.rz;
  return fmaf(fmaf(-st.z, q, e), st.rz, q);
}
template <bool SIG, bool GRAD = false>
FP8MOE_DEV float score_of(float x, const RowStat& st) {
  return SIG ? (GRAD ? side_score(sigmoid_side(x)) : sigmoid_rn(x)) : over_z(expf(x - st.m), st);
}
// s: sigmoids (GRAD: their sides), or the softmax's e^(x - m) before the division
// by z
template <int V, int G, bool SIG, bool GRAD = false>
FP8MOE_DEV RowStat row_scores(const float (&x)[V], float (&s)[V]) {
  RowStat st{0.0f, 0.0f, 0.0f};
  if constexpr (SIG) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = GRAD ? sigmoid_side(x[i]) : sigmoid_rn(x[i]);
  } else {
    float m = NEG_INF;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = lane_max<G>(m);
    st.m = m == NEG_INF ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = expf(x[i] - st.m);
  }
  if constexpr (SIG && GRAD) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = side_score(s[i]);
    st.z = row_sum<V, G>(f);
  } else {
    st.z = row_sum<V, G>(s);
  }
  st.rz = st.z < 2.9387359e-39f ? 0.0f : __frcp_rn(st.z);   // (below that 1 / z is beyond fp32, as for z = 0)
  return st;
}

// loss from counts and probability sums; every thread of the CTA calls it.
// part: this CTA's share of sum n_e P_e (thread 0 has the result)
FP8MOE_DEV float cta_sum(float v, float* red) {
  v = lane_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  if (threadIdx.x < 32) v = lane_sum(threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0.0f);
  return v;
}
FP8MOE_DEV float loss_of(float np, int tokens, int E, int k) {
  const float N = fmaxf((float)tokens, 1.0f);
  return np * __fdiv_rn((float)E, (float)k) / (N * N);
}

// Slots of a token's choice that a lane looks after: its k <= G * slots<G>().
template <int G>
constexpr int slots() { return G >= 8 ? 1 : 8 / G; }

// A lane's two best experts that rank after (lk, li), b1 = 0 or b2 = 0 where
// there is none; PACK: keys differ, and carry their ids.
template <int V, int G, bool PACK, bool AFTER>
FP8MOE_DEV void best_two(const uint32_t (&key)[V], int l, uint32_t lk, int li, uint32_t& b1, uint32_t& b2, int& i1, int& i2) {
  b1 = b2 = 0u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert<V, G>(l, i);
    uint32_t x = key[i];
    if constexpr (PACK) {
      if (AFTER && x >= lk) x = 0u;
      b2 = max(b2, min(b1, x));
      b1 = max(b1, x);
    } else {
      if (AFTER && (x > lk || (x == lk && e <= li))) x = 0u;
      const bool c1 = x > b1, c2 = x > b2;   // ids rise with i: the first of equal keys stays ahead
      b2 = c1 ? b1 : c2 ? x : b2;
      i2 = c1 ? i1 : c2 ? e : i2;
      b1 = c1 ? x : b1;
      i1 = c1 ? e : i1;
    }
  }
}

// k rounds: the token's largest key, then the lowest id that has it (PACK: the
// key's lower half says which).  Lane l ends with slots l, l + G, ..
//
// two: a lane's two best experts are kept at hand, so that a round costs the
// same for any V; a lane that loses both looks through its experts again.  Fewer
// instructions where lanes, their experts and rounds are many (65536 x 256, top
// 8: 61.0 us against 67.6, 65536 x 384, top 6: 112 against 129; over 16 lanes of
// eight 46.3 against 41.6, with four experts a lane 8.8 against 8.4 on 4096 x 128,
// with two rounds 38.4 against 37.2), but a longer way for one token (4096 x
// 256: 10.2 against 10.0).
template <int V, int G, bool PACK>
FP8MOE_DEV void choose(uint32_t (&key)[V], int (&my_e)[slots<G>()], int k, int l, bool two) {
  if (V >= 8 && G == 32 && two) {
    my_e[0] = 0;
    uint32_t b1, b2, lk = 0u;
    int i1 = 0, i2 = 0, li = 0;
    best_two<V, G, PACK, false>(key, l, 0u, 0, b1, b2, i1, i2);
    for (int j = 0; j < k; ++j) {
      const uint32_t top = lane_umax<G>(b1);
      bool mine = b1 == top;
      uint32_t e = 0xFFFFu - (top & 0xFFFFu);
      if constexpr (!PACK) {
        e = lane_umin<G>(mine ? (uint32_t)i1 : 0xffffffffu);
        mine = mine && e == (uint32_t)i1;
      }
      if (l == j) my_e[0] = (int)e;
      if (mine) {
        lk = b1, li = i1;
        b1 = b2, i1 = i2;
        b2 = 0u;
      }
      if (__any_sync(0xffffffffu, mine && b1 == 0u)) {
        uint32_t n1, n2;
        int m1 = 0, m2 = 0;
        best_two<V, G, PACK, true>(key, l, lk, li, n1, n2, m1, m2);
        if (mine && b1 == 0u) b1 = n1, b2 = n2, i1 = m1, i2 = m2;
      }
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < slots<G>(); ++q) {
    my_e[q] = 0;
    for (int j = q * G; j < k && j < (q + 1) * G; ++j) {
      uint32_t bk = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) bk = max(bk, key[i]);
      const uint32_t top = lane_umax<G>(bk);
      if constexpr (PACK) {
        if (l == j % G) my_e[q] = (int)(0xFFFFu - (top & 0xFFFFu));
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] == top) key[i] = 0u;
      } else {
        uint32_t be = 0xffffffffu;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (key[i] == top) be = (uint32_t)expert<V, G>(l, i);
        const uint32_t e = lane_umin<G>(be);
        if (l == j % G) my_e[q] = (int)e;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e == (uint32_t)expert<V, G>(l, i)) key[i] = 0u;
      }
    }
  }
}

// G lanes take a token, a lane V experts; a warp 32 / G tokens at a time.
template <int V, int G, bool SIG>
__global__ void __launch_bounds__(most_warps<V>() * 32) k_router_fwd(RouterArgs a) {
  constexpr int S = slots<G>();
  constexpr int TPW = 32 / G;
  extern __shared__ __align__(16) float rsm[];
  __shared__ float red[32];
  const int RW = blockDim.x >> 5;
  float* cp = rsm;                      // [RW][G V]
  int* cn = (int*)(rsm + RW * G * V);   // [E + 1]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % G;
  const bool sums = a.counts != nullptr;
  // the joining kernel may take its place; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;");
  float acc[V] = {};
  int tokens = 0;
  if (sums) {
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) cn[e] = 0;
    __syncthreads();
  }
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = a.bias && expert<V, G>(l, i) < a.E ? a.bias[expert<V, G>(l, i)] : 0.0f;
  for (int64_t tw = ((int64_t)blockIdx.x * RW + warp) * TPW; tw < a.T; tw += (int64_t)gridDim.x * RW * TPW) {
    const int64_t t = tw + lane / G;   // past T: no token, nothing stored
    const bool row = t < a.T, on = row && (!a.mask || a.mask[t] != 0);
    float x[V], s[V];
    load_row<V, G>(a, t, l, on, x);
    const RowStat st = row_scores<V, G, SIG>(x, s);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float p = over_z(s[i], st);
      acc[i] += p;
      // dead experts stay below every other whatever their bias
      const float f = !a.bias ? x[i] : x[i] == NEG_INF ? NEG_INF : (SIG ? s[i] : p) + bias[i];
      key[i] = expert<V, G>(l, i) < a.E ? order_key(f) : 0u;
    }
    tokens += on;
    int my_e[S];
    if (a.bf16 && !a.bias) {
      // a bf16 logit leaves the key's lower half to the expert: the lowest id
      // has the largest key, and one maximum a round is enough
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] != 0u) key[i] = (key[i] & 0xFFFF0000u) | (uint32_t)(0xFFFF - expert<V, G>(l, i));
      choose<V, G, true>(key, my_e, a.k, l, a.two);
    } else {
      choose<V, G, false>(key, my_e, a.k, l, a.two);
    }
    // lane l: the weights of slots l, l + G, .. from their logits
    float w[S], z = 1.0f;
#pragma unroll
    for (int q = 0; q < S; ++q) {
      w[q] = 0.0f;
      if (q * G + l < a.k && row) {
        const float xe = on ? logit_at(a, t, my_e[q]) : NEG_INF;
        w[q] = score_of<SIG>(xe, st);
        if (sums && xe != NEG_INF) atomicAdd(&cn[my_e[q]], 1);
      }
    }
    if (a.renorm) {
      z = slot_sum<G>(w);
      z = z == 0.0f ? 1.0f : z;
    }
#pragma unroll
    for (int q = 0; q < S; ++q) {
      if (q * G + l < a.k && row) {
        a.idx[t * a.k + q * G + l] = my_e[q];
        a.w[t * a.k + q * G + l] = (a.renorm ? __fdiv_rn(w[q], z) : w[q]) * a.route_scale;
      }
    }
  }
  if (!sums) return;
  // the lanes that share experts, in lane order, then the warps
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int o = G; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  if (lane < G) {
#pragma unroll
    for (int i = 0; i < V; ++i) cp[warp * G * V + expert<V, G>(l, i)] = acc[i];
  }
  if (l == 0) atomicAdd(&cn[a.E], tokens);
  __syncthreads();
  const bool single = gridDim.x == 1;
  float* pp = single ? a.psum : (float*)a.workspace + (int64_t)blockIdx.x * a.E;
  int* pn = single ? a.counts : (int*)((float*)a.workspace + (int64_t)gridDim.x * a.E) + (int64_t)blockIdx.x * (a.E + 1);
  float np = 0.0f;
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
    const int n = cn[e];
    pn[e] = n;
    if (e < a.E) {
      const float* c = cp + e;
      float v = c[0];
#pragma unroll 4
      for (int i = 1; i < RW; ++i) v += c[i * G * V];
      pp[e] = v;
      np = fmaf((float)n, v, np);
    }
  }
  if (single) {
    np = cta_sum(np, red);
    if (threadIdx.x == 0) a.loss[0] = loss_of(np, cn[a.E], a.E, a.k);
  }
}

// Counts, probability sums and the loss from the CTAs' partials, in order: one
// cluster of JOIN CTAs, CTA c with every JOIN-th block of 32 experts (a warp a
// slice of the partials, a lane an expert).
constexpr int JOIN = 8, JOIN_WARPS = 16, JOIN_U = 10;
__global__ void __cluster_dims__(JOIN, 1, 1) __launch_bounds__(JOIN_WARPS * 32) k_router_join(RouterArgs a, int parts) {
  __shared__ float sp[JOIN_WARPS][32], share[JOIN];
  __shared__ int sn[JOIN_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = blockIdx.x;
  const float* pp = (const float*)a.workspace;
  const int* pn = (const int*)(pp + (int64_t)parts * a.E);
  // a remote store needs its target CTA to have started: waited for below
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the token counts, in flight beside the sums
  int tok = 0;
  if (rank == 0 && warp == 0)
    for (int i = lane; i < parts; i += 32) tok += __ldcg(pn + (int64_t)i * (a.E + 1) + a.E);
  float np = 0.0f, v = 0.0f;
  int n = 0, last = -1;   // the block whose results are stored at the end
  for (int e0 = rank * 32; e0 < a.E; e0 += JOIN * 32) {
    const int e = e0 + lane;
    if (last >= 0) {
      if (warp == 0) a.psum[last + lane] = v, a.counts[last + lane] = n;
      __syncthreads();   // sp, sn are read
    }
    last = e0;
    v = 0.0f;
    n = 0;
    if (e < a.E) {
      // every load of a round in flight at once (one round up to 160 parts)
      for (int i0 = warp; i0 < parts; i0 += JOIN_WARPS * JOIN_U) {
        float vv[JOIN_U];
        int nn[JOIN_U];
#pragma unroll
        for (int j = 0; j < JOIN_U; ++j) {
          const int i = i0 + j * JOIN_WARPS;
          vv[j] = i < parts ? __ldcg(pp + (int64_t)i * a.E + e) : 0.0f;
          nn[j] = i < parts ? __ldcg(pn + (int64_t)i * (a.E + 1) + e) : 0;
        }
#pragma unroll
        for (int j = 0; j < JOIN_U; ++j) {
          v += vv[j];
          n += nn[j];
        }
      }
    }
    sp[warp][lane] = v;
    sn[warp][lane] = n;
    __syncthreads();
    if (warp == 0 && e < a.E) {
#pragma unroll
      for (int i = 1; i < JOIN_WARPS; ++i) {
        v += sp[i][lane];
        n += sn[i][lane];
      }
      np = fmaf((float)n, v, np);
    }
  }
  // every CTA's share of sum n_e P_e into rank 0's shared memory
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == 0) {
    np = lane_sum(np);
    if (lane == 0) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(&share[rank])));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(np) : "memory");
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // (after the arrival, whose release would wait for these stores)
  if (warp == 0 && last >= 0 && last + lane < a.E) {
    a.psum[last + lane] = v;
    a.counts[last + lane] = n;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && warp == 0) {
    tok = __reduce_add_sync(0xffffffffu, tok);
    np = lane_sum(lane < JOIN ? share[lane] : 0.0f);
    if (lane == 0) {
      a.counts[a.E] = tok;
      a.loss[0] = loss_of(np, tok, a.E, a.k);
    }
  }
}

template <int V, int G, bool SIG>
__global__ void __launch_bounds__(most_warps<V>() * 32) k_router_bwd(RouterArgs a) {
  constexpr int TPW = 32 / G, S = slots<G>(), P = piece<V>();
  extern __shared__ __align__(16) float rsm[];
  const int RW = blockDim.x >> 5;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % G;
  float* ubuf = rsm + (warp * TPW + lane / G) * G * V;   // the chosen experts' u
  float c[V];
  float coef = 0.0f;
  if (a.dloss) coef = a.dloss[0] * loss_of(1.0f, a.counts_in[a.E], a.E, a.k);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert<V, G>(l, i);
    c[i] = a.dloss && e < a.E ? coef * (float)a.counts_in[e] : 0.0f;
    ubuf[e] = 0.0f;
  }
  __syncwarp();
  for (int64_t tw = ((int64_t)blockIdx.x * RW + warp) * TPW; tw < a.T; tw += (int64_t)gridDim.x * RW * TPW) {
    const int64_t t = tw + lane / G;   // past T: no token, nothing stored
    const bool row = t < a.T, on = row && (!a.mask || a.mask[t] != 0);
    // lane l: the token's slots l, l + G, ..
    int e[S];
    float dwj[S], xj[S];
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int j = q * G + l;
      e[q] = -1;
      dwj[q] = xj[q] = 0.0f;
      if (a.dw && j < a.k && on) {
        e[q] = a.idx_in[t * a.k + j];
        if (e[q] < 0 || e[q] >= a.E) e[q] = -1;
        dwj[q] = a.dw[t * a.k + j];
      }
    }
    float x[V], s[V];
    load_row<V, G>(a, t, l, on, x);
#pragma unroll
    for (int q = 0; q < S; ++q)
      if (e[q] >= 0) xj[q] = logit_at(a, t, e[q]);
    const RowStat st = row_scores<V, G, SIG, true>(x, s);
    float pc = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) pc = fmaf(over_z(SIG ? side_score(s[i]) : s[i], st), c[i], pc);
    pc = lane_sum<G>(pc);
    float us = 0.0f;
    if (a.dw) {
      // the slots' scores, from the logits themselves
      float u[S], sc[S];
#pragma unroll
      for (int q = 0; q < S; ++q) {
        sc[q] = e[q] >= 0 ? score_of<SIG, true>(xj[q], st) : 0.0f;
        u[q] = sc[q] * (a.renorm ? 1.0f : dwj[q]);
      }
      if (a.renorm) {
        const float z = slot_sum<G>(sc);
        float d = 0.0f;
#pragma unroll
        for (int q = 0; q < S; ++q) {
          u[q] = __fdiv_rn(u[q], z == 0.0f ? 1.0f : z);
          d += dwj[q] * u[q];
        }
        d = lane_sum<G>(d);
#pragma unroll
        for (int q = 0; q < S; ++q) u[q] *= dwj[q] - d;
      }
#pragma unroll
      for (int q = 0; q < S; ++q) us += u[q] *= a.route_scale;
      if constexpr (!SIG) us = lane_sum<G>(us);
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (e[q] >= 0) atomicAdd(&ubuf[e[q]], u[q]);
      __syncwarp();
    }
    if (row) {
#pragma unroll
      for (int p = 0; p < V; p += P) {
        const int e0 = expert<V, G>(l, p);
        float o[P];
        if constexpr (P == 4) {
          const float4 b = *reinterpret_cast<const float4*>(ubuf + e0);
          o[0] = b.x, o[1] = b.y, o[2] = b.z, o[3] = b.w;
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) o[i] = ubuf[e0 + i];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          o[i] += over_z(SIG ? side_score(s[p + i]) : s[p + i], st) * (c[p + i] - pc - (SIG ? 0.0f : us));
          if (SIG) o[i] *= side_rest(s[p + i]);
        }
        if (P > 1 && a.wide) {
          if (e0 >= a.E) break;
          if (a.bf16) {
            uint16_t* at = (uint16_t*)a.dlogits + t * a.E + e0;
            if constexpr (P == 4) *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(pk(o[0], o[1])), pack_bf16x2(pk(o[2], o[3])));
            if constexpr (P == 2) *reinterpret_cast<uint32_t*>(at) = pack_bf16x2(pk(o[0], o[1]));
          } else {
            float* at = (float*)a.dlogits + t * a.E + e0;
            if constexpr (P == 4) *reinterpret_cast<float4*>(at) = make_float4(o[0], o[1], o[2], o[3]);
            if constexpr (P == 2) at[0] = o[0], at[1] = o[1];
          }
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (e0 + i >= a.E) break;
            if (a.bf16) {
              ((__nv_bfloat16*)a.dlogits)[t * a.E + e0 + i] = __float2bfloat16_rn(o[i]);
            } else {
              ((float*)a.dlogits)[t * a.E + e0 + i] = o[i];
            }
          }
        }
      }
    }
    if (a.dw) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (e[q] >= 0) ubuf[e[q]] = 0.0f;
      __syncwarp();
    }
  }
}

// dw[t, j] = sum over n of dout[t, n] * y[row_of[t, j], n]: L lanes take a token
// (several tokens a warp, or several warps a token), a lane every L-th chunk of
// 16 bytes, of UK rows of y at a time.  The row numbers rather than pointers are
// kept (-1: missing, or no row of y), so that four CTAs fit an SM (16384 tokens x 6 rows of 2048: 70.5 us against
// 80.0 with three; what spills is outside the loop's loads).
template <int L, int UK>
__global__ void __launch_bounds__(256, 4) k_route_weight_grad(const uint16_t* __restrict__ dout,
                                                              const uint16_t* __restrict__ y,
                                                              const int32_t* __restrict__ row_of, uint32_t rows,
                                                              int64_t T, int64_t N, int k, float* __restrict__ dw) {
  constexpr int WPT = L / 32;   // warps per token (0: less than one)
  __shared__ float red[8][UK];
  const int warp = threadIdx.x >> 5, l = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int64_t nv = N / 8;
  for (int j0 = 0; j0 < k; j0 += UK) {
    int row[UK];
    float acc[UK];
#pragma unroll
    for (int j = 0; j < UK; ++j) {
      row[j] = t < T && j0 + j < k ? row_of[t * k + j0 + j] : -1;
      if ((uint32_t)row[j] >= rows) row[j] = -1;
      acc[j] = 0.0f;
    }
    if (t < T) {
      for (int64_t v = l; v < nv; v += L) {
        const uint4 d = ld_nc16(dout + t * N + v * 8);
        uint4 q[UK];
#pragma unroll
        for (int j = 0; j < UK; ++j) q[j] = row[j] < 0 ? make_uint4(0, 0, 0, 0) : ld_nc16(y + row[j] * N + v * 8);
        const uint32_t dd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < UK; ++j) {
          const uint32_t qq[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
          if (row[j] < 0) continue;
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
      acc[j] = lane_sum<(L < 32 ? L : 32)>(acc[j]);
      if (WPT > 1 && (threadIdx.x & 31) == 0) red[warp][j] = acc[j];
    }
    if (WPT > 1) __syncthreads();
    if (t < T && l == 0) {
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

// The same with y in MXFP8 (row-major scales): a lane's chunk is 16 codes, half a
// block, whose products are summed before the block's power of two.  For a missing
// row the loop reads row 0 and the result is dropped: choosing in the loop cost a
// fifth of its instructions (60000 x 128 x 8: 42 us, 26 without).  Bound by HBM, at
// 1.03 bytes a value of y: 4096 x 7168 x 8 53 us = 5.7 TB/s (85% of a copy's rate; its
// 2048 CTAs are four and a half rounds, and the warps wait for memory), 8189 x 2048 x 6
// 26.6 us (78%); whole CTAs a token, or persistent ones, are no faster.
//
// Sums that are not finite are taken once more: dout times a code (up to 448) may be
// beyond fp32 where with the block's power of two it is not.  Where eight products' sum is
// not finite, they are taken of gradients times 2^-16 (exact: bf16's last place is 2^-133),
// and the sums are added in 64 bits; what is NaN stays so.  (4096 x 7168 x 8: 53 us, 970
// where that holds for every sum.)  A warp's tokens have `lanes` lanes each; of a token's n
// sums in dw those are taken that need it, at the end of a token, where nothing else is in
// registers.
__device__ __noinline__ void far_sums(const uint16_t* dout, const uint8_t* yq, const uint8_t* ys, const int32_t* row_of,
                                      uint32_t rows, uint32_t N, int n, bool on, float* dw, uint32_t lanes) {
  const uint32_t l = threadIdx.x & (lanes - 1);
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint32_t row = on ? (uint32_t)row_of[j] : 0xFFFFFFFFu;
    const bool far = row < rows && !(fabsf(dw[j]) <= 3.402823466e38f);
    double sum = 0.0;
#pragma unroll 1
    for (uint32_t v = l; far && v < N / 8 && sum == sum; v += lanes) {
      const uint4 d = ld_nc16(dout + v * 8);
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(yq + (uint64_t)row * N + v * 8));
      const float power = mx_power((uint32_t)__ldg(ys + (uint64_t)row * (N / 32) + (v >> 2)));
      auto dot = [&](float by) {
        uint64_t s = fma2(mul2(unpk_bf16(d.x), pk(by, by)), e4m3x2_f32(q.x), 0);
        s = fma2(mul2(unpk_bf16(d.y), pk(by, by)), e4m3x2_f32(q.x >> 16), s);
        s = fma2(mul2(unpk_bf16(d.z), pk(by, by)), e4m3x2_f32(q.y), s);
        return sum_of(fma2(mul2(unpk_bf16(d.w), pk(by, by)), e4m3x2_f32(q.y >> 16), s));
      };
      const float s = dot(1.0f);
      sum += fabsf(s) <= 3.402823466e38f ? (double)s * (double)power : (double)dot(0x1p-16f) * (65536.0 * (double)power);
    }
    for (uint32_t o = lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (far && l == 0) dw[j] = (float)sum;
  }
}

// (Of one choice five CTAs an SM: 65536 x 1024 38 us, 43 with the four that registers would allow.)
template <int L, int UK>
__global__ void __launch_bounds__(256, UK == 1 ? 5 : 3)
    k_route_weight_grad_ckpt(const uint16_t* __restrict__ dout, const uint8_t* __restrict__ yq, const uint8_t* __restrict__ ys,
                             const int32_t* __restrict__ row_of, uint32_t rows, int64_t T, uint32_t N, int k,
                             float* __restrict__ dw) {
  constexpr int WPT = L / 32;
  __shared__ float red[8][UK];
  const int warp = threadIdx.x >> 5, l = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const uint32_t nv = rows > 0 ? N / 16 : 0, ns = N / 32;
  for (int j0 = 0; j0 < k; j0 += UK) {
    uint32_t row[UK];
    bool there[UK];
    float acc[UK];
#pragma unroll
    for (int j = 0; j < UK; ++j) {
      row[j] = t < T && j0 + j < k ? (uint32_t)row_of[t * k + j0 + j] : 0xFFFFFFFFu;
      there[j] = row[j] < rows;
      row[j] = there[j] ? row[j] : 0u;
      acc[j] = 0.0f;
    }
    if (t < T) {
      for (uint32_t v = l; v < nv; v += L) {
        const uint16_t* dv = dout + t * N + v * 16;
        const uint4 d0 = ld_nc16(dv), d1 = ld_nc16(dv + 8);
        const uint8_t *qv = yq + v * 16, *sv = ys + (v >> 1);
        uint4 q[UK];
        uint32_t b[UK];
#pragma unroll
        for (int j = 0; j < UK; ++j) {
          q[j] = ld_nc16(qv + (uint64_t)row[j] * N);
          b[j] = (uint32_t)__ldg(sv + (uint64_t)row[j] * ns);
        }
        const uint64_t d[8] = {unpk_bf16(d0.x), unpk_bf16(d0.y), unpk_bf16(d0.z), unpk_bf16(d0.w),
                               unpk_bf16(d1.x), unpk_bf16(d1.y), unpk_bf16(d1.z), unpk_bf16(d1.w)};
#pragma unroll
        for (int j = 0; j < UK; ++j) {
          const uint32_t qq[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
          uint64_t s = 0;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            s = fma2(d[2 * h], e4m3x2_f32(qq[h]), s);
            s = fma2(d[2 * h + 1], e4m3x2_f32(qq[h] >> 16), s);
          }
          acc[j] = fmaf(sum_of(s), mx_power(b[j]), acc[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < UK; ++j) {
      acc[j] = lane_sum<(L < 32 ? L : 32)>(acc[j]);
      if (WPT > 1 && (threadIdx.x & 31) == 0) red[warp][j] = acc[j];
    }
    if (WPT > 1) __syncthreads();
    bool far = false;
    if (t < T && l == 0) {
#pragma unroll
      for (int j = 0; j < UK; ++j) {
        float v = acc[j];
        if (WPT > 1)
          for (int i = 1; i < WPT; ++i) v += red[warp + i][j];
        far |= there[j] && !(fabsf(v) <= 3.402823466e38f);
        if (j0 + j < k) dw[t * k + j0 + j] = there[j] ? v : 0.0f;
      }
    }
    if (__any_sync(0xffffffffu, far)) {   // (of a token's warps the first)
      __syncwarp();
      far_sums(dout + t * N, yq, ys, row_of + t * k + j0, rows, N, min(UK, k - j0), t < T, dw + t * k + j0, L < 32 ? L : 32);
    }
    if (WPT > 1) __syncthreads();
  }
}

// Warps per CTA: one CTA per SM, of as many warps as it gets tokens to fill:
// few partial sums, and tokens spread over the SMs (512 tokens: 3.7 us with CTAs
// of four warps, 6.4 with CTAs of 32, without the sums).
template <int V, int G>
int cta_warps(int64_t T, int64_t sms) {
  const int64_t want = (T + sms * (32 / G) - 1) / (sms * (32 / G));
  return want < 4 ? 4 : want > most_warps<V>() ? most_warps<V>() : (int)want;
}

template <int V, int G, bool SIG>
cudaError_t run_fwd(RouterArgs a, int num_sms, cudaStream_t st) {
  a.two = a.k >= 4 && a.T >= 2 * most_warps<V>() * (int64_t)num_sms;
  const bool sums = a.counts != nullptr;
  const bool single = sums && a.T <= SINGLE_CTA_T;
  const int RW = cta_warps<V, G>(a.T, single ? 1 : num_sms), rows = RW * (32 / G);
  const int smem = sums ? (RW * G * V + a.E + 1) * 4 : 0;   // probability sums per warp, counts
  int64_t blocks = single ? 1 : (a.T + rows - 1) / rows;
  const int64_t most = (int64_t)num_sms * (32 / most_warps<V>());
  if (blocks > most) blocks = most;
  if (sums && blocks > ROUTER_MAX_PARTS) blocks = ROUTER_MAX_PARTS;
  k_router_fwd<V, G, SIG><<<(unsigned)blocks, RW * 32, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !sums || blocks == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(JOIN);
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_router_join, a, (int)blocks);
}
template <int V, int G, bool SIG>
cudaError_t run_bwd(const RouterArgs& a, int num_sms, cudaStream_t st) {
  const int RW = cta_warps<V, G>(a.T, num_sms), rows = RW * (32 / G);
  const int smem = rows * G * V * 4;
  int64_t blocks = (a.T + rows - 1) / rows;
  const int64_t most = (int64_t)num_sms * (64 / most_warps<V>());
  if (blocks > most) blocks = most;
  k_router_bwd<V, G, SIG><<<(unsigned)blocks, RW * 32, smem, st>>>(a);
  return cudaGetLastError();
}

// Lanes per token: a whole warp, or for many tokens over few experts a lane to
// every eight of them, so that the steps that do not depend on the experts are
// shared by more tokens (65536 tokens forward: 8 experts, top 2, 7.4 us with one
// lane against 22.8 with 32; 16, top 4, 9.5 against 27.2; 64, top 6, 18.3
// against 27.9; 65536 x 128, top 8, 40 against 45 before both got faster).
// Below eight (32) tokens an SM a warp's shorter way counts for as much or more
// (2048 x 64, top 6: 6.3 us either way; 4096 x 128: 8.3 with 32, 8.8 with 16).
// The backward starts at two lanes: one lane's eight slots took 4.3 us on 4096 x
// 8 against 3.5.  The choice needs k <= lanes x slots.
int lanes_per_token(const RouterArgs& a, int num_sms) {
  if (a.E <= 64 && a.k <= 8 && a.T >= 8 * (int64_t)num_sms)
    return a.E <= 8 && !a.dlogits ? 1 : a.E <= 16 ? 2 : a.E <= 32 ? 4 : 8;
  if (a.E > 64 && a.E <= 128 && a.k <= 16 && a.T >= 32 * (int64_t)num_sms) return 16;
  return 32;
}

}  // namespace

#define FP8MOE_ROUTER(V, G, FN)                                                                               \
  if (g == G && a.E <= G * V)                                                                                 \
    return a.score == FP8MOE_SCORE_SIGMOID ? FN<V, G, true>(a, num_sms, st) : FN<V, G, false>(a, num_sms, st);
#define FP8MOE_ROUTER_ALL(FN)                                                                                 \
  FP8MOE_ROUTER(8, 2, FN) FP8MOE_ROUTER(8, 4, FN) FP8MOE_ROUTER(8, 8, FN) FP8MOE_ROUTER(8, 16, FN)            \
  FP8MOE_ROUTER(1, 32, FN) FP8MOE_ROUTER(2, 32, FN) FP8MOE_ROUTER(4, 32, FN) FP8MOE_ROUTER(8, 32, FN)         \
  FP8MOE_ROUTER(16, 32, FN) FP8MOE_ROUTER(32, 32, FN)

// T == 0: one CTA writes the empty sums
cudaError_t launch_router_fwd(const RouterArgs& a, int num_sms, cudaStream_t st) {
  const int g = lanes_per_token(a, num_sms);
  FP8MOE_ROUTER(8, 1, run_fwd)
  FP8MOE_ROUTER_ALL(run_fwd)
  return cudaErrorInvalidValue;
}
cudaError_t launch_router_bwd(const RouterArgs& a, int num_sms, cudaStream_t st) {
  const int g = lanes_per_token(a, num_sms);
  FP8MOE_ROUTER_ALL(run_bwd)
  return cudaErrorInvalidValue;
}
#undef FP8MOE_ROUTER_ALL
#undef FP8MOE_ROUTER

cudaError_t launch_route_weight_grad(const void* dout, const void* y, int64_t rows, const int32_t* row_of, int64_t T,
                                     int64_t N, int64_t k, float* dw, int num_sms, cudaStream_t st) {
  const uint16_t *d = (const uint16_t*)dout, *yp = (const uint16_t*)y;
  // Lanes per token. Few enough that a lane has chunks to do and a CTA's tokens
  // overlap their dependent loads (60000 tokens x 8 rows of 128: 24.6 us with 16,
  // 39.3 with 32, 109 with 128; of 256: 43.9, 44.3, 111; 49311 x 5 of 528: 57.0,
  // 58.7, 82.4; 8192 x 1 of 1024: 5.5 with 32, 7.5 with 128); many where rows are
  // long, as few long-lived CTAs leave SMs idle at the end (30000 x 8 of 1024:
  // 85.4 with 128, 87.0 with 32; 4096 x 8 of 7168: 79.5 with 256, 80.4 with 128,
  // 81.4 with 32; 2000 x 2 of 8192: 17.8 with 256, 20.2 with 128), and where the
  // tokens would not give every SM a CTA (64 x 8 of 7168: 5.5 with 256, 25.1 with 32).
  const int64_t nv = N / 8;
  int L = nv <= 48 ? 16 : nv < 128 || (k == 1 && nv < 512) ? 32 : nv < 512 ? 128 : 256;
  while (L < 256 && L < nv && T * L < (int64_t)256 * num_sms) L = L == 32 ? 128 : 2 * L;
  const unsigned grid = (unsigned)((T + 256 / L - 1) / (256 / L));
  auto run = [&](auto kern) { kern<<<grid, 256, 0, st>>>(d, yp, row_of, (uint32_t)rows, T, N, (int)k, dw); };
#define FP8MOE_WG(UK)                                     \
  if (L == 16) run(k_route_weight_grad<16, UK>);          \
  else if (L == 32) run(k_route_weight_grad<32, UK>);     \
  else if (L == 128) run(k_route_weight_grad<128, UK>);   \
  else run(k_route_weight_grad<256, UK>)
  switch (k) {
    case 1: FP8MOE_WG(1); break;
    case 2: FP8MOE_WG(2); break;
    case 3:
    case 4: FP8MOE_WG(4); break;
    case 5:
    case 6: FP8MOE_WG(6); break;
    default: FP8MOE_WG(8);
  }
#undef FP8MOE_WG
  return cudaGetLastError();
}

cudaError_t launch_route_weight_grad_ckpt(const void* dout, const void* yq, const uint8_t* ys, int64_t rows,
                                          const int32_t* row_of, int64_t T, int64_t N, int64_t k, float* dw, int num_sms,
                                          cudaStream_t st) {
  // lanes per token by the rule of the bf16 form, of chunks twice as long
  const int64_t nv = N / 16;
  int L = nv <= 8 ? 8 : nv <= 48 ? 16 : nv < 256 || (k == 1 && nv < 512) ? 32 : nv < 512 ? 128 : 256;
  while (L < 256 && L < nv && T * L < (int64_t)256 * num_sms) L = L == 32 ? 128 : 2 * L;
  const unsigned grid = (unsigned)((T + 256 / L - 1) / (256 / L));
  auto run = [&](auto kern) {
    kern<<<grid, 256, 0, st>>>((const uint16_t*)dout, (const uint8_t*)yq, ys, row_of, (uint32_t)rows, T, (uint32_t)N, (int)k, dw);
  };
#define FP8MOE_WG(UK)                                          \
  if (L == 8) run(k_route_weight_grad_ckpt<8, UK>);            \
  else if (L == 16) run(k_route_weight_grad_ckpt<16, UK>);     \
  else if (L == 32) run(k_route_weight_grad_ckpt<32, UK>);     \
  else if (L == 128) run(k_route_weight_grad_ckpt<128, UK>);   \
  else run(k_route_weight_grad_ckpt<256, UK>)
  switch (k) {
    case 1: FP8MOE_WG(1); break;
    case 2: FP8MOE_WG(2); break;
    case 3:
    case 4: FP8MOE_WG(4); break;
    case 5:
    case 6: FP8MOE_WG(6); break;
    default: FP8MOE_WG(8);
  }
#undef FP8MOE_WG
  return cudaGetLastError();
}

}  // namespace fp8moe
