// The whole expert layer of a few tokens on MXFP8 weights, in one launch:
//
//   out[t] = sum_j w[t, j] * W2[e] (silu(W1g[e] x[t]) * (W1u[e] x[t])),  e = idx[t, j]
//
// Bound by the weights' bytes: every expert that some token chose is read once,
// 3 H F codes and their scales, for 2 flops a code and token.  So the weights
// are the M operand of the tensor cores' block-scaled product (128 rows of one
// expert, straight from HBM to shared memory to tcgen05.mma, never converted),
// and the tokens its N operand.
//
// The tokens keep all their digits.  In a block of 32 values scaled so that the
// largest lies in [128, 256), the nearest e4m3 value leaves a rest of at most 8,
// which times 2^5 is again such a block, with its own scale: a bf16 value is two
// such terms exactly (8 bits, four and four), an fp32 value three to 2^-13.  The
// terms are further columns of N, where the tensor core has room: N is at least
// 16, and the weights' arrival leaves it idle most of the time.
//
// Both products are one stream of 16 KB pieces (128 rows x 128 of K) over all
// (expert, row tile, k) in order, cut into equal runs, one per CTA; a tile's
// partial sums (fp32, at most a few per tile) go to the workspace and are added
// in order after a grid-wide meeting.  The producer does not take part in the
// meetings: while the others add, it fills its ring with W2.
//   warps 0-3   accumulators to partial sums;  4  weights by TMA;  5  MMA issue;
//   warps 6-13  the tokens' terms, one group of four warps a piece in turn.
#include <cooperative_groups.h>
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "moe_ops.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace fp8moe {
namespace {

constexpr int DC_THREADS = 448;
constexpr int DC_JOIN = 384;              // threads that add partial sums: all but the producer's and the issuer's
constexpr int DC_WARP_TMA = 4, DC_WARP_MMA = 5, DC_WARP_B = 6;
constexpr int DC_A_BYTES = 128 * 128;
constexpr int DC_NB = DECODE_ENTRY_PAIRS;   // pairs of one entry: a pass over an expert's weights
constexpr int DC_ACC = 3 * DC_NB;         // TMEM columns of an accumulator
constexpr int DC_SF = 2 * DC_ACC;         // first TMEM column of the scales: 12 per slot
constexpr int DC_MAX_BS = 8;
static_assert(DC_SF + 12 * DC_MAX_BS <= 512, "tensor memory");
constexpr int DC_DEAD = 0xFFFF;

__host__ __device__ constexpr int up16(int v) { return (v + 15) / 16 * 16; }

// Shared memory: rings of weights (sa slots) and of terms (sb slots), the plan.
struct DecodeSmem {
  int sa, sb, b_bytes, sfb_bytes;
  int sfa, b, sfb, bars, plan, total;     // the weights' ring is at 0
};

// The plan of a call, in shared memory: the live pairs (token, choice) in the
// order of their experts, cut into entries of one expert and at most DC_NB pairs.
struct Plan {
  uint32_t* ent;      // expert | first pair << 10 | pairs << 20
  float* w;           // [P] weights of the pairs
  uint16_t* order;    // [live] pair of each place
  uint16_t* pos;      // [P] place of each pair, or DC_DEAD
  uint16_t* ent_of;   // [live] entry of each place
  int* num;           // live pairs, entries
  FP8MOE_DEV Plan(uint8_t* p, int P, int max_ent) {
    num = (int*)p;
    ent = (uint32_t*)(p + 16);
    w = (float*)(ent + max_ent);
    order = (uint16_t*)(w + P);
    pos = order + P;
    ent_of = pos + P;
  }
};

FP8MOE_DEV bool live_pair(int e, float w, int E) { return e >= 0 && e < E && w != 0.0f; }

// At most 32 pairs, one warp: ranks by comparing every two.
FP8MOE_DEV void plan_warp(const DecodeArgs& a, const Plan& pl, int lane) {
  const int P = a.P;
  int e = lane < P ? __ldg(a.idx + lane) : -1;
  const float w = lane < P ? __ldg(a.w + lane) : 0.0f;
  const bool live = live_pair(e, w, a.E);
  if (!live) e = INT32_MAX;
  int rank = 0, before = 0, same = 0;
  for (int q = 0; q < P; ++q) {
    const int eq = __shfl_sync(0xffffffffu, e, q);
    rank += eq < e || (eq == e && q < lane);
    before += eq == e && q < lane;
    same += eq == e;
  }
  const uint32_t heads = __ballot_sync(0xffffffffu, live && before == 0);
  int ent = 0;
  for (int q = 0; q < P; ++q) {
    const int eq = __shfl_sync(0xffffffffu, e, q);
    ent += (heads >> q & 1) && eq < e;
  }
  if (lane < P) {
    pl.w[lane] = w;
    pl.pos[lane] = (uint16_t)(live ? rank : DC_DEAD);
  }
  if (live) {
    pl.order[rank] = (uint16_t)lane;
    pl.ent_of[rank] = (uint16_t)ent;
    if (before == 0) pl.ent[ent] = (uint32_t)e | (uint32_t)rank << 10 | (uint32_t)same << 20;
  }
  const int n = __popc(__ballot_sync(0xffffffffu, live));
  if (lane == 0) pl.num[0] = n, pl.num[1] = __popc(heads);
  __syncwarp();
}

// More pairs, the whole block: counts per expert, their scan, and a pair's
// place among its expert's by counting the earlier ones (their order decides
// which entry of a crowded expert a pair is in, so it is not left to atomics).
// scratch: E + P + 64 words.
FP8MOE_DEV void plan_block(const DecodeArgs& a, const Plan& pl, int* scratch) {
  int *cnt = scratch, *ids = scratch + a.E, *tot = ids + a.P;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int e = tid; e < a.E; e += DC_THREADS) cnt[e] = 0;
  __syncthreads();
  for (int p = tid; p < a.P; p += DC_THREADS) {
    const int e = __ldg(a.idx + p);
    const float w = __ldg(a.w + p);
    const bool live = live_pair(e, w, a.E);
    pl.w[p] = w;
    ids[p] = live ? e : -1;
    if (live) atomicAdd(cnt + e, 1);
  }
  __syncthreads();
  // scan of (pairs, entries) in one word, chunks of 32 experts
  const int chunks = (a.E + 31) / 32;
  for (int c = warp; c < chunks; c += DC_THREADS / 32) {
    const int e = c * 32 + lane, n = e < a.E ? cnt[e] : 0;
    const uint32_t own = (uint32_t)n << 16 | (uint32_t)((n + DC_NB - 1) / DC_NB);
    uint32_t v = own;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) tot[c] = (int)v;
    if (e < a.E) cnt[e] = (int)(v - own);
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t own = lane < chunks ? (uint32_t)tot[lane] : 0;
    uint32_t v = own;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    tot[lane] = (int)(v - own);
    if (lane == 31) pl.num[0] = (int)(v >> 16), pl.num[1] = (int)(v & 0xFFFFu);
  }
  __syncthreads();
  for (int p = tid; p < a.P; p += DC_THREADS) {
    const int e = ids[p];
    if (e < 0) {
      pl.pos[p] = DC_DEAD;
      continue;
    }
    int before = 0, after = 0;
    for (int q = 0; q < p; ++q) before += ids[q] == e;
    const uint32_t base = (uint32_t)cnt[e] + (uint32_t)tot[e >> 5];
    const int place = (int)(base >> 16) + before, ent = (int)(base & 0xFFFFu) + before / DC_NB;
    pl.order[place] = (uint16_t)p;
    pl.pos[p] = (uint16_t)place;
    pl.ent_of[place] = (uint16_t)ent;
    if (before % DC_NB == 0) {
      for (int q = p; q < a.P && after < DC_NB; ++q) after += ids[q] == e;
      pl.ent[ent] = (uint32_t)e | (uint32_t)place << 10 | (uint32_t)after << 20;
    }
  }
  __syncthreads();
}

// One product's stream of pieces: nent entries x rt row tiles x kt pieces.
struct Stream {
  uint32_t C, runs;   // pieces, CTAs that have a run of them
  int rt, kt;
  FP8MOE_DEV Stream(int nent, int rt_, int kt_, uint32_t grid) : rt(rt_), kt(kt_) {
    C = (uint32_t)nent * rt * kt;
    const uint32_t want = (C + DECODE_MIN_RUN - 1) / DECODE_MIN_RUN;
    runs = want < grid ? want : grid;
  }
  FP8MOE_DEV uint32_t first(uint32_t cta) const { return cta < runs ? cta * C / runs : C; }
  FP8MOE_DEV uint32_t owner(uint32_t c) const { return ((c + 1) * runs - 1) / C; }
  // partial sums of a tile: the CTAs whose runs meet it
  FP8MOE_DEV int parts(uint32_t tile) const { return (int)(owner(tile * kt + kt - 1) - owner(tile * kt)) + 1; }
};

// A CTA's place in a stream, stepped piece by piece.
struct Walk {
  uint32_t left;      // pieces to go in this run
  int ent, row, k;    // entry, row tile, piece of K
  uint32_t tile;
  FP8MOE_DEV Walk(const Stream& s, uint32_t cta) {
    const uint32_t lo = s.first(cta), hi = s.first(cta + 1);
    left = hi - lo;
    tile = lo / s.kt;
    k = (int)(lo - tile * s.kt);
    ent = (int)(tile / s.rt);
    row = (int)(tile - (uint32_t)ent * s.rt);
  }
  FP8MOE_DEV bool last(const Stream& s) const { return left == 1 || k == s.kt - 1; }   // of its tile, in this run
  FP8MOE_DEV void step(const Stream& s) {
    --left;
    if (++k == s.kt) {
      k = 0;
      ++tile;
      if (++row == s.rt) row = 0, ++ent;
    }
  }
};

FP8MOE_DEV void cp_scales(uint32_t taddr, uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d));
}
FP8MOE_DEV void mma_mx1(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb));
}
FP8MOE_DEV void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
FP8MOE_DEV void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
FP8MOE_DEV uint32_t ld_acquire_gpu(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// one CTA more at a meeting, and the (bounded) wait for the others; one thread
FP8MOE_DEV void meet(uint32_t* count, uint32_t n, int* status, volatile int* abort_flag) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
  const uint64_t t0 = globaltimer();
  while (ld_acquire_gpu(count) < n) {
    if (globaltimer() - t0 > 2 * WAIT_LIMIT_NS) {   // (a CTA whose own wait ran out still comes)
      set_status(status, FP8MOE_ERR_TIMEOUT);
      *abort_flag = 1;
      return;
    }
  }
}

// two e4m3 codes -> their values
FP8MOE_DEV float2 e4m3x2_value(uint32_t c) {
  uint32_t h;
  asm("{\n .reg .b16 s;\n cvt.u16.u32 s, %1;\n cvt.rn.f16x2.e4m3x2 %0, s;\n}" : "=r"(h) : "r"(c));
  float2 v;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}" : "=f"(v.x), "=f"(v.y) : "r"(h));
  return v;
}

// Eight neighbouring values of a row to NT terms each (rows r0 .. of the term
// tile, 128-byte swizzle; scale bytes in 128x4 order).  Four lanes hold a block.
// A block that is not finite becomes NaN, and so does its token.
template <int NT>
FP8MOE_DEV void put_terms(float (&v)[8], uint8_t* tile, uint8_t* sf, int r0, int j, bool on) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, m, o);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(u));
  }
  const uint32_t field = (__float_as_uint(m) >> 23) & 0xFFu;
  // (blocks below 2^-110 are not scaled all the way up: the last term's byte stays above 0)
  const uint32_t ef = field < 17u ? 17u : field;
  const bool finite = field != 255u;
  const float mul = __uint_as_float((261u - ef) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= mul;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = cvt_e4m3x2(v[2 * i], v[2 * i + 1]);
      if (t + 1 < NT) {
        const float2 b = e4m3x2_value(c[i]);
        v[2 * i] = (v[2 * i] - b.x) * 32.0f;
        v[2 * i + 1] = (v[2 * i + 1] - b.y) * 32.0f;
      }
    }
    uint2 q = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (!finite) q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (!on) continue;
    const int r = r0 + t;
    *reinterpret_cast<uint2*>(tile + r * 128 + (((j >> 1) ^ (r & 7)) << 4) + (j & 1) * 8) = q;
    if ((j & 3) == 0)
      sf[(r >> 7) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j >> 2)] = (uint8_t)(finite ? ef - 7u - 5u * t : 127u);
  }
}

__global__ void __launch_bounds__(DC_THREADS, 1)
    k_decode(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2, DecodeArgs a, DecodeSmem L) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ int abort_s;
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cta = blockIdx.x, grid = gridDim.x;
  volatile int* abort_flag = &abort_s;
  uint64_t* a_full = (uint64_t*)(smem + L.bars);
  uint64_t* a_empty = a_full + L.sa;
  uint64_t* b_full = a_empty + L.sa;
  uint64_t* b_empty = b_full + L.sb;
  uint64_t* acc_full = b_empty + L.sb;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  const Plan pl(smem + L.plan, a.P, a.max_ent);
  auto fail = [&]() {
    set_status(a.status, FP8MOE_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == DC_WARP_TMA && lane == 0) {
    abort_s = 0;
    for (int i = 0; i < L.sa; ++i) mbar_init(&a_full[i], 1), mbar_init(&a_empty[i], 1);
    for (int i = 0; i < L.sb; ++i) mbar_init(&b_full[i], 4), mbar_init(&b_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], 4);
    mbar_init(drain, 1);
    mbar_fence_init();
  }
  if (warp == DC_WARP_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_s)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  if (cta == 0 && tid < 3) a.meets[tid * 32] = 0;
  if (a.P <= 32) {
    if (warp == DC_WARP_TMA) plan_warp(a, pl, lane);
  } else {
    plan_block(a, pl, (int*)(smem + L.b));   // (ends with a block barrier)
  }

  // ---- the producer's first ring fills leave before the grid meets
  // (piece i of the CTA's two runs goes to slot i % sa)
  uint32_t issued = 0;
  auto produce = [&](const Stream& s1, const Stream& s2, Walk& w1, Walk& w2, uint32_t upto) {
    for (; issued < upto; ++issued) {
      const bool one = w1.left > 0;
      const Stream& s = one ? s1 : s2;
      Walk& w = one ? w1 : w2;
      const int slot = (int)(issued % (uint32_t)L.sa);
      const uint32_t turn = issued / (uint32_t)L.sa;
      if (!mbar_wait(&a_empty[slot], (turn & 1u) ^ 1u, abort_flag)) {
        fail();
        return;
      }
      const int e = (int)(pl.ent[w.ent] & 1023u);
      if (!(a.stall && cta == 0 && issued == 0)) {
        mbar_expect_tx(&a_full[slot], DC_A_BYTES + 512);
        tma_load_3d(smem + slot * DC_A_BYTES, one ? &tm1 : &tm2, &a_full[slot], w.k * 128, w.row * 128, e);
        bulk_load(smem + L.sfa + slot * 512, (one ? a.s1 : a.s2) + (((int64_t)e * s.rt + w.row) * s.kt + w.k) * 512, 512,
                  &a_full[slot]);
      }
      w.step(s);
    }
  };
  const int K1 = a.H, K2 = a.F, R1 = 2 * a.F, R2 = a.H;
  const int rt1 = (R1 + 127) / 128, kt1 = (K1 + 127) / 128, rt2 = (R2 + 127) / 128, kt2 = (K2 + 127) / 128;
  if (warp == DC_WARP_TMA && lane == 0) {
    const int ne = pl.num[1];
    const Stream s1(ne, rt1, kt1, grid), s2(ne, rt2, kt2, grid);
    Walk w1(s1, cta), w2(s2, cta);
    const uint32_t all = w1.left + w2.left;
    produce(s1, s2, w1, w2, all < (uint32_t)L.sa ? all : (uint32_t)L.sa);
  }
  __syncwarp();
  // the meetings' counters are zero, the barriers exist, the plan is made
  cooperative_groups::this_grid().sync();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  const int nlive = pl.num[0], nent = pl.num[1];
  const Stream s1(nent, rt1, kt1, grid), s2(nent, rt2, kt2, grid);

  if (warp == DC_WARP_TMA) {
    // ======================= weights =======================
    if (lane == 0) {
      Walk w1(s1, cta), w2(s2, cta);
      const uint32_t all = w1.left + w2.left;
      for (uint32_t i = 0; i < issued; ++i) w1.left > 0 ? w1.step(s1) : w2.step(s2);
      produce(s1, s2, w1, w2, all);
      // no copy stays in flight after a wait that ran out
      if (*abort_flag)
        for (uint32_t i = issued > (uint32_t)L.sa ? issued - L.sa : 0; i < issued; ++i)
          if (!(a.stall && cta == 0 && i == 0)) (void)mbar_wait(&a_full[i % L.sa], (i / (uint32_t)L.sa) & 1u, nullptr);
    }
    __syncwarp();
  } else if (warp == DC_WARP_MMA) {
    // ======================= products =======================
    if (lane == 0) {
      uint32_t n = 0, seg = 0;
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Stream& s = ph ? s2 : s1;
        const int K = ph ? K2 : K1, terms = ph ? 3 : 2;
        bool fresh = true;
        for (Walk w(s, cta); w.left > 0; w.step(s), ++n) {
          const int sa = (int)(n % (uint32_t)L.sa), sb = (int)(n % (uint32_t)L.sb);
          if (fresh && !mbar_wait(&acc_empty[seg & 1], ((seg >> 1) & 1u) ^ 1u, abort_flag)) ok = false;
          if (!ok || !mbar_wait(&a_full[sa], (n / (uint32_t)L.sa) & 1u, abort_flag) ||
              !mbar_wait(&b_full[sb], (n / (uint32_t)L.sb) & 1u, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const int cols = up16((int)(pl.ent[w.ent] >> 20) * terms);
          const uint32_t sf = tmem + DC_SF + sb * 12, d = tmem + (seg & 1) * DC_ACC;
          const uint32_t sfb = smem_u32(smem + L.sfb + sb * L.sfb_bytes);
          cp_scales(sf, smem_u32(smem + L.sfa + sa * 512));
          cp_scales(sf + 4, sfb);
          if (cols > 128) cp_scales(sf + 8, sfb + 512);
          const uint64_t ad = sdesc_sw128(smem_u32(smem + sa * DC_A_BYTES));
          const uint64_t bd = sdesc_sw128(smem_u32(smem + L.b + sb * L.b_bytes));
          const uint32_t id = (uint32_t)(cols >> 3) << 17 | 1u << 23 | 8u << 24;
          const int blocks = min(4, (K - w.k * 128) / 32);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < blocks)
              mma_mx1(d, ad + 2 * k, bd + 2 * k, id | (uint32_t)k << 4 | (uint32_t)k << 29, sf, sf + 4, !fresh || k > 0);
          tc_commit(&a_empty[sa]);
          tc_commit(&b_empty[sb]);
          fresh = w.last(s);
          if (fresh) tc_commit(&acc_full[seg++ & 1]);
        }
      }
      // every product has completed before tensor memory is given back
      tc_commit(drain);
      if (!mbar_wait(drain, 0, nullptr)) set_status(a.status, FP8MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    const bool epi = warp < 4;
    const int jt = epi ? tid : tid - 64;           // thread among those that add
    uint32_t n = 0, seg = 0;                       // pieces and segments so far
    // ======================= terms =======================
    auto terms_of = [&](auto phase) {
      constexpr int PH = decltype(phase)::value, NT = PH ? 3 : 2;
      const Stream& s = PH ? s2 : s1;
      const int K = PH ? K2 : K1;
      const int group = (warp - DC_WARP_B) >> 2, sub = ((warp - DC_WARP_B) & 3) * 2 + (lane >> 4), j = lane & 15;
      auto load = [&](const Walk& w, int i, uint32_t ent, uint4 (&r)[2]) {
        const int place = (int)(ent >> 10 & 1023u) + i, k = w.k * 128 + j * 8;
        if (i >= (int)(ent >> 20) || k >= K) return;
        if constexpr (PH == 0) {
          r[0] = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)(pl.order[place] / a.k) * a.ldx + k));
        } else {
          const uint4* p = reinterpret_cast<const uint4*>(a.act + (int64_t)place * a.F + k);
          r[0] = __ldcg(p);
          r[1] = __ldcg(p + 1);
        }
      };
      uint4 next[2] = {};
      Walk w(s, cta);
      const uint32_t total = w.left;
      const uint32_t n0 = n;
      // (the groups alternate over both runs together)
      auto skip = [&]() {
        w.step(s);
        ++n;
      };
      while (w.left > 0 && (n & 1u) != (uint32_t)group) skip();
      if (w.left > 0) load(w, sub, pl.ent[w.ent], next);
      while (w.left > 0) {
        const int sb = (int)(n % (uint32_t)L.sb);
        const uint32_t ent = pl.ent[w.ent], turn = n / (uint32_t)L.sb;
        const int pairs = (int)(ent >> 20), k0 = w.k * 128;
        uint4 cur[2] = {next[0], next[1]};
        Walk here = w;
        skip();
        if (w.left > 0) skip();
        if (w.left > 0) load(w, sub, pl.ent[w.ent], next);
        if (!mbar_wait(&b_empty[sb], (turn & 1u) ^ 1u, abort_flag)) {
          fail();
          break;
        }
        uint8_t *tile = smem + L.b + sb * L.b_bytes, *sf = smem + L.sfb + sb * L.sfb_bytes;
        for (int i0 = 0; i0 < pairs; i0 += 8) {
          const int i = i0 + sub;
          if (i0 > 0) load(here, i, ent, cur);
          float v[8];
          if constexpr (PH == 0) {
            const uint32_t q[4] = {cur[0].x, cur[0].y, cur[0].z, cur[0].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) v[2 * c] = bf16_lo(q[c]), v[2 * c + 1] = bf16_hi(q[c]);
          } else {
            const uint32_t q[8] = {cur[0].x, cur[0].y, cur[0].z, cur[0].w, cur[1].x, cur[1].y, cur[1].z, cur[1].w};
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = __uint_as_float(q[c]);
          }
          const bool on = i < pairs && k0 + j * 8 < K;
          // (a block's four lanes are on or off together; the shuffles are the warp's)
          if (__any_sync(0xffffffffu, on)) put_terms<NT>(v, tile, sf, i * NT, j, on);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_full[sb]);
      }
      n = n0 + total;
    };
    // ======================= accumulators =======================
    auto sums_of = [&](auto phase) {
      constexpr int PH = decltype(phase)::value, NT = PH ? 3 : 2;
      const Stream& s = PH ? s2 : s1;
      const int R = PH ? R2 : R1;
      for (Walk w(s, cta); w.left > 0; w.step(s)) {
        if (!w.last(s)) continue;
        const uint32_t ent = pl.ent[w.ent];
        const int first = (int)(ent >> 10 & 1023u), pairs = (int)(ent >> 20);
        const int part = (int)(cta - s.owner(w.tile * s.kt));
        const int row = w.row * 128 + warp * 32 + lane;
        float* dst = a.part + ((int64_t)part * nlive + first) * R + row;
        const uint32_t buf = seg & 1;
        if (!mbar_wait(&acc_full[buf], (seg >> 1) & 1u, abort_flag)) {
          fail();
          break;
        }
        ++seg;
        tc_fence_after();
        const uint32_t src = tmem + buf * DC_ACC + ((uint32_t)(warp * 32) << 16);
        for (int i0 = 0; i0 < pairs; i0 += 8) {
          uint32_t r[24];
#pragma unroll
          for (int c = 0; c < NT; ++c) tmem_ld8(src + i0 * NT + c * 8, *reinterpret_cast<uint32_t(*)[8]>(r + c * 8));
          tmem_ld_wait();
          if (i0 + 8 >= pairs) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v = 0.0f;   // the smallest term first
#pragma unroll
            for (int t = NT - 1; t >= 0; --t) v += __uint_as_float(r[i * NT + t]);
            if (i0 + i < pairs && row < R) dst[(int64_t)(i0 + i) * R] = v;
          }
        }
      }
    };
    // partial sums of a tile in order, four neighbouring rows
    auto gather = [&](const Stream& s, int R, int place, int ent, int row) {
      const int parts = s.parts((uint32_t)ent * s.rt + row / 128);
      const float4* p = reinterpret_cast<const float4*>(a.part + (int64_t)place * R + row);
      const int64_t step = (int64_t)nlive * R / 4;
      float4 v = __ldcg(p);
      for (int i = 1; i < parts; ++i) {
        const float4 u = __ldcg(p + i * step);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      return v;
    };
    // task i of a join: runs of eight tasks a CTA in turn
    const uint32_t t0 = (((uint32_t)jt >> 3) * grid + cta) * 8 + (jt & 7), tstep = DC_JOIN / 8 * grid * 8;

    using One = std::integral_constant<int, 0>;
    using Two = std::integral_constant<int, 1>;
    auto meeting = [&](int i) {
      if (epi) {
        if (tid == 0) meet(a.meets + 32 * i, grid, a.status, abort_flag);
      }
      bar_sync(2, DC_JOIN);
    };
    if (epi) {
      sums_of(One{});
      __threadfence();
      bar_sync(1, 128);
    } else {
      terms_of(One{});
    }
    meeting(0);
    // the activation, from the first product's partial sums
    {
      const uint32_t per = (uint32_t)a.F / 4, tasks = (uint32_t)nlive * per;
      for (uint32_t i = t0; i < tasks; i += tstep) {
        const int place = (int)(i / per), f = (int)(i - (uint32_t)place * per) * 4, ent = pl.ent_of[place];
        const float4 g = gather(s1, R1, place, ent, f), u = gather(s1, R1, place, ent, a.F + f);
        float4 o;
        o.x = g.x / (1.0f + expf(-g.x)) * u.x;
        o.y = g.y / (1.0f + expf(-g.y)) * u.y;
        o.z = g.z / (1.0f + expf(-g.z)) * u.z;
        o.w = g.w / (1.0f + expf(-g.w)) * u.w;
        __stcg(reinterpret_cast<float4*>(a.act + (int64_t)place * a.F + f), o);
      }
    }
    __threadfence();
    bar_sync(2, DC_JOIN);
    meeting(1);
    if (epi) {
      sums_of(Two{});
      __threadfence();
      bar_sync(1, 128);
    } else {
      terms_of(Two{});
    }
    meeting(2);
    // the weighted sum over a token's experts
    {
      const uint32_t per = (uint32_t)a.H / 4, tasks = (uint32_t)a.T * per;
      for (uint32_t i = t0; i < tasks; i += tstep) {
        const int t = (int)(i / per), h = (int)(i - (uint32_t)t * per) * 4;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j = 0; j < a.k; ++j) {
          const int place = pl.pos[t * a.k + j];
          if (place == DC_DEAD) continue;
          const float wj = pl.w[t * a.k + j];
          const float4 v = gather(s2, R2, place, pl.ent_of[place], h);
          o.x = fmaf(wj, v.x, o.x), o.y = fmaf(wj, v.y, o.y), o.z = fmaf(wj, v.z, o.z), o.w = fmaf(wj, v.w, o.w);
        }
        *reinterpret_cast<uint2*>(a.out + (int64_t)t * a.H + h) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == DC_WARP_MMA) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Largest number of partial sums of a tile, whatever the routing, when at least
// `ents` entries are live: a run has at least `s` pieces.
int64_t most_parts(int64_t ents, int64_t rt, int64_t kt) {
  constexpr int64_t grid = DECODE_MAX_CTAS;
  const int64_t C = ents * rt * kt;
  const int64_t s = C < DECODE_MIN_RUN ? 1 : C < grid * DECODE_MIN_RUN ? (DECODE_MIN_RUN + 1) / 2 : C / grid;
  const int64_t p = (kt - 1) / s + 2;
  return p < kt ? p : kt;
}
// floats of the partial sums [parts][live pairs][R]: the most over any number of live pairs
int64_t part_floats(int64_t P, int64_t R, int64_t K) {
  const int64_t rt = (R + 127) / 128, kt = (K + 127) / 128;
  int64_t most = 0;
  for (int64_t ents = 1; (ents - 1) * DC_NB < P; ++ents) {
    const int64_t n = ents * DC_NB < P ? ents * DC_NB : P;
    const int64_t v = most_parts(ents, rt, kt) * n * R;
    if (v > most) most = v;
  }
  return most;
}

DecodeSmem layout(int P, int max_ent, int max_smem) {
  DecodeSmem L{};
  const int nb = P < DC_NB ? (P + 7) / 8 * 8 : DC_NB, rows = up16(3 * nb);
  L.b_bytes = (rows * 128 + 1023) / 1024 * 1024;
  L.sfb_bytes = rows > 128 ? 1024 : 512;
  L.sb = nb <= 16 ? 6 : nb <= 32 ? 4 : 2;
  const int plan = 16 + max_ent * 4 + P * 10;
  const int bars = 8 * (2 * 16 + 2 * DC_MAX_BS + 8);
  const int fixed = L.sb * (L.b_bytes + L.sfb_bytes) + bars + plan + 64;
  L.sa = (max_smem - 2048 - fixed) / (DC_A_BYTES + 512);   // 1024 to align the rings, 1024 for what is static
  if (L.sa > 13) L.sa = 13;
  L.b = L.sa * DC_A_BYTES;
  L.sfa = L.b + L.sb * L.b_bytes;
  L.sfb = L.sfa + L.sa * 512;
  L.bars = L.sfb + L.sb * L.sfb_bytes;
  L.plan = L.bars + bars;
  L.total = (L.plan + plan + 15) / 16 * 16;
  return L;
}

int64_t max_entries(int64_t P, int64_t E) { return (P < E ? P : E) + P / DC_NB; }

}  // namespace

// pieces are counted in 32 bits, times the CTAs
bool decode_fits(int64_t P, int64_t E, int64_t H, int64_t F) {
  const int64_t kh = (H + 127) / 128, kf = (F + 127) / 128, f2 = (2 * F + 127) / 128;
  return max_entries(P, E) * kh * (f2 > kf ? f2 : kf) * DECODE_MAX_CTAS < (int64_t)1 << 32;
}

int64_t decode_workspace_bytes(int64_t P, int64_t H, int64_t F) {
  const int64_t p1 = part_floats(P, 2 * F, H), p2 = part_floats(P, H, F);
  return DECODE_MEETS_BYTES + ((p1 > p2 ? p1 : p2) + P * F) * (int64_t)sizeof(float);
}

cudaError_t launch_decode(DecodeArgs a, void* workspace, int num_sms, int max_smem, cudaStream_t st) {
  a.P = a.T * a.k;
  a.max_ent = (int)max_entries(a.P, a.E);
  const DecodeSmem L = layout(a.P, a.max_ent, max_smem);
  if (L.sa < 2 || (a.P > 32 && (a.E + a.P + 64) * 4 > L.sb * L.b_bytes)) return cudaErrorNotSupported;
  const int64_t c1 = (int64_t)a.max_ent * ((2 * a.F + 127) / 128) * ((a.H + 127) / 128);
  const int64_t c2 = (int64_t)a.max_ent * ((a.H + 127) / 128) * ((a.F + 127) / 128);
  const int64_t c = c1 > c2 ? c1 : c2, want = (c + DECODE_MIN_RUN - 1) / DECODE_MIN_RUN;
  int64_t grid = num_sms < DECODE_MAX_CTAS ? num_sms : DECODE_MAX_CTAS;
  if (want < grid) grid = want;
  const int64_t p1 = part_floats(a.P, 2 * (int64_t)a.F, a.H), p2 = part_floats(a.P, a.H, a.F);
  a.meets = (uint32_t*)workspace;
  a.part = (float*)((uint8_t*)workspace + DECODE_MEETS_BYTES);
  a.act = a.part + (p1 > p2 ? p1 : p2);
  a.stall = take_ring_stall_hook();
  CUtensorMap tm[2];
  const int64_t R[2] = {2 * (int64_t)a.F, a.H}, K[2] = {a.H, a.F};
  const uint8_t* q[2] = {a.q1, a.q2};
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[3] = {(cuuint64_t)K[i], (cuuint64_t)R[i], (cuuint64_t)a.E};
    const cuuint64_t strides[2] = {(cuuint64_t)K[i], (cuuint64_t)(K[i] * R[i])};
    const cuuint32_t box[3] = {128, 128, 1};
    if (!make_tmap(&tm[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, q[i], 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(k_decode, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem - 1024);
  if (e != cudaSuccess) return e;
  void* args[] = {&tm[0], &tm[1], &a, const_cast<DecodeSmem*>(&L)};
  return cudaLaunchCooperativeKernel((const void*)k_decode, dim3((unsigned)grid), dim3(DC_THREADS), args, L.total + 1024, st);
}

}  // namespace fp8moe
