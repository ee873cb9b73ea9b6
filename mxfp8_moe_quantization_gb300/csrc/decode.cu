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
// in order after a grid-wide meeting.  The terms are made once, into the
// workspace, as the tensor core reads them (128-byte swizzle, 128x4 scales): a
// piece's share of them is one bulk copy.  The weights' producer takes no part in
// the meetings: while the others add, it fills its ring with W2.
//   warps 0-3  accumulators to partial sums;  4  weights by TMA;  5  MMA issue;
//   6  terms and scales to shared memory;  0-3 and 7-13  terms, sums, results.
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
constexpr int DC_WARP_TMA = 4, DC_WARP_MMA = 5, DC_WARP_B = 6;
constexpr int DC_JOIN = DC_THREADS - 96;  // threads that make terms and add partial sums: all but those three warps'
constexpr int DC_A_BYTES = 128 * 128;
constexpr int DC_NB = DECODE_ENTRY_PAIRS;   // pairs of one entry: a pass over an expert's weights
constexpr int DC_ACC = 3 * DC_NB;         // TMEM columns of an accumulator
constexpr int DC_SF = 2 * DC_ACC;         // first TMEM column of the scales: 12 per slot
constexpr int DC_MAX_BS = 8;
static_assert(DC_SF + 12 * DC_MAX_BS <= 512, "tensor memory");
constexpr int DC_DEAD = 0xFFFF;

__host__ __device__ constexpr int up16(int v) { return (v + 15) / 16 * 16; }

// Shared memory: the ring of weights (sa slots, at 0), that of terms with the
// terms' and the weights' scales (sb slots each), the plan.
struct DecodeSmem {
  int sa, sb, b_bytes, sfb_bytes;
  int sfa, b, sfb, bars, plan, total;
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

// A CTA's run of a stream, segment by segment: the pieces of one tile that are
// in the run.
struct Run {
  uint32_t left, tile;   // pieces to go, this segment's among them; row tile over all entries
  int n, k;              // pieces of this segment, the first one's place along K
  int ent, row;
  FP8MOE_DEV Run(const Stream& s, uint32_t cta) {
    const uint32_t lo = s.first(cta);
    left = s.first(cta + 1) - lo;
    tile = lo / s.kt;
    k = (int)(lo - tile * s.kt);
    ent = (int)(tile / s.rt);
    row = (int)(tile - (uint32_t)ent * s.rt);
    n = (int)min(left, (uint32_t)(s.kt - k));
  }
  FP8MOE_DEV void next(const Stream& s) {
    left -= n;
    k = 0;
    ++tile;
    if (++row == s.rt) row = 0, ++ent;
    n = (int)min(left, (uint32_t)s.kt);
  }
};

// A place in a ring and the parity of its turn.
struct Slot {
  int i = 0;
  uint32_t turn = 0;
  FP8MOE_DEV void step(int by, int size) {
    i += by;
    if (i >= size) i -= size, turn ^= 1u;
  }
};

// descriptor of a 128x4 scale tile: 32 rows of 16 bytes, no swizzle
FP8MOE_DEV uint64_t sdesc_scales(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
FP8MOE_DEV void cp_scales(uint32_t taddr, uint64_t d) {
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
// One CTA more at a meeting; the (bounded) wait until all have come.  One thread.
// (A CTA whose own wait ran out still comes: the limit is twice that.)
FP8MOE_DEV void come(uint32_t* count) { asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory"); }
FP8MOE_DEV bool came(const uint32_t* count, uint32_t n, int* status, volatile int* abort_flag) {
  if (ld_acquire_gpu(count) >= n) return true;
  const uint64_t t0 = globaltimer();
  while (ld_acquire_gpu(count) < n) {
    if (globaltimer() - t0 > 2 * WAIT_LIMIT_NS) {
      set_status(status, FP8MOE_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// two e4m3 codes -> their values
FP8MOE_DEV float2 e4m3x2_value(uint32_t c) {
  uint32_t h;
  asm("{\n .reg .b16 s;\n cvt.u16.u32 s, %1;\n cvt.rn.f16x2.e4m3x2 %0, s;\n}" : "=r"(h) : "r"(c));
  float2 v;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}" : "=f"(v.x), "=f"(v.y) : "r"(h));
  return v;
}

// Eight neighbouring values of a row, place 8 j in the piece, to NT terms each:
// rows r0 .. of the piece's tile.  Four lanes hold a block.  A block that is not
// finite becomes NaN, and so does its token.
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
    for (int i = 0; i < L.sb; ++i) mbar_init(&b_full[i], 1), mbar_init(&b_empty[i], 1);
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
    if (warp == DC_WARP_TMA) {
      plan_warp(a, pl, lane);
      asm volatile("bar.arrive 3, %0;" ::"n"(DC_THREADS) : "memory");
    } else {
      bar_sync(3, DC_THREADS);
    }
  } else {
    plan_block(a, pl, (int*)(smem + L.b));   // (ends with a block barrier)
  }

  const int K1 = a.H, K2 = a.F, R1 = 2 * a.F, R2 = a.H;
  const int rt1 = (R1 + 127) / 128, kt1 = (K1 + 127) / 128, rt2 = (R2 + 127) / 128, kt2 = (K2 + 127) / 128;
  // ---- weights: a ring fill per piece, of the first product's run and then of
  // the second's; `first` fills leave before the grid meets
  auto produce = [&](uint32_t from, uint32_t upto) {
    Slot slot;
    uint32_t i = 0;
    for (int ph = 0; ph < 2; ++ph) {
      const Stream s(pl.num[1], ph ? rt2 : rt1, ph ? kt2 : kt1, grid);
      const CUtensorMap* tm = ph ? &tm2 : &tm1;
      for (Run r(s, cta); r.left > 0; r.next(s)) {
        if (i >= upto) return i;
        const int e = (int)(pl.ent[r.ent] & 1023u);
        int x = r.k * 128;
        for (int c = 0; c < r.n; ++c, ++i, x += 128, slot.step(1, L.sa)) {
          if (i < from) continue;
          if (i >= upto) return i;
          uint64_t* bar = &a_full[slot.i];
          if (!mbar_wait(&a_empty[slot.i], slot.turn ^ 1u, abort_flag)) {
            fail();
            return i;
          }
          if (a.stall && cta == 0 && i == 0) continue;
          mbar_expect_tx(bar, DC_A_BYTES);
          tma_load_3d(smem + slot.i * DC_A_BYTES, tm, bar, x, r.row * 128, e);
        }
      }
    }
    return i;
  };
  uint32_t issued = 0;
  const bool epi = warp < 4, joins = epi || warp > DC_WARP_B;
  const int jt = epi ? tid : tid - 96;             // thread among those that make terms and add
  // a piece's terms and their scales in the workspace
  auto tile_of = [&](uint32_t ent, int c, int kt, int nt) {
    return a.terms + ((int64_t)(ent >> 10 & 1023u) * kt + (int64_t)c * (int)(ent >> 20)) * nt * 128;
  };
  auto sf_of = [&](int e, int c, int kt) { return a.term_scales + ((int64_t)e * kt + c) * L.sfb_bytes; };
  if (warp == DC_WARP_TMA) {
    if (lane == 0) issued = produce(0, (uint32_t)L.sa);
    __syncwarp();
  } else if (joins) {
    // the first product's terms: sixteen threads a pair's piece
    const int units = pl.num[0] * kt1, step = (int)grid * (DC_JOIN / 16), j = jt & 15;
    for (int u = (jt >> 4) * (int)grid + (int)cta; u - (jt >> 4 & 1) * (int)grid < units; u += step) {
      const bool on = u < units;                    // (a warp has two pieces, and shuffles)
      const int place = on ? u / kt1 : 0, c = on ? u - place * kt1 : 0, k = c * 128 + j * 8;
      const int e = pl.ent_of[place];
      const uint32_t ent = pl.ent[e];
      const bool in = on && k < K1;
      float v[8] = {};
      if (in) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)(pl.order[place] / a.k) * a.ldx + k));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
      }
      put_terms<2>(v, tile_of(ent, c, kt1, 2), sf_of(e, c, kt1), (place - (int)(ent >> 10 & 1023u)) * 2, j, in);
    }
    asm volatile("fence.proxy.async;" ::: "memory");   // bulk copies of other CTAs read them
  }
  // the meetings' counters are zero, the barriers exist, the plan and the first terms are made
  cooperative_groups::this_grid().sync();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  const int nlive = pl.num[0], nent = pl.num[1];
  const Stream s1(nent, rt1, kt1, grid), s2(nent, rt2, kt2, grid);

  if (warp == DC_WARP_TMA) {
    // ======================= weights =======================
    if (lane == 0) {
      issued = produce(issued, UINT32_MAX);
      // no copy stays in flight after a wait that ran out
      if (*abort_flag)
        for (uint32_t i = issued > (uint32_t)L.sa ? issued - L.sa : 0; i < issued; ++i)
          if (!(a.stall && cta == 0 && i == 0)) (void)mbar_wait(&a_full[i % L.sa], (i / (uint32_t)L.sa) & 1u, nullptr);
    }
    __syncwarp();
  } else if (warp == DC_WARP_MMA) {
    // ======================= products =======================
    if (lane == 0) {
      Slot sa, sb, acc;
      const uint64_t ad0 = sdesc_sw128(smem_u32(smem)), bd0 = sdesc_sw128(smem_u32(smem + L.b));
      const uint64_t sfa0 = sdesc_scales(smem_u32(smem + L.sfa)), sfb0 = sdesc_scales(smem_u32(smem + L.sfb));
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Stream& s = ph ? s2 : s1;
        const int tail = ((ph ? K2 : K1) / 32 - 1) % 4 + 1;   // blocks of a row's last piece
        for (Run r(s, cta); r.left > 0 && ok; r.next(s)) {
          const int cols = up16((int)(pl.ent[r.ent] >> 20) * (ph ? 3 : 2));
          const uint32_t id = (uint32_t)(cols >> 3) << 17 | 1u << 23 | 8u << 24, d = tmem + acc.i * DC_ACC;
          if (!mbar_wait(&acc_empty[acc.i], acc.turn ^ 1u, abort_flag)) ok = false;
          uint32_t add = 0;
          for (int c = 0; c < r.n; ++c) {
            if (!ok || !mbar_wait(&a_full[sa.i], sa.turn, abort_flag) || !mbar_wait(&b_full[sb.i], sb.turn, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sf = tmem + DC_SF + sb.i * 12;
            const uint64_t sfb = sfb0 + (uint32_t)(sb.i * L.sfb_bytes >> 4);
            cp_scales(sf, sfa0 + (uint32_t)(sb.i * 32));
            cp_scales(sf + 4, sfb);
            if (cols > 128) cp_scales(sf + 8, sfb + 32);
            const uint64_t ad = ad0 + (uint32_t)(sa.i * (DC_A_BYTES >> 4)), bd = bd0 + (uint32_t)(sb.i * L.b_bytes >> 4);
            auto block = [&](int k, uint32_t plus) {
              mma_mx1(d, ad + 2 * k, bd + 2 * k, id | (uint32_t)k << 4 | (uint32_t)k << 29, sf, sf + 4, plus);
            };
            if (tail == 4 || r.k + c + 1 < s.kt) {
              block(0, add), block(1, 1), block(2, 1), block(3, 1);
            } else {
              block(0, add);
              if (tail > 1) block(1, 1);
              if (tail > 2) block(2, 1);
            }
            add = 1;
            tc_commit(&a_empty[sa.i]);
            tc_commit(&b_empty[sb.i]);
            sa.step(1, L.sa);
            sb.step(1, L.sb);
          }
          if (!ok) break;
          tc_commit(&acc_full[acc.i]);
          acc.step(1, 2);
        }
      }
      if (!ok) fail();
      // every product has completed before tensor memory is given back
      tc_commit(drain);
      if (!mbar_wait(drain, 0, nullptr)) set_status(a.status, FP8MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == DC_WARP_B) {
    // ======================= terms and scales =======================
    if (lane == 0) {
      Slot slot;
      uint32_t i = 0;
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Stream& s = ph ? s2 : s1;
        const int nt = ph ? 3 : 2;
        if (ph == 1 && !came(a.meets + 32, grid, a.status, abort_flag)) break;
        asm volatile("fence.proxy.async;" ::: "memory");
        for (Run r(s, cta); r.left > 0 && ok; r.next(s)) {
          const uint32_t ent = pl.ent[r.ent];
          const int rows = (int)(ent >> 20) * nt;
          const uint32_t bytes = (uint32_t)rows * 128, sfb = rows <= 32 ? (uint32_t)rows * 16 : rows <= 128 ? 512 : 1024;
          const uint8_t* b = tile_of(ent, r.k, s.kt, nt);
          const uint8_t* sb = sf_of(r.ent, r.k, s.kt);
          const uint8_t* sa = (ph ? a.s2 : a.s1) + (((int64_t)(ent & 1023u) * s.rt + r.row) * s.kt + r.k) * 512;
          for (int c = 0; c < r.n; ++c, ++i, b += bytes, sb += L.sfb_bytes, sa += 512, slot.step(1, L.sb)) {
            if (!mbar_wait(&b_empty[slot.i], slot.turn ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            uint64_t* bar = &b_full[slot.i];
            mbar_expect_tx(bar, bytes + sfb + 512);
            bulk_load(smem + L.b + slot.i * L.b_bytes, b, bytes, bar);
            bulk_load(smem + L.sfb + slot.i * L.sfb_bytes, sb, sfb, bar);
            bulk_load(smem + L.sfa + slot.i * 512, sa, 512, bar);
          }
        }
      }
      if (!ok) fail();
      if (*abort_flag)
        for (uint32_t n = i > (uint32_t)L.sb ? i - L.sb : 0; n < i; ++n)
          (void)mbar_wait(&b_full[n % L.sb], (n / (uint32_t)L.sb) & 1u, nullptr);
    }
    __syncwarp();
  } else {
    // ======================= accumulators =======================
    Slot acc;
    auto sums_of = [&](auto phase) {
      constexpr int PH = decltype(phase)::value, NT = PH ? 3 : 2;
      const Stream& s = PH ? s2 : s1;
      const int R = PH ? R2 : R1;
      for (Run r(s, cta); r.left > 0; r.next(s)) {
        const uint32_t ent = pl.ent[r.ent];
        const int first = (int)(ent >> 10 & 1023u), pairs = (int)(ent >> 20);
        const int part = (int)(cta - s.owner(r.tile * s.kt));
        const int row = r.row * 128 + warp * 32 + lane;
        float* dst = a.part + ((int64_t)part * nlive + first) * R + row;
        if (!mbar_wait(&acc_full[acc.i], acc.turn, abort_flag)) {
          fail();
          break;
        }
        tc_fence_after();
        const uint32_t src = tmem + acc.i * DC_ACC + ((uint32_t)(warp * 32) << 16);
        for (int i0 = 0; i0 < pairs; i0 += 8) {
          uint32_t q[24];
#pragma unroll
          for (int c = 0; c < NT; ++c) tmem_ld8(src + i0 * NT + c * 8, *reinterpret_cast<uint32_t(*)[8]>(q + c * 8));
          tmem_ld_wait();
          if (i0 + 8 >= pairs) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc.i]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v = 0.0f;   // the smallest term first
#pragma unroll
            for (int t = NT - 1; t >= 0; --t) v += __uint_as_float(q[i * NT + t]);
            if (i0 + i < pairs && row < R) dst[(int64_t)(i0 + i) * R] = v;
          }
        }
        acc.step(1, 2);
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
    using One = std::integral_constant<int, 0>;
    using Two = std::integral_constant<int, 1>;
    // the accumulating warps come to meeting i and wait for it, with the others
    auto meeting = [&](int i) {
      if (epi) {
        bar_sync(1, 128);
        if (tid == 0) {
          __threadfence();
          come(a.meets + 32 * i);
          (void)came(a.meets + 32 * i, grid, a.status, abort_flag);
        }
      }
      bar_sync(2, DC_JOIN);
    };
    if (epi) sums_of(One{});
    meeting(0);
    // the activation, from the first product's partial sums, and its terms:
    // sixteen threads a pair's piece
    {
      const int units = nlive * kt2, step = (int)grid * (DC_JOIN / 16), j = jt & 15;
      for (int u = (jt >> 4) * (int)grid + (int)cta; u - (jt >> 4 & 1) * (int)grid < units; u += step) {
        const bool on = u < units;
        const int place = on ? u / kt2 : 0, c = on ? u - place * kt2 : 0, f = c * 128 + j * 8;
        const int e = pl.ent_of[place];
        const uint32_t ent = pl.ent[e];
        const bool in = on && f < a.F;
        float v[8] = {};
        if (in) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 g = gather(s1, R1, place, e, f + 4 * h), y = gather(s1, R1, place, e, a.F + f + 4 * h);
            v[4 * h] = g.x / (1.0f + expf(-g.x)) * y.x;
            v[4 * h + 1] = g.y / (1.0f + expf(-g.y)) * y.y;
            v[4 * h + 2] = g.z / (1.0f + expf(-g.z)) * y.z;
            v[4 * h + 3] = g.w / (1.0f + expf(-g.w)) * y.w;
          }
        }
        put_terms<3>(v, tile_of(ent, c, kt2, 3), sf_of(e, c, kt2), (place - (int)(ent >> 10 & 1023u)) * 3, j, in);
      }
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    bar_sync(2, DC_JOIN);
    if (tid == 0) {
      __threadfence();
      come(a.meets + 32);
    }
    if (epi) sums_of(Two{});
    meeting(2);
    // the weighted sum over a token's experts, four neighbouring columns a thread,
    // runs of eight threads' a CTA in turn
    {
      const uint32_t per = (uint32_t)a.H / 4, tasks = (uint32_t)a.T * per;
      for (uint32_t i = (((uint32_t)jt >> 3) * grid + cta) * 8 + (jt & 7); i < tasks; i += DC_JOIN * grid) {
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

// bytes of the scales of a piece's terms
constexpr int term_scale_bytes(int P) { return 3 * (P < DC_NB ? P : DC_NB) > 128 ? 1024 : 512; }

DecodeSmem layout(int P, int max_ent, int max_smem) {
  DecodeSmem L{};
  const int nb = P < DC_NB ? P : DC_NB;
  L.b_bytes = (up16(3 * nb) * 128 + 1023) / 1024 * 1024;
  L.sfb_bytes = term_scale_bytes(P);
  L.sb = nb <= 8 ? 8 : nb <= 16 ? 6 : nb <= 32 ? 4 : 3;
  const int plan = 16 + max_ent * 4 + P * 10;
  const int bars = 8 * (2 * 16 + 2 * DC_MAX_BS + 8);
  const int fixed = L.sb * (L.b_bytes + L.sfb_bytes + 512) + bars + plan + 64;
  L.sa = (max_smem - 2048 - fixed) / DC_A_BYTES;   // 1024 to align the rings, 1024 for what is static
  if (L.sa > 13) L.sa = 13;
  L.b = L.sa * DC_A_BYTES;
  L.sfa = L.b + L.sb * L.b_bytes;
  L.sfb = L.sfa + L.sb * 512;
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

// What the workspace holds behind the counters: partial sums, terms, their
// scales.  Both products' in turn in the same place.
struct DecodeSpace {
  int64_t parts, terms, scales;   // bytes
};
static DecodeSpace space_of(int64_t P, int64_t E, int64_t H, int64_t F) {
  const int64_t p1 = part_floats(P, 2 * F, H), p2 = part_floats(P, H, F);
  const int64_t kh = (H + 127) / 128, kf = (F + 127) / 128;
  return {(p1 > p2 ? p1 : p2) * (int64_t)sizeof(float), P * 128 * (2 * kh > 3 * kf ? 2 * kh : 3 * kf),
          max_entries(P, E) * (kh > kf ? kh : kf) * term_scale_bytes((int)P)};
}

int64_t decode_workspace_bytes(int64_t P, int64_t E, int64_t H, int64_t F) {
  const DecodeSpace w = space_of(P, E, H, F);
  return DECODE_MEETS_BYTES + w.parts + w.terms + w.scales;
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
  const DecodeSpace w = space_of(a.P, a.E, a.H, a.F);
  a.meets = (uint32_t*)workspace;
  a.part = (float*)((uint8_t*)workspace + DECODE_MEETS_BYTES);
  a.terms = (uint8_t*)a.part + w.parts;
  a.term_scales = a.terms + w.terms;
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
