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
// The tokens keep their digits.  In a block of 32 values scaled so that the
// largest lies in [128, 256), the nearest e4m3 value leaves a rest of at most 8,
// which times 2^5 is again such a block, with its own scale: a term has five bits
// of a value, down to a last place of 2^-9.  Two hold a bf16 value exactly from 2^-14 of its
// block's largest on, and what is smaller to 2^-22 of that largest; four hold an fp32
// value to 2^-19 of itself, or 2^-32 of the largest.  (With three, to 2^-14, one of a
// hundred outputs was the neighbour of the bf16 number that it should be; with four one
// of a thousand, as with five, and half of that with the sums in chains, see Stream.)
// The terms are further columns of N, where the tensor core has room: N is at least
// 16, and the weights' arrival leaves it idle most of the time.
//
// Both products are one stream of 32 KB pieces (128 rows x 256 of K) over all
// (expert, row tile, k) in order, cut into equal runs, one per CTA; a tile's
// partial sums (fp32, at most a few per tile) go to the workspace and are added
// in order after a grid-wide meeting.  The terms of x and of the activation are
// made once, into the workspace, as the tensor core reads them, and copied to a
// ring beside the weights'; through registers, as bulk copies queue behind the
// weights' in flight.  Where an expert has few pairs, every CTA makes the terms of its
// own run on the way to the ring instead, from x and from the first product's partial
// sums, which saves two of the four meetings.  The weights' producer takes no part
// in the meetings: while the others add, it fills its ring with W2.
// Measured in a graph: one token of 6 of 64 experts of 1408 x 2048 19 us (8 of bytes, the rest
// the way through two products: 10.5 for a layer of almost no weights), of 8 of 256 of 2048 x
// 7168 66 us = 5.5 TB/s, 23 such 892 us = 6.7 TB/s; 64 of one of 16 of 8192 x 5120 330 us = 6.3 TB/s.
//   warps 0-3  accumulators to partial sums;  4  weights by TMA;  5  MMA issue;
//   6  scales to tensor memory;  7-14  terms to shared memory;  all but 4-6  terms
//   and the final sums.
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "moe_ops.h"
#include "swiglu.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace fp8moe {
namespace {

constexpr int DC_THREADS = 480;
constexpr int DC_WARP_TMA = 4, DC_WARP_MMA = 5, DC_WARP_SF = 6, DC_WARP_B = 7;
constexpr int DC_BWARPS = DC_THREADS / 32 - DC_WARP_B;
constexpr int DC_JOIN = DC_THREADS - 96;  // threads that make terms and add partial sums: all but warps 4-6's
constexpr int DC_G = 2;                   // tiles of 128 x 128 in a piece
constexpr int DC_TILE = 128 * 128, DC_A_BYTES = DC_G * DC_TILE;
constexpr int DC_MAX_SLOTS = 6;
constexpr int X_TERMS = 2, ACT_TERMS = 4;   // of a value of x, of the activation
constexpr int DC_DEAD = 0xFFFF;

__host__ __device__ constexpr int up16(int v) { return (v + 15) / 16 * 16; }

// Division by a number that the host knows.
struct Div {
  uint32_t d, m;   // m: 2^32 / d, rounded down (and below 2^32)
  __host__ __device__ Div() : d(1), m(0xFFFFFFFFu) {}
  explicit Div(int64_t by) : d((uint32_t)by), m(by > 1 ? (uint32_t)(((int64_t)1 << 32) / by) : 0xFFFFFFFFu) {}
  FP8MOE_DEV uint32_t quot(uint32_t n) const {
    const uint32_t q = __umulhi(n, m);   // the quotient or one less
    return n - q * d >= d ? q + 1 : q;
  }
};

// Shared memory: the rings of weights (at 0), of their scales, of terms and their
// scales (a piece has the same slot in all), the plan.
struct DecodeSmem {
  int slots, b_bytes;
  int team_log, teams;                     // 2^team_log warps fill a slot of terms together
  int acc, accs;                           // tensor memory columns of an accumulator; accumulators
  int chain;                               // pieces that are added in one
  int sfa, b, bars, plan, total;
  // tiles and pieces of the products' K, tiles of their rows; the grid; H / 4; choices
  Div kt[2], kp[2], rt[2], grid, quads, k;
};

// The terms of an entry of n pairs, piece by piece: DC_G tiles of their rows,
// rounded up to 8, then the tiles' scales (of up to 32 rows that is the first part
// of a 128x4 tile).
struct TermTiles {
  int rows, sf;   // rows of a tile; bytes of its scales
  __host__ __device__ constexpr TermTiles(int terms) : rows((terms + 7) / 8 * 8), sf(rows <= 32 ? rows * 16 : rows <= 128 ? 512 : 1024) {}
  __host__ __device__ constexpr int bytes() const { return DC_G * (rows * 128 + sf); }
};

// The plan of a call, in shared memory: the live pairs (token, choice) in the
// order of their experts, cut into entries of one expert and at most nb pairs.
struct Plan {
  uint32_t* ent;      // expert | first pair << 10 | pairs << 20
  float* w;           // [P] weights of the pairs
  uint16_t* order;    // [live] pair of each place
  uint16_t* pos;      // [P] place of each pair, or DC_DEAD
  uint16_t* ent_of;   // [live] entry of each place
  int* num;           // live pairs, entries, the largest entry's pairs
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
  const bool head = live && before % a.nb == 0;
  const uint32_t heads = __ballot_sync(0xffffffffu, head);
  int ent = before / a.nb;
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
    if (head) pl.ent[ent] = (uint32_t)e | (uint32_t)rank << 10 | (uint32_t)min(a.nb, same - before) << 20;
  }
  const int n = __popc(__ballot_sync(0xffffffffu, live));
  const uint32_t most = __reduce_max_sync(0xffffffffu, live ? (uint32_t)min(a.nb, same) : 0u);
  if (lane == 0) pl.num[0] = n, pl.num[1] = __popc(heads), pl.num[2] = (int)most;
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
    const uint32_t own = (uint32_t)n << 16 | (uint32_t)((n + a.nb - 1) / a.nb);
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
    if (lane == 31) pl.num[0] = (int)(v >> 16), pl.num[1] = (int)(v & 0xFFFFu), pl.num[2] = 0;
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
    const int place = (int)(base >> 16) + before, ent = (int)(base & 0xFFFFu) + before / a.nb;
    pl.order[place] = (uint16_t)p;
    pl.pos[p] = (uint16_t)place;
    pl.ent_of[place] = (uint16_t)ent;
    if (before % a.nb == 0) {
      for (int q = p; q < a.P && after < a.nb; ++q) after += ids[q] == e;
      pl.ent[ent] = (uint32_t)e | (uint32_t)place << 10 | (uint32_t)after << 20;
      atomicMax(pl.num + 2, after);
    }
  }
  __syncthreads();
}

FP8MOE_DEV float reciprocal(float x) {   // to 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One product's stream of pieces: nent entries x row tiles x pieces of K, in runs
// of `base` pieces, one more for the first `rest` CTAs.  At most `chain` pieces in a row
// are added in an accumulator, as the tensor core's sums are cut off, not rounded.
struct Stream {
  uint32_t C, runs, base, rest;   // pieces; CTAs that have a run of them
  float per0, per1;               // 1 / base, 1 / (base + 1)
  const Div &rt, &kp;
  const int& chain;
  FP8MOE_DEV Stream(int nent, const Div& rt_, const Div& kp_, const Div& grid, const int& chain_)
      : rt(rt_), kp(kp_), chain(chain_) {
    static_assert(DECODE_MIN_RUN == 2, "base of a short stream");
    C = (uint32_t)nent * rt.d * kp.d;
    const uint32_t want = (C + 1) / 2;
    runs = want < grid.d ? want : grid.d;
    base = want < grid.d ? (C == 2 * runs ? 2 : 1) : grid.quot(C);
    rest = C - base * runs;
    per0 = reciprocal((float)base);
    per1 = reciprocal((float)(base + 1));
  }
  FP8MOE_DEV uint32_t first(uint32_t cta) const { return cta < runs ? cta * base + min(cta, rest) : C; }
  // the CTA whose run has piece c: below 2^8, so that the quotient in fp32 is off by
  // one at most
  FP8MOE_DEV uint32_t owner(uint32_t c) const {
    const uint32_t wide = rest * (base + 1);
    const bool late = c >= wide;
    const uint32_t n = late ? c - wide : c, d = late ? base : base + 1;
    uint32_t q = (uint32_t)((float)n * (late ? per0 : per1));
    if (q * d > n) --q;
    if (n - q * d >= d) ++q;
    return late ? q + rest : q;
  }
  // partial sums of a tile: the CTAs whose runs meet it
  FP8MOE_DEV int parts(uint32_t tile) const { return (int)(owner(tile * kp.d + kp.d - 1) - owner(tile * kp.d)) + 1; }
};

// A CTA's run of a stream, segment by segment: the pieces of one tile that are
// in the run, a chain of them at a time.
struct Run {
  uint32_t left, tile;   // pieces to go, this segment's among them; row tile over all entries
  int n, k;              // pieces of this segment, the first one's place along K
  int ent, row;
  FP8MOE_DEV Run(const Stream& s, uint32_t cta) {
    const uint32_t lo = s.first(cta);
    left = s.first(cta + 1) - lo;
    tile = s.kp.quot(lo);
    k = (int)(lo - tile * s.kp.d);
    ent = (int)s.rt.quot(tile);
    row = (int)(tile - (uint32_t)ent * s.rt.d);
    n = segment(s);
  }
  FP8MOE_DEV int segment(const Stream& s) const { return min(min((int)left, (int)s.kp.d - k), s.chain); }
  FP8MOE_DEV void next(const Stream& s) {
    left -= n;
    k += n;
    if (k == (int)s.kp.d) {
      k = 0;
      ++tile;
      if (++row == (int)s.rt.d) row = 0, ++ent;
    }
    n = segment(s);
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

// True in one lane of a converged warp, which the compiler then knows to be alone: its
// descriptors need no loop over lanes (a copy of scales 10 cycles to issue, 50 with
// lane == 0).
FP8MOE_DEV bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

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
FP8MOE_DEV void prefetch_tmap(const CUtensorMap* m) { asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory"); }
FP8MOE_DEV void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// Grid-wide meetings: a counter each, to which every CTA of a launch adds one.
// They are the library's own, per device, as no caller's memory starts at zero: a
// CTA fills an SM's shared memory and the grid all SMs, so that no two launches
// run at a time, and each leaves its counters one grid further.  (A CTA that gives
// up still comes.)
enum { MEET_X = 0, MEET_SUMS, MEET_ACT, MEET_END, DC_MEETS };
__device__ unsigned long long g_meets[2][DC_MEETS][16];   // of calls with four meetings, and with two
FP8MOE_DEV uint64_t ld_acquire_gpu(const unsigned long long* p) {
  uint64_t v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
// One thread comes for its CTA, which is at a barrier, and waits until the counter
// says n: all have come.  (With twice the limit of the waits before it.)
FP8MOE_DEV void come(unsigned long long* count) {
  asm volatile("red.release.gpu.global.add.u64 [%0], 1;" ::"l"(count) : "memory");
}
FP8MOE_DEV void came(unsigned long long* count, uint64_t n, int* status, volatile int* abort_flag) {
  if (ld_acquire_gpu(count) >= n) return;
  const uint64_t t0 = globaltimer();
  while (ld_acquire_gpu(count) < n) {
    if (globaltimer() - t0 > 2 * WAIT_LIMIT_NS) {
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

// silu(g) u of two sums each.  Below -80 the sigmoid is that of -80 times e^(g + 80), as
// two factors of half the exponent: they and every product on the way are normal as
// long as the result can differ from 0 (|u| < 2^128: down to g = -195, where the rounded
// exponents leave 2^-15 of it), and no product is beyond fp32 that the result is not
// (-300 stands for every gate below).  (Packed and without branches: eight divisions and
// expf in a row took 1.5 us of a token's way, most of it to fetch their instructions.)
FP8MOE_DEV void act_of_sums(const float* g, const float* u, float* v) {
  auto near = [](float x) { return fminf(fmaxf(x, -80.0f), 80.0f); };
  auto half = [](float x) {   // e^((x + 80) / 2), at most 1
    float h;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(fminf(x + 80.0f, 0.0f) * 0.72134752f));
    return h;
  };
  const uint64_t f = pk(half(g[0]), half(g[1]));
  const uint64_t s = mul2(pk(nanmax(g[0], -300.0f), nanmax(g[1], -300.0f)), sigmoid2(pk(near(g[0]), near(g[1]))));
  unpk(mul2(mul2(mul2(s, pk(u[0], u[1])), f), f), v[0], v[1]);
}

// NT terms of eight neighbouring values of a row, four lanes a block: codes, and
// the byte of the first term's scale (each further one's is 5 less).  A block that
// is not finite becomes NaN, and so does its token.
template <int NT>
struct Terms {
  uint2 q[NT];
  uint32_t byte;
  bool finite;
  FP8MOE_DEV explicit Terms(float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, m, o);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(u));
    }
    const uint32_t field = (__float_as_uint(m) >> 23) & 0xFFu;
    // (the smallest blocks are not scaled all the way up: the last term's byte is not below 0)
    constexpr uint32_t LEAST = 7 + 5 * (NT - 1);
    const uint32_t ef = field < LEAST ? LEAST : field;
    finite = field != 255u;
    byte = ef - 7u;
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
      q[t] = finite ? make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
  }
  // to rows r0 .. of a tile, place 8 j in it: 128-byte swizzle; scales in 128x4 order
  FP8MOE_DEV void put(uint8_t* tile, uint8_t* sf, int r0, int j) const {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = r0 + t;
      *reinterpret_cast<uint2*>(tile + r * 128 + (((j >> 1) ^ (r & 7)) << 4) + (j & 1) * 8) = q[t];
      if ((j & 3) == 0)
        sf[(r >> 7) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j >> 2)] = (uint8_t)(finite ? byte - 5u * t : 127u);
    }
  }
};

// What the host knows of a call: nothing (the plan decides how terms are made), that
// entries have few pairs (made on the way), that they have at most two.  (One token of 6 of
// 64 experts of 1408 x 2048: 20.4 us if the plan decides, 19.5 as one of few, 19.3.)
enum { DC_ANY = 0, DC_FEW, DC_TWO };
template <int FORM>
__global__ void __launch_bounds__(DC_THREADS, 1)
    k_decode(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2, DecodeArgs a, DecodeSmem L) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ int abort_s;
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t cta = blockIdx.x, grid = gridDim.x;
  volatile int* abort_flag = &abort_s;
  uint64_t* a_full = (uint64_t*)(smem + L.bars);
  uint64_t* b_full = a_full + L.slots;
  uint64_t* sf_full = b_full + L.slots;
  uint64_t* empty = sf_full + L.slots;
  uint64_t* acc_full = empty + L.slots;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;   // the issuer's, the copier's
  const Plan pl(smem + L.plan, a.P, a.max_ent);
  auto fail = [&]() {
    set_status(a.status, FP8MOE_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == DC_WARP_TMA && lane == 0) {
    prefetch_tmap(&tm1);
    prefetch_tmap(&tm2);
  }
  if (warp == DC_WARP_MMA) {
    if (lane == 0) abort_s = 0;
    if (lane < L.slots)
      mbar_init(&a_full[lane], 1), mbar_init(&b_full[lane], 1 << L.team_log), mbar_init(&sf_full[lane], 1), mbar_init(&empty[lane], 1);
    if (lane < 2) mbar_init(&acc_full[lane], 1), mbar_init(&acc_empty[lane], 4), mbar_init(&drain[lane], 1);
    mbar_fence_init();
  }
  if (warp == DC_WARP_SF) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_s)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  const int K1 = a.H, K2 = a.F, R1 = 2 * a.F, R2 = a.H;
  const int kt1 = (int)L.kt[0].d, kt2 = (int)L.kt[1].d;
  const bool epi = warp < 4;
  const int jt = epi ? tid : tid - 96;             // thread among those that make terms and add
  // The terms' units: a pair's tile, sixteen threads each, a warp's two a grid apart.
  const int unit0 = (jt >> 4) * (int)grid + (int)cta, unit_step = (int)grid * (DC_JOIN / 16), j16 = jt & 15;
  auto x_at = [&](int u) {                         // this thread's eight values of x
    const int p = (int)L.kt[0].quot(u), k = (u - p * kt1) * 128 + j16 * 8;
    return u < a.P * kt1 && k < K1 ? __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)L.k.quot(p) * a.ldx + k))
                                   : make_uint4(0, 0, 0, 0);
  };
  uint4 x0 = make_uint4(0, 0, 0, 0);               // the first unit's, on its way while the plan is made
  if (FORM == DC_ANY && (warp < DC_WARP_TMA || warp >= DC_WARP_B)) x0 = x_at(unit0);
  if (a.P <= 32) {
    if (warp == DC_WARP_TMA) plan_warp(a, pl, lane);
    __syncthreads();
  } else {
    plan_block(a, pl, (int*)(smem + L.b));   // (ends with a block barrier)
  }
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  const int nlive = pl.num[0], nent = pl.num[1];
  // Terms made on the way where entries have few pairs: no more than 8, as a warp of a
  // team takes two at a time and must not be slower than the weights, and 1.2 on average.
  // (In a graph, made and copied: 12 tokens of 2 of 256 experts of 1408 x 2048 (1.05 pairs
  // an entry) 45 us and 47, 23 of 3 of 256 of 2048 x 7168 (1.13) 413 and 417; 16 of 6 of 160 of
  // 1024 x 4096 (1.3) 157 and 156, 23 of 8 of 256 of 2048 x 7168 (1.4) 902 and 893.  With
  // cold caches the copies are 0 to 2 us better with the first two, 5 and 15 with the others.)
  const bool direct = FORM != DC_ANY || (L.team_log == 1 && pl.num[2] <= 8 && 5 * nlive <= 6 * nent);
  const Stream s1(nent, L.rt[0], L.kp[0], L.grid, L.chain), s2(nent, L.rt[1], L.kp[1], L.grid, L.chain);
  using First = std::integral_constant<int, X_TERMS>;      // the products, by their terms
  using Second = std::integral_constant<int, ACT_TERMS>;

  if (warp == DC_WARP_TMA) {
    // ======================= weights =======================
    // The first fills leave behind this CTA's terms of x: in front of them, what
    // follows them meets its first instructions and loads in a full memory system.
    if (!direct) bar_sync(1, DC_JOIN + 32);
    if (elected()) {
      Slot slot;
      uint32_t i = 0;
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Stream& s = ph ? s2 : s1;
        const CUtensorMap* tm = ph ? &tm2 : &tm1;
        const int kt = ph ? kt2 : kt1;
        for (Run r(s, cta); r.left > 0 && ok; r.next(s)) {
          const int e = (int)(pl.ent[r.ent] & 1023u);
          int x = r.k * DC_G;   // the piece's first tile
          const uint8_t* sc = (ph ? a.s2 : a.s1) + (((int64_t)e * s.rt.d + r.row) * kt + x) * 512;
          for (int c = 0; c < r.n; ++c, ++i, x += DC_G, sc += DC_G * 512, slot.step(1, L.slots)) {
            uint64_t* bar = &a_full[slot.i];
            if (!mbar_wait(&empty[slot.i], slot.turn ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            if (a.stall && cta == 0 && i == 0) continue;
            const int tiles = min(DC_G, kt - x);
            uint8_t* dst = smem + slot.i * DC_A_BYTES;
            mbar_expect_tx(bar, tiles * (DC_TILE + 512));
#pragma unroll
            for (int g = 0; g < DC_G; ++g)
              if (g < tiles) tma_load_3d(dst + g * DC_TILE, tm, bar, (x + g) * 128, r.row * 128, e);
            bulk_load(smem + L.sfa + slot.i * DC_G * 512, sc, tiles * 512, bar);
          }
        }
      }
      if (!ok) fail();
      // no copy stays in flight after a wait that ran out
      if (*abort_flag)
        for (uint32_t n = i > (uint32_t)L.slots ? i - L.slots : 0; n < i; ++n)
          if (!(a.stall && cta == 0 && n == 0)) (void)mbar_wait(&a_full[n % L.slots], (n / (uint32_t)L.slots) & 1u, nullptr);
    }
    __syncwarp();
  } else if (warp == DC_WARP_MMA) {
    // ======================= products =======================
    if (elected()) {
      Slot slot, acc;
      const uint64_t ad0 = sdesc_sw128(smem_u32(smem)), bd0 = sdesc_sw128(smem_u32(smem + L.b));
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Stream& s = ph ? s2 : s1;
        const int kt = ph ? kt2 : kt1;
        const int tail = ((ph ? K2 : K1) / 32 - 1) % 4 + 1;   // blocks of a row's last tile
        for (Run r(s, cta); r.left > 0 && ok; r.next(s)) {
          const TermTiles tt((int)(pl.ent[r.ent] >> 20) * (ph ? ACT_TERMS : X_TERMS));
          const int cols = up16(tt.rows);
          const uint32_t id = (uint32_t)(cols >> 3) << 17 | 1u << 23 | 8u << 24, d = tmem + acc.i * L.acc;
          if (!mbar_wait(&acc_empty[acc.i], acc.turn ^ 1u, abort_flag)) ok = false;
          uint32_t add = 0;
          for (int c = 0; c < r.n; ++c) {
            if (!ok || !mbar_wait(&a_full[slot.i], slot.turn, abort_flag) || !mbar_wait(&b_full[slot.i], slot.turn, abort_flag) ||
                !mbar_wait(&sf_full[slot.i], slot.turn, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t at_b = (uint32_t)(slot.i * L.b_bytes);
#pragma unroll
            for (int g = 0; g < DC_G; ++g) {
              const int left = kt - (r.k + c) * DC_G - g;   // tiles of the row from this one on
              if (left <= 0) break;
              const uint32_t sf = tmem + L.accs * L.acc + (slot.i * DC_G + g) * 12;
              const uint64_t ad = ad0 + ((uint32_t)(slot.i * DC_A_BYTES + g * DC_TILE) >> 4);
              const uint64_t bd = bd0 + ((at_b + (uint32_t)(g * tt.rows * 128)) >> 4);
              auto block = [&](int k, uint32_t plus) {
                mma_mx1(d, ad + 2 * k, bd + 2 * k, id | (uint32_t)k << 4 | (uint32_t)k << 29, sf, sf + 4, plus);
              };
              if (tail == 4 || left > 1) {
                block(0, add), block(1, 1), block(2, 1), block(3, 1);
              } else {
                block(0, add);
                if (tail > 1) block(1, 1);
                if (tail > 2) block(2, 1);
              }
              add = 1;
            }
            tc_commit(&empty[slot.i]);   // (once a piece: a commit holds its thread up for as long as seven products)
            slot.step(1, L.slots);
          }
          if (!ok) break;
          tc_commit(&acc_full[acc.i]);
          acc.step(1, L.accs);
        }
      }
      if (!ok) fail();
      // every product has completed before tensor memory is given back
      tc_commit(&drain[0]);
      if (!mbar_wait(&drain[0], 0, nullptr)) set_status(a.status, FP8MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == DC_WARP_SF) {
    // ======================= scales to tensor memory =======================
    // From a thread of their own the copies overlap the products.  A slot's columns
    // are free when its terms are new: the products of its last turn are over.
    if (elected()) {
      Slot slot;
      const uint64_t sfa0 = sdesc_scales(smem_u32(smem + L.sfa)), sfb0 = sdesc_scales(smem_u32(smem + L.b));
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Stream& s = ph ? s2 : s1;
        const int kt = ph ? kt2 : kt1;
        for (Run r(s, cta); r.left > 0 && ok; r.next(s)) {
          const TermTiles tt((int)(pl.ent[r.ent] >> 20) * (ph ? ACT_TERMS : X_TERMS));
          for (int c = 0; c < r.n; ++c) {
            if (!mbar_wait(&a_full[slot.i], slot.turn, abort_flag) || !mbar_wait(&b_full[slot.i], slot.turn, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < DC_G; ++g) {
              if ((r.k + c) * DC_G + g >= kt) break;
              const uint32_t sf = tmem + L.accs * L.acc + (slot.i * DC_G + g) * 12;
              const uint64_t sfb = sfb0 + ((uint32_t)(slot.i * L.b_bytes + DC_G * tt.rows * 128 + g * tt.sf) >> 4);
              cp_scales(sf, sfa0 + (uint32_t)((slot.i * DC_G + g) * 32));
              cp_scales(sf + 4, sfb);
              if (tt.rows > 128) cp_scales(sf + 8, sfb + 32);
            }
            tc_commit(&sf_full[slot.i]);
            slot.step(1, L.slots);
          }
        }
      }
      if (!ok) fail();
      tc_commit(&drain[1]);
      if (!mbar_wait(&drain[1], 0, nullptr)) set_status(a.status, FP8MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    // every meeting's count when all have come: the last one's stands still until
    // this CTA has been at the others
    uint64_t meets;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(meets) : "l"(g_meets[direct][MEET_END]));
    meets += grid;
    // (`meanwhile`: what the next step can work out without the others' results)
    auto meeting = [&](int i, auto meanwhile) {
      bar_sync(2, DC_JOIN);
      if (tid == 0) come(g_meets[direct][i]);
      meanwhile();
      if (tid == 0) came(g_meets[direct][i], meets, a.status, abort_flag);
      bar_sync(2, DC_JOIN);
    };

    // Partial sums in order, of four neighbouring rows each; N in flight together.
    struct Parts {
      const float4* p;
      int n;
    };
    auto parts_of = [&](const Stream& s, const float* part, int R, int place, int row) {
      const uint32_t tile = (uint32_t)pl.ent_of[place] * s.rt.d + row / 128;
      return Parts{reinterpret_cast<const float4*>(part + (int64_t)place * R + row), s.parts(tile)};
    };
    auto gather = [&](int R, const auto& src, auto& v) {
      constexpr int N = std::extent_v<std::remove_reference_t<decltype(v)>>;
      const int64_t step = (int64_t)nlive * R / 4;
      int most = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = src[i].n > 0 ? __ldcg(src[i].p) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        most = max(most, src[i].n);
      }
      for (int q = 1; q < most; ++q) {
        float4 u[N];
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = q < src[i].n ? __ldcg(src[i].p + q * step) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i].x += u[i].x, v[i].y += u[i].y, v[i].z += u[i].z, v[i].w += u[i].w;
      }
    };
    // where an entry's terms are in the workspace
    auto terms_of = [&](int e, uint32_t ent, int kp, int nt) {
      return a.terms + (int64_t)kp * DC_G * ((nt * (int)(ent >> 10 & 1023u) + 7 * e) * 128 + 1024 * e);
    };

    // ======================= terms into shared memory =======================
    // Teams of warps take the pieces of both runs in turn.  (Not more teams than
    // slots: a slot's barrier tells the last turn from the one before, and a team
    // that has filled its last piece knows that the slots' turns before are over.)
    const int team = (warp - DC_WARP_B) >> L.team_log, rank = (warp - DC_WARP_B) & ((1 << L.team_log) - 1);
    Slot slot;
    slot.step(team, L.slots);
    Run r(s1, cta);                           // of the stream to come, at the team's next piece
    int c = team;                                    // this, counted in r's segment
    auto enter = [&](const Stream& s) {
      while (r.left > 0 && c >= r.n) {
        c -= r.n;
        r.next(s);
      }
    };
    if (!epi) enter(s1);
    auto feed = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      const Stream& s = NT == X_TERMS ? s1 : s2;
      for (; team < L.teams && r.left > 0; c += L.teams, slot.step(L.teams, L.slots), enter(s)) {
        const uint32_t ent = pl.ent[r.ent];
        const TermTiles tt((int)(ent >> 20) * NT);
        uint4* dst = reinterpret_cast<uint4*>(smem + L.b + slot.i * L.b_bytes);
        const uint4* src = reinterpret_cast<const uint4*>(terms_of(r.ent, ent, s.kp.d, NT) + (int64_t)(r.k + c) * tt.bytes());
        // 16 bytes at a time, 4 KB in flight a warp
        const int chunks = tt.bytes() / 16, at = rank * 32 + lane, step = 32 << L.team_log;
        bool ready = false, ok = true;
        for (int i0 = at; i0 - lane < chunks; i0 += 8 * step) {
          uint4 q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i0 + step * i < chunks) q[i] = __ldcg(src + i0 + step * i);
          if (!ready) ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot.i], slot.turn ^ 1u, abort_flag));
          ready = true;
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i0 + step * i < chunks) dst[i0 + step * i] = q[i];
        }
        if (!ok) {
          fail();
          break;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_full[slot.i]);
      }
      // c is past the run's end: into the next run
    };
    // The same, made here: a warp a tile, two pairs at a time, half a warp each, the next
    // two's values on their way meanwhile.
    auto make = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      const Stream& s = NT == X_TERMS ? s1 : s2;
      const int K = NT == X_TERMS ? K1 : K2, half = lane >> 4;
      int pair = 0;         // r and c's piece: the first of the two
      struct Values {
        uint32_t ent;
        int pair;
        bool in;
        uint4 x;            // of x; or the first two partial sums of gate and up
        float4 q[NT == X_TERMS ? 1 : 4], u[NT == X_TERMS ? 1 : 4];
        Parts g, y;
      } next;
      auto fetch = [&]() {
        next.ent = pl.ent[r.ent];
        next.pair = pair + half;
        const int place = (int)(next.ent >> 10 & 1023u) + next.pair, k = ((r.k + c) * DC_G + rank) * 128 + j16 * 8;
        next.in = next.pair < (int)(next.ent >> 20) && k < K;
        if constexpr (NT == X_TERMS) {
          next.x = make_uint4(0, 0, 0, 0);
          if (next.in)
            next.x = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)L.k.quot(pl.order[place]) * a.ldx + k));
        } else {
          const int64_t step = (int64_t)nlive * R1 / 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) next.q[i] = next.u[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (next.in) {
            next.g = parts_of(s1, a.part1, R1, place, k), next.y = parts_of(s1, a.part1, R1, place, a.F + k);
#pragma unroll
            for (int i = 0; i < 2; ++i) next.q[i] = __ldcg(next.g.p + i), next.q[2 + i] = __ldcg(next.y.p + i);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (next.g.n > 1) next.u[i] = __ldcg(next.g.p + step + i);
              if (next.y.n > 1) next.u[2 + i] = __ldcg(next.y.p + step + i);
            }
          }
        }
      };
      bool more = team < L.teams && r.left > 0;
      if (more) fetch();
      while (more) {
        const Values now = next;
        const int pairs = (int)(now.ent >> 20);
        pair += 2;
        if (FORM == DC_TWO || pair >= pairs) {
          pair = 0;
          c += L.teams;
          enter(s);
        }
        more = r.left > 0;
        if (more) fetch();
        float v[8];
        if constexpr (NT == X_TERMS) {
          const uint32_t w[4] = {now.x.x, now.x.y, now.x.z, now.x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
        } else {
          float4 z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            z[i] = make_float4(now.q[i].x + now.u[i].x, now.q[i].y + now.u[i].y, now.q[i].z + now.u[i].z, now.q[i].w + now.u[i].w);
          if (now.in) {
            const int64_t step = (int64_t)nlive * R1 / 4;
            auto more = [&](const Parts& p, float4& z0, float4& z1) {
              for (int i = 2; i < p.n; ++i) {
                const float4 e = __ldcg(p.p + i * step), f = __ldcg(p.p + i * step + 1);
                z0.x += e.x, z0.y += e.y, z0.z += e.z, z0.w += e.w;
                z1.x += f.x, z1.y += f.y, z1.z += f.z, z1.w += f.w;
              }
            };
            more(now.g, z[0], z[1]);
            more(now.y, z[2], z[3]);
          }
          const float gs[8] = {z[0].x, z[0].y, z[0].z, z[0].w, z[1].x, z[1].y, z[1].z, z[1].w};
          const float us[8] = {z[2].x, z[2].y, z[2].z, z[2].w, z[3].x, z[3].y, z[3].z, z[3].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) act_of_sums(gs + 2 * i, us + 2 * i, v + 2 * i);
        }
        __syncwarp();
        const Terms<NT> terms(v);
        if ((FORM == DC_TWO || now.pair == half) && !__all_sync(0xffffffffu, mbar_wait(&empty[slot.i], slot.turn ^ 1u, abort_flag))) {
          fail();
          break;
        }
        const TermTiles tt(pairs * NT);
        uint8_t* dst = smem + L.b + slot.i * L.b_bytes;
        if (now.in) terms.put(dst + rank * tt.rows * 128, dst + DC_G * tt.rows * 128 + rank * tt.sf, now.pair * NT, j16);
        if (FORM != DC_TWO && now.pair - half + 2 < pairs) continue;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_full[slot.i]);
        slot.step(L.teams, L.slots);
      }
    };
    // ======================= accumulators to partial sums =======================
    Slot acc;
    auto drain_acc = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      const Stream& s = NT == X_TERMS ? s1 : s2;
      const int R = NT == X_TERMS ? R1 : R2;
      float* part = NT == X_TERMS ? a.part1 : a.part2;
      uint32_t before = 0xFFFFFFFFu;               // the tile of the segment before
      for (Run r(s, cta); r.left > 0; r.next(s)) {
        const uint32_t ent = pl.ent[r.ent];
        const bool again = r.tile == before;       // added to what this thread has written
        before = r.tile;
        const int first = (int)(ent >> 10 & 1023u), pairs = (int)(ent >> 20);
        const int mine = (int)(cta - s.owner(r.tile * s.kp.d));
        const int row = r.row * 128 + warp * 32 + lane;
        float* dst = part + ((int64_t)mine * nlive + first) * R + row;
        if (!mbar_wait(&acc_full[acc.i], acc.turn, abort_flag)) {
          fail();
          break;
        }
        tc_fence_after();
        const uint32_t src = tmem + acc.i * L.acc + ((uint32_t)(warp * 32) << 16);
        for (int i0 = 0; i0 < pairs; i0 += 8) {
          uint32_t q[8 * NT];
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
            if (i0 + i < pairs && row < R) {
              float* p = dst + (int64_t)(i0 + i) * R;
              *p = again ? *p + v : v;
            }
          }
        }
        acc.step(1, L.accs);
      }
    };
    // ======================= terms into the workspace =======================
    auto put = [&](const auto& terms, int place, int c, int kp) {
      constexpr int NT = sizeof(terms.q) / sizeof(uint2);
      const int e = pl.ent_of[place];
      const uint32_t ent = pl.ent[e];
      const TermTiles tt((int)(ent >> 20) * NT);
      uint8_t* p = terms_of(e, ent, kp, NT) + (int64_t)(c / DC_G) * tt.bytes();
      terms.put(p + c % DC_G * tt.rows * 128, p + DC_G * tt.rows * 128 + c % DC_G * tt.sf,
                (place - (int)(ent >> 10 & 1023u)) * NT, j16);
    };
    const int back = (jt >> 4 & 1) * (int)grid;     // a warp stays together for its shuffles
    if (!direct) {
      for (int u = unit0, units = a.P * kt1; u - back < units; u += unit_step) {
        const uint4 q = u == unit0 ? x0 : x_at(u);
        float v[8] = {bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y), bf16_lo(q.z), bf16_hi(q.z), bf16_lo(q.w), bf16_hi(q.w)};
        const Terms<X_TERMS> terms(v);
        const int p = (int)L.kt[0].quot(u), c = u - p * kt1, place = u < units ? pl.pos[p] : DC_DEAD;
        if (place != DC_DEAD && c * 128 + j16 * 8 < K1) put(terms, place, c, s1.kp.d);
      }
      asm volatile("bar.arrive 1, %0;" ::"n"(DC_JOIN + 32) : "memory");
      meeting(MEET_X, [] {});
    }
    if (epi) {
      drain_acc(First{});
    } else if (direct) {
      make(First{});
    } else {
      feed(First{});
    }
    // the activation, a unit a pair's tile
    struct Act {
      int place, c;
      bool in;
      Parts g, y;
    } next;
    const int units = nlive * kt2;
    auto act_of = [&](int u) {
      Act n;
      n.place = u < units ? (int)L.kt[1].quot(u) : 0, n.c = u - n.place * kt2;
      const int f = n.c * 128 + j16 * 8;
      n.in = u < units && f < K2;
      n.g = n.in ? parts_of(s1, a.part1, R1, n.place, f) : Parts{nullptr, 0};
      n.y = n.in ? parts_of(s1, a.part1, R1, n.place, a.F + f) : Parts{nullptr, 0};
      return n;
    };
    auto second_run = [&] {
      if (epi) return;
      r = Run(s2, cta);
      enter(s2);
    };
    if (direct) {
      meeting(MEET_SUMS, second_run);
    } else {
      meeting(MEET_SUMS, [&] { next = act_of(unit0); });
      for (int u = unit0; u - back < units; u += unit_step) {
        const Parts src[4] = {next.g, {next.g.p + 1, next.g.n}, next.y, {next.y.p + 1, next.y.n}};
        float4 q[4];
        gather(R1, src, q);
        const float gs[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
        const float us[8] = {q[2].x, q[2].y, q[2].z, q[2].w, q[3].x, q[3].y, q[3].z, q[3].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) act_of_sums(gs + 2 * i, us + 2 * i, v + 2 * i);
        const Terms<ACT_TERMS> terms(v);
        if (next.in) put(terms, next.place, next.c, s2.kp.d);
        if (u + unit_step - back < units) next = act_of(u + unit_step);
      }
      meeting(MEET_ACT, second_run);
    }
    if (epi) {
      drain_acc(Second{});
    } else if (direct) {
      make(Second{});
    } else {
      feed(Second{});
    }
    // the weighted sum over a token's experts, four neighbouring columns a thread,
    // runs of eight threads' a CTA in turn
    const uint32_t tasks = (uint32_t)a.T * L.quads.d;
    const uint32_t task0 = (((uint32_t)jt >> 3) * grid + cta) * 8 + (jt & 7);
    Parts src[8];
    auto parts_at = [&](int t, int h, int j0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int place = j0 + j < a.k ? pl.pos[t * a.k + j0 + j] : DC_DEAD;
        src[j] = place != DC_DEAD ? parts_of(s2, a.part2, R2, place, h) : Parts{nullptr, 0};
      }
    };
    int t, h;
    auto task_of = [&](uint32_t i) {
      if (i >= tasks) return;
      t = (int)L.quads.quot(i), h = (int)(i - (uint32_t)t * L.quads.d) * 4;
      parts_at(t, h, 0);
    };
    meeting(MEET_END, [&] { task_of(task0); });
    for (uint32_t i = task0; i < tasks; i += DC_JOIN * grid) {
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int j0 = 0; j0 < a.k; j0 += 8) {
        if (j0 > 0) parts_at(t, h, j0);
        float4 v[8];
        gather(R2, src, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (src[j].n == 0) continue;
          const float w = pl.w[t * a.k + j0 + j];
          o.x = fmaf(w, v[j].x, o.x), o.y = fmaf(w, v[j].y, o.y), o.z = fmaf(w, v[j].z, o.z), o.w = fmaf(w, v[j].w, o.w);
        }
      }
      *reinterpret_cast<uint2*>(a.out + (int64_t)t * a.H + h) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
      task_of(i + DC_JOIN * grid);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == DC_WARP_SF) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

int64_t pieces_of(int64_t K) { return ((K + 127) / 128 + DC_G - 1) / DC_G; }

// Largest number of partial sums of a tile, whatever the routing, when at least
// `ents` entries are live: a run has at least `s` pieces.
int64_t most_parts(int64_t ents, int64_t rt, int64_t kt) {
  constexpr int64_t grid = DECODE_MAX_CTAS;
  const int64_t C = ents * rt * kt;
  const int64_t s = C < DECODE_MIN_RUN ? 1 : C < grid * DECODE_MIN_RUN ? (DECODE_MIN_RUN + 1) / 2 : C / grid;
  const int64_t p = (kt - 1) / s + 2;
  return p < kt ? p : kt;
}
// Pairs of an entry, that is, of one reading of an expert: its terms have to fit a
// ring slot, and larger slots leave room for fewer: up to 20 pairs four, up to 32
// three, 64 (which N has room for) two.  T, which is enough where a token's choices
// differ, as long as there is room for four; beyond that room for more than most experts
// get.  (23 tokens of 8 of 256 experts of 2048 x 7168: 812 us with three slots for up to 24
// pairs, 733 with four for 20; 64 of 1 of 16 of 8192 x 5120 340 and 328.)
int entry_pairs(int64_t T, int64_t k, int64_t E) {
  const int64_t each = T * k / E;   // pairs an expert gets on average
  return T < 2 ? 2 : T <= 20 ? (int)T : each <= 12 ? 20 : each <= 24 ? 32 : 64;
}

// floats of the partial sums [parts][live pairs][R]: the most over any number of live pairs
int64_t part_floats(int64_t P, int64_t nb, int64_t R, int64_t K) {
  const int64_t rt = (R + 127) / 128, kp = pieces_of(K);
  int64_t most = 0;
  for (int64_t ents = 1; (ents - 1) * nb < P; ++ents) {
    const int64_t n = ents * nb < P ? ents * nb : P;
    const int64_t v = most_parts(ents, rt, kp) * n * R;
    if (v > most) most = v;
  }
  return most;
}

DecodeSmem layout(int P, int nb, int max_ent, int max_smem) {
  DecodeSmem L{};
  // (up to 8 rows that no term fills are read behind a tile, up to 512 bytes behind its scales)
  L.b_bytes = (TermTiles(ACT_TERMS * nb).bytes() + 1023) / 1024 * 1024;
  L.acc = ACT_TERMS * ((nb + 7) / 8 * 8);   // (the drain reads eight pairs' columns at a time)
  const int plan = 16 + max_ent * 4 + P * 10;
  const int bars = 8 * (4 * DC_MAX_SLOTS + 8);
  const int fixed = 1024 + bars + plan + 64;
  // 1024 to align the rings, 1024 for what is static
  L.slots = (max_smem - 2048 - fixed) / (DC_A_BYTES + DC_G * 512 + L.b_bytes);
  if (L.slots > DC_MAX_SLOTS) L.slots = DC_MAX_SLOTS;
  // Outputs that differ from the exact ones' bf16, 64 tokens of 1 of 16 experts of 8192 x
  // 5120: 1.10 of a thousand without chains, 0.78 with 16 pieces, 0.52 with eight, 0.46 with
  // four (products in 32 bits: 0.41), at the same time down to eight; four take 1% more.
  // More pairs take longer to add up (64 choices of each of 8 experts of 4096 x 2048 116 us
  // without or with 16, 128 with eight).
  L.chain = nb <= 20 ? 8 : 16;
  // (entries of 64 pairs fill half of tensor memory: no second accumulator)
  L.accs = 2 * L.acc + 12 * DC_G * L.slots <= 512 ? 2 : 1;
  L.team_log = L.slots >= 3 ? 1 : 2;
  L.teams = (DC_BWARPS >> L.team_log) < L.slots ? DC_BWARPS >> L.team_log : L.slots;
  L.b = L.slots * DC_A_BYTES;
  L.sfa = L.b + L.slots * L.b_bytes + 1024;
  L.bars = L.sfa + L.slots * DC_G * 512;
  L.plan = L.bars + bars;
  L.total = (L.plan + plan + 15) / 16 * 16;
  return L;
}

int64_t max_entries(int64_t P, int64_t E, int64_t nb) { return (P < E ? P : E) + P / nb; }

}  // namespace

// pieces are counted in 32 bits, times the CTAs
bool decode_fits(int64_t T, int64_t k, int64_t E, int64_t H, int64_t F) {
  const int64_t h = (H + 127) / 128, f2 = (2 * F + 127) / 128, c1 = pieces_of(H) * f2, c2 = pieces_of(F) * h;
  return max_entries(T * k, E, entry_pairs(T, k, E)) * (c1 > c2 ? c1 : c2) * DECODE_MAX_CTAS < (int64_t)1 << 32;
}

// What the workspace holds: both products' partial sums, and terms with their
// scales, both products' in turn in the same place.
struct DecodeSpace {
  int64_t part1, part2, terms;   // bytes
};
static DecodeSpace space_of(int64_t T, int64_t k, int64_t E, int64_t H, int64_t F) {
  const int64_t P = T * k, nb = entry_pairs(T, k, E), ents = max_entries(P, E, nb);
  auto terms = [&](int64_t K, int64_t nt) { return pieces_of(K) * DC_G * ((nt * P + 7 * ents) * 128 + 1024 * ents); };
  const int64_t t1 = terms(H, X_TERMS), t2 = terms(F, ACT_TERMS);
  return {part_floats(P, nb, 2 * F, H) * (int64_t)sizeof(float), part_floats(P, nb, H, F) * (int64_t)sizeof(float),
          t1 > t2 ? t1 : t2};
}

int64_t decode_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t F) {
  const DecodeSpace w = space_of(T, k, E, H, F);
  return w.part1 + w.part2 + w.terms;
}

cudaError_t launch_decode(DecodeArgs a, void* workspace, int num_sms, int max_smem, cudaStream_t st) {
  a.P = a.T * a.k;
  a.nb = entry_pairs(a.T, a.k, a.E);
  a.max_ent = (int)max_entries(a.P, a.E, a.nb);
  DecodeSmem L = layout(a.P, a.nb, a.max_ent, max_smem);
  if (num_sms > DECODE_MAX_CTAS || L.slots < 2 || L.accs * L.acc + 12 * DC_G * L.slots > 512 ||
      (a.P > 32 && (a.E + a.P + 64) * 4 > L.slots * L.b_bytes))
    return cudaErrorNotSupported;
  const DecodeSpace w = space_of(a.T, a.k, a.E, a.H, a.F);
  a.part1 = (float*)workspace;
  a.part2 = (float*)((uint8_t*)workspace + w.part1);
  a.terms = (uint8_t*)a.part2 + w.part2;
  a.stall = take_ring_stall_hook();
  CUtensorMap tm[2];
  const int64_t R[2] = {2 * (int64_t)a.F, a.H}, K[2] = {a.H, a.F};
  for (int i = 0; i < 2; ++i)
    L.kt[i] = Div((K[i] + 127) / 128), L.kp[i] = Div(pieces_of(K[i])), L.rt[i] = Div((R[i] + 127) / 128);
  L.grid = Div(num_sms), L.quads = Div(a.H / 4), L.k = Div(a.k);
  const uint8_t* q[2] = {a.q1, a.q2};
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[3] = {(cuuint64_t)K[i], (cuuint64_t)R[i], (cuuint64_t)a.E};
    const cuuint64_t strides[2] = {(cuuint64_t)K[i], (cuuint64_t)(K[i] * R[i])};
    const cuuint32_t box[3] = {128, 128, 1};
    if (!make_tmap(&tm[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, q[i], 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  // Up to eight tokens no entry has more than eight pairs; two at most of an expert on
  // average (6 of 64 experts of 1408 x 2048: four tokens 43.5 us by copies of terms, 40.8
  // made on the way, eight 67.8 and 65.2).  Their choices are not known here: eight tokens
  // that all have the same one of 8 experts of 4096 x 2048 take 26 us, 22 by copies.
  const bool few = a.T <= 8 && a.P <= 2 * a.E && L.team_log == 1;
  const void* kern = !few        ? (const void*)k_decode<DC_ANY>
                     : a.nb == 2 ? (const void*)k_decode<DC_TWO>
                                 : (const void*)k_decode<DC_FEW>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem - 1024);
  if (e != cudaSuccess) return e;
  void* args[] = {&tm[0], &tm[1], &a, &L};
  return cudaLaunchCooperativeKernel(kern, dim3((unsigned)num_sms), dim3(DC_THREADS), args, L.total + 1024, st);
}

}  // namespace fp8moe
