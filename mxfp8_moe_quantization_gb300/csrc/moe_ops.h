// Arguments of the operators around the expert products: the router and the
// gated activation (internal).
#pragma once
#include <stdint.h>

namespace fp8moe {

struct RouterArgs {
  const void* logits;   // [T, E], row stride ld; fp32 or bf16
  int bf16;
  int wide;             // E a multiple of 4, rows of logits and dlogits aligned to four elements
  int64_t T, ld;
  int E, k;
  int score;            // FP8MOE_SCORE_*
  int two;              // the choice keeps every lane's two best at hand
  int renorm;
  float route_scale;
  const float* bias;    // [E] or NULL: added to the score for the choice alone
  const uint8_t* mask;  // [T] or NULL: 0 = not a token
  // forward outputs (counts, psum and loss together or not at all)
  int32_t* idx;         // [T, k]
  float* w;             // [T, k]
  int32_t* counts;      // [E + 1]
  float* psum;          // [E]
  float* loss;          // [1]
  void* workspace;
  // backward
  const int32_t* idx_in;
  const int32_t* counts_in;
  const float* dw;      // [T, k] or NULL
  const float* dloss;   // [1] or NULL
  void* dlogits;        // [T, E] of the logits' type
};

// CTAs of the forward whose partial counts and sums the workspace holds
constexpr int ROUTER_MAX_PARTS = 512;
constexpr int ROUTER_MAX_E = 1024;
constexpr int ROUTER_MAX_K = 32;

struct SwigluArgs {
  const uint16_t* dout;  // [M, F], backward only
  const uint16_t* h;     // [M, 2F], row stride ldh: gate | up
  int64_t M, F, ldh;
  const int32_t* offs;
  int E0, E1;            // groups of s0's / s1's layout, 0 where it is not grouped
  uint16_t* out;         // [M, W] bf16 or NULL (W = F forward, 2F backward)
  uint8_t *q0, *s0, *q1, *s1;
  int s0_layout, s1_layout;
  int num_sms;
  int* status;
  int stall;             // test hook: the first CTA's first warp never loads its first tile
};

}  // namespace fp8moe
