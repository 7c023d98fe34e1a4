// act.hpp -- activations of gated blocks and their derivatives, in 32 bits.
#pragma once

#include "../../include/gemm.h"
#include "common.hpp"

namespace dgemm {

// The logistic function of t, and of -t: neither loses digits where it is small,
// down to the smallest normal number, below which it is 0.  exp(x) for x = -|t| is
// 2^(x log2 e), the product's rounding error made up for to first order, so that
// no digits are lost for large |t| either; the hardware's 2^x and reciprocal are
// good to a unit in the last place, its 2^x is 0 where it is below 2^-126 (silu:
// gates below -87.3, off by less than 88 * 2^-126 there; with 2^(y + 64) and 2^-64
// instead 4096 x 8192 x 64 takes 46.3 us for 43.9, 4096 x 8192 x 4096 473 for 468).
// (Half the instructions of expf and a division: [dG dU] of 4096 x 4096 halves from
// memory 46 to 28 us together with wider loads.)
struct Logistic {
  float up, down;
};
__device__ __forceinline__ Logistic logistic(float t) {
  constexpr float kLog2e = 1.44269504088896341f;        // rounded to 1.44269502162933
  constexpr float kLog2eLow = 1.92596299e-8f;            // what the rounding left out
  constexpr float kLn2 = 0.69314718055994531f;
  const float x = fmaxf(-fabsf(t), -150.0f);             // (exp(-150) is 0; no infinities)
  const float y = x * kLog2e;
  const float low = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -y));
  const float p = __builtin_amdgcn_exp2f(y);
  const float e = __builtin_fmaf(p, low * kLn2, p);
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  return t >= 0.0f ? Logistic{big, small} : Logistic{small, big};
}

constexpr float kGeluScale = 1.5957691216057308f;   // sqrt(8/pi): 0.5 (1 + tanh(t)) is logistic(2 t)
constexpr float kGeluCubic = 0.044715f;

// act(g): a NaN stays one.
//   silu       g / (1 + exp(-g))
//   gelu       g Phi(g), Phi(g) = erfc(-g / sqrt 2) / 2 (no digits lost for g < 0)
//   gelu_tanh  g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2
//   relu       max(g, 0)
__device__ __forceinline__ float act_value(int act, float g) {
  if (act == GEMM_ACT_SILU) return g * logistic(g).up;
  if (act == GEMM_ACT_GELU) return 0.5f * g * erfcf(g * -0.70710678118654752f);
  if (act == GEMM_ACT_GELU_TANH)
    return g * logistic(kGeluScale * (g + kGeluCubic * g * g * g)).up;
  return g <= 0.0f ? 0.0f : g;
}

// act(g) and act'(g).
__device__ __forceinline__ void act_both(int act, float g, float &value, float &slope) {
  if (act == GEMM_ACT_SILU) {
    const Logistic s = logistic(g);
    value = g * s.up;
    slope = s.up * (1.0f + g * s.down);
  } else if (act == GEMM_ACT_GELU) {
    const float p = 0.5f * erfcf(g * -0.70710678118654752f);
    value = g * p;
    slope = p + g * (0.39894228040143268f * expf(-0.5f * g * g));
  } else if (act == GEMM_ACT_GELU_TANH) {
    const Logistic s = logistic(kGeluScale * (g + kGeluCubic * g * g * g));
    value = g * s.up;
    // (g * g is limited where it would leave fp32: s.down or s.up is 0 there)
    slope = s.up + g * s.up * s.down *
                       (kGeluScale * (1.0f + 3.0f * kGeluCubic * fminf(g * g, 1e30f)));
  } else {
    value = g <= 0.0f ? 0.0f : g;
    slope = g <= 0.0f ? 0.0f : (g == g ? 1.0f : g);
  }
}

}  // namespace dgemm
