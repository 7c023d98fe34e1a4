// act.hpp -- activations of gated blocks and their derivatives, in 32 bits.
#pragma once

#include "../../include/gemm.h"
#include "common.hpp"

namespace dgemm {

// The logistic function of t, and of -t: neither loses digits where it is small.
struct Logistic {
  float up, down;
};
__device__ __forceinline__ Logistic logistic(float t) {
  const float e = expf(-fabsf(t));
  const float big = 1.0f / (1.0f + e), small = e * big;
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
  if (act == GEMM_ACT_SILU) return g / (1.0f + expf(-g));
  if (act == GEMM_ACT_GELU) return 0.5f * g * erfcf(g * -0.70710678118654752f);
  if (act == GEMM_ACT_GELU_TANH)
    return g / (1.0f + expf(-kGeluScale * (g + kGeluCubic * g * g * g)));
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
    slope = s.up + g * s.up * s.down * (kGeluScale * (1.0f + 3.0f * kGeluCubic * g * g));
  } else {
    value = g <= 0.0f ? 0.0f : g;
    slope = g <= 0.0f ? 0.0f : (g == g ? 1.0f : g);
  }
}

}  // namespace dgemm
