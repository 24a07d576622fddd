// The activation functions and their derivatives, in fp32.
#pragma once

#include <cuda_runtime.h>

#include "../../include/mpopt.h"

namespace mpopt {
namespace {

// sqrt(2/pi) and the cubic's coefficient of the tanh form of GELU; with
// (1 + tanh u) / 2 = sigmoid(2 u) both activations are u * sigmoid(t(u)).
// 1 / (1 + 2^(-t log2 e)) from the two approximate instructions: each is within
// 2 units, and the rounding of t log2 e adds 2^-23 |t| of the value, far below
// the bf16 rounding that follows.  Below t = -87 the value, under 2^-126, is 0.
__device__ __forceinline__ float sigmoid(float t) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

constexpr float kGelu2 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluCubic = 0.044715f;

template <int kAct>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == OPT_ACT_RELU) return z > 0.f || z != z ? z : 0.f;
  if constexpr (kAct == OPT_ACT_GELU) return z * sigmoid(kGelu2 * (z + kGeluCubic * z * z * z));
  if constexpr (kAct == OPT_ACT_SILU) return z * sigmoid(z);
  return z;
}

template <int kAct>
__device__ __forceinline__ float activate_grad(float z) {
  if constexpr (kAct == OPT_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (kAct == OPT_ACT_GELU) {
    // z^2 kept finite: p (1 - p) is 0 where it would not be
    const float p = sigmoid(kGelu2 * (z + kGeluCubic * z * z * z));
    return p + z * p * (1.f - p) * (kGelu2 * (1.f + 3.f * kGeluCubic * fminf(z * z, 1e30f)));
  }
  if constexpr (kAct == OPT_ACT_SILU) {
    const float p = sigmoid(z);
    return p + z * p * (1.f - p);
  }
  return 1.f;
}

template <int kAct>
struct ActTag {
  static constexpr int value = kAct;
};

// Calls f with the activation as a compile-time tag: one branch for a block
// of elements instead of one for each.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  switch (act) {
    case OPT_ACT_RELU: f(ActTag<OPT_ACT_RELU>{}); break;
    case OPT_ACT_GELU: f(ActTag<OPT_ACT_GELU>{}); break;
    case OPT_ACT_SILU: f(ActTag<OPT_ACT_SILU>{}); break;
    default: f(ActTag<OPT_ACT_NONE>{}); break;
  }
}

}  // namespace
}  // namespace mpopt
