// The activations of the gated projections, in fp32.
#pragma once

#include "mhc_ops.cuh"

namespace mhc {

// 1 / (1 + exp(-q)); below -87 it may be 0 instead of a number under 1e-37.
__device__ __forceinline__ float logistic(float q) { return __fdividef(1.f, 1.f + __expf(-q)); }

constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.044715f;  // 2 sqrt(2 / pi); gelu(g) ~ g logistic(A (g + B g^3))

template <int ACT>
__device__ __forceinline__ float activate(float g) {
  if constexpr (ACT == MHC_ACT_SILU) return g * logistic(g);
  if constexpr (ACT == MHC_ACT_GELU) return g * (0.5f * erfcf(g * -0.70710678f));
  if constexpr (ACT == MHC_ACT_GELU_TANH) return g * logistic(kGeluA * (g + kGeluB * g * g * g));
  return g > 0.f || g != g ? g : 0.f;
}

// The activation and its derivative.
template <int ACT>
__device__ __forceinline__ float2 activate_grad(float g) {
  if constexpr (ACT == MHC_ACT_SILU) {
    const float s = logistic(g);
    return make_float2(g * s, s + g * s * (1.f - s));
  }
  if constexpr (ACT == MHC_ACT_GELU) {
    const float p = 0.5f * erfcf(g * -0.70710678f);
    return make_float2(g * p, p + g * 0.3989422804f * __expf(-0.5f * g * g));
  }
  if constexpr (ACT == MHC_ACT_GELU_TANH) {
    const float s = logistic(kGeluA * (g + kGeluB * g * g * g));
    // (the square stays finite: s (1 - s) is 0 there, and 0 times infinity would be a NaN)
    return make_float2(g * s, s + g * s * (1.f - s) * kGeluA * (1.f + 3.f * kGeluB * fminf(g * g, 1e30f)));
  }
  return g > 0.f || g != g ? make_float2(g, 1.f) : make_float2(0.f, 0.f);
}

// g[i] = act(g[i]) * u[i].  The choice stands outside the loop, so the elements' chains of
// exponential and reciprocal overlap.
template <int N>
__device__ __forceinline__ void activate_product(float* g, const float* u, int act) {
  switch (act) {
    case MHC_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = activate<MHC_ACT_SILU>(g[i]) * u[i];
      break;
    case MHC_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = activate<MHC_ACT_GELU>(g[i]) * u[i];
      break;
    case MHC_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = activate<MHC_ACT_GELU_TANH>(g[i]) * u[i];
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = activate<MHC_ACT_RELU>(g[i]) * u[i];
  }
}

inline bool act_ok(int a) { return a >= MHC_ACT_SILU && a <= MHC_ACT_RELU; }
// Whether two memory ranges share a byte.
inline bool bytes_overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace mhc
