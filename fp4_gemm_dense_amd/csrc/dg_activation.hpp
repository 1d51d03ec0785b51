// Activation functions and their derivatives (fp32), for the linear layers' epilogue
// (mxfp4_tile.hpp) and its backward pass (activation.hip).
//
// Three kinds, chosen by a uniform branch:
//   clamp    max(u, lo): the identity (lo = -infinity) and ReLU (lo = 0)
//   sigmoid  u * s, s = 1 / (1 + exp(-w)), w = u * (c1 + c3 u^2): SiLU (c1 = 1, c3 = 0), and GELU's
//            tanh form, since (1 + tanh(t)) / 2 = 1 / (1 + exp(-2t))
//   erf      u * Phi(u), Phi the normal distribution: GELU
// Phi comes from its tail, Phi(-a) = exp(-a^2 / 2) Q(a) for a >= 0, Q = t P(t) with t = 1 / (1 + 0.31 a): the
// form of Hastings' approximations (Approximations for Digital Computers, 1955), with P fitted here to Q
// itself, so that the tail keeps its relative error: measured against erfc in fp64 at 4 million a, 5e-7 of Q
// (its two fp32 roundings among it), 5.3e-7 of the tail up to a = 1, 9e-7 up to 4, and a^2 2^-24 from the
// exponent beyond, to 12.9, where exp leaves fp32's range.
// w beyond +-128 is held there (exp is 0 or infinity long before).  A NaN stays one.  u = -infinity
// stays in the identity, gives 0 in ReLU and NaN in the others, since 0 times infinity is none.
#pragma once

#include "dg_device.hpp"

namespace dg {

enum ActKind : int { ACT_KIND_CLAMP = 0, ACT_KIND_SIGMOID = 1, ACT_KIND_ERF = 2 };
struct Activation {
  int kind;
  float lo, c1, c3;
};

// A dg_activation value's (without its gated flag); false for an unknown one.  (mxfp4_linear.hip)
bool activation_of(int activation, Activation* a);

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float act_sigmoid(float u, const Activation& a) {
  const float x = __builtin_amdgcn_fmed3f(u, -128.f, 128.f);
  const float w = x * fmaf(a.c3 * x, x, a.c1);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * w));
}
// Phi(-|u|) and exp(-u^2 / 2), |u| held at 128
__device__ __forceinline__ float act_tail(float u, float* gauss) {
  const float a = fminf(fabsf(u), 128.f);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.31f, a, 1.f));
  const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * a * a);
  float q = 0.03591233857945959f;
  q = fmaf(q, t, -0.14191437636991855f);
  q = fmaf(q, t, 0.1556324890392326f);
  q = fmaf(q, t, -0.015455668418189962f);
  q = fmaf(q, t, 0.110422000256297f);
  q = fmaf(q, t, 0.10766985083583845f);
  q = fmaf(q, t, 0.12407775802946899f);
  q = fmaf(q, t, 0.12365569061357982f);
  *gauss = e;
  return e * q * t;
}
__device__ __forceinline__ float act_phi(float u, float* gauss) {
  const float tail = act_tail(u, gauss);
  return u < 0.f ? tail : 1.f - tail;
}

// The first N of v become their activations.
template <int N, int M>
__device__ __forceinline__ void activate(float (&v)[M], const Activation& a) {
  if (a.kind == ACT_KIND_CLAMP) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = v[e] < a.lo ? a.lo : v[e];
  } else if (a.kind == ACT_KIND_SIGMOID) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] *= act_sigmoid(v[e], a);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float g;
      v[e] *= act_phi(v[e], &g);
    }
  }
}

// act(u) and its derivative (ReLU's at 0: 0), of kind KIND.
template <int KIND, int N>
__device__ __forceinline__ void activate_both(const float (&u)[N], float (&y)[N], float (&dy)[N], const Activation& a) {
  if constexpr (KIND == ACT_KIND_CLAMP) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      y[e] = u[e] < a.lo ? a.lo : u[e];
      dy[e] = u[e] > a.lo || a.lo < 0.f ? 1.f : 0.f;   // (ReLU of a NaN: 0)
    }
  } else if constexpr (KIND == ACT_KIND_SIGMOID) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float s = act_sigmoid(u[e], a), x = __builtin_amdgcn_fmed3f(u[e], -128.f, 128.f);
      y[e] = u[e] * s;
      dy[e] = u[e] == u[e] ? s + x * s * (1.f - s) * fmaf(3.f * a.c3 * x, x, a.c1) : u[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float g;
      const float phi = act_phi(u[e], &g), x = __builtin_amdgcn_fmed3f(u[e], -128.f, 128.f);
      y[e] = u[e] * phi;
      dy[e] = u[e] == u[e] ? fmaf(x * g, 0.3989422804014327f, phi) : u[e];
    }
  }
}

}  // namespace dg
