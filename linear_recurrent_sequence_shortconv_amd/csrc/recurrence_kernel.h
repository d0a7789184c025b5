// Gates of the gated recurrence h_t = a_t h_{t-1} + u_t, value by value, and
// their derivatives.  With s = sigma(i), or 1,
//   log      a = e^f,                 u = s x
//   sigmoid  a = sigma(f),            u = (1 - a) s x
//   power    a = e^(-lam sigma(f)),   u = (1 - a^2)^(1/2) s x
// u = c s x throughout, with c = 1, 1 - a, or (1 - a^2)^(1/2).
#pragma once

#include "block_ops.h"
#include "vec_io.h"

namespace prism {

// Exponential, reciprocal and root: of bf16 inputs by the hardware's (1 ulp
// each; the exponential's argument adds 2^-24 of its size), of fp32 inputs by
// the library's.
template <typename E> __device__ inline float gate_exp(float x) {
  if constexpr (sizeof(E) == 2) return __builtin_amdgcn_exp2f(1.44269504f * x);
  return expf(x);
}
template <typename E> __device__ inline float gate_rcp(float x) {
  if constexpr (sizeof(E) == 2) return __builtin_amdgcn_rcpf(x);
  return 1.f / x;
}
template <typename E> __device__ inline float gate_sqrt(float x) {
  if constexpr (sizeof(E) == 2) return __builtin_amdgcn_sqrtf(x);
  return sqrtf(x);
}

// 1 - sigma(z) from e = e^-z and p = sigma(z) = 1 / (1 + e), to its own size (1 - p
// of a p near 1 would keep few digits); where e is infinite, 1.
__device__ inline float other_side(float e, float p) { return p == 0.f ? 1.f : e * p; }
template <typename E>
__device__ inline void sigmoid_pair(float z, float& p, float& q) {
  const float e = gate_exp<E>(-z);
  p = gate_rcp<E>(1.f + e);
  q = other_side(e, p);
}

// 1 - e^-z for z >= 0, aa = e^-z: below 1/8 by its series (1 - aa would be off by
// 2^-24 / z of itself; the first term left out is 2^-24 of the sum).
__device__ inline float one_minus_exp(float z, float aa) {
  float s = fmaf(z, 1.f / 120.f, -1.f / 24.f);
  s = fmaf(z, s, 1.f / 6.f);
  s = fmaf(z, s, -0.5f);
  s = fmaf(z, s, 1.f);
  return z < 0.125f ? z * s : 1.f - aa;
}

// What the gates of a value keep between the two sweeps of a tile: a, and k, from
// which c follows (sigmoid: c itself; power: e^-f).
struct GateValue {
  float a, k;
};
template <typename E, int G>
__device__ inline GateValue gate_value(float f, float lam) {
  GateValue g;
  if constexpr (G == GATE_LOG) {
    g.a = gate_exp<E>(f);
    g.k = 1.f;
  } else if constexpr (G == GATE_SIGMOID) {
    sigmoid_pair<E>(f, g.a, g.k);
  } else {
    g.k = gate_exp<E>(-f);
    g.a = gate_exp<E>(-lam * gate_rcp<E>(1.f + g.k));
  }
  return g;
}

template <typename E, int G, bool INP>
__device__ inline void gate_inputs(float x, float f, float i, float lam, float& a, float& u) {
  u = x;
  if constexpr (G == GATE_POWER) {
    const float p = gate_rcp<E>(1.f + gate_exp<E>(-f));
    a = gate_exp<E>(-lam * p);
    u *= gate_sqrt<E>(one_minus_exp(2.f * lam * p, a * a));
  } else {
    const GateValue g = gate_value<E, G>(f, lam);
    a = g.a;
    if (G == GATE_SIGMOID) u *= g.k;
  }
  if (INP) u *= gate_rcp<E>(1.f + gate_exp<E>(-i));
}

constexpr float NORMAL = 0x1p-126f;   // the smallest normal number

// Gradients of a value's inputs from g, that of h_t, ag = a_t g and h_{t-1}; dl: its
// part of the gradient of lam.  Where 1 - a^2 is below fp32's normal range (the
// hardware takes no root of such numbers) the root's part is left out: it is
// shut_gradients'; `low` then becomes true.
template <typename E, int G, bool INP>
__device__ inline void gate_gradients(const GateValue& v, float x, float i, float lam, float before, float g, float ag,
                                      float& dx, float& df, float& di, float& dl, bool& low) {
  float s = 1.f, t = 0.f, c = 1.f;
  if (INP) sigmoid_pair<E>(i, s, t);
  const float xi = INP ? s * x : x;
  dl = 0.f;
  if constexpr (G == GATE_LOG) {
    df = ag * before;
  } else if constexpr (G == GATE_SIGMOID) {
    c = v.k;
    df = ag * (before - xi) * c;
  } else {
    const float p = gate_rcp<E>(1.f + v.k);
    const float square = one_minus_exp(2.f * lam * p, v.a * v.a);
    const bool normal = square >= NORMAL;
    low = low || !normal;
    float slope;
    if constexpr (sizeof(E) == 2) {
      const float r = __builtin_amdgcn_rsqf(square);
      c = normal ? square * r : square;
      slope = normal ? v.a * r : 0.f;
    } else {
      c = sqrtf(square);
      slope = normal ? v.a / c : 0.f;
    }
    dl = -p * (ag * fmaf(-slope, xi, before));   // -p times the gradient of log a
    df = lam * other_side(v.k, p) * dl;
  }
  dx = g * c * s;
  di = INP ? dx * x * t : 0.f;
}

// Power gates that are nearly shut: 1 - a^2 = 2 lam sigma(f) below fp32's normal
// range, though neither factor is 0.
__device__ inline bool nearly_shut(float lam, float p) { return 2.f * lam * p < NORMAL && lam > 0.f && p > 0.f; }
// Their gradients.  Both factors are scaled by 2^64 by themselves, and the root's slope,
// which can leave the range, meets its sigma(f) first.  dl: the root's
// part alone.  Where a factor is 0 the slope is infinite, and its part is left out.
template <typename E, bool INP>
__device__ inline bool shut_gradients(const GateValue& v, float x, float i, float lam, float before, float g, float ag,
                                      float& dx, float& df, float& di, float& dl) {
  const float p = gate_rcp<E>(1.f + v.k);
  if (!nearly_shut(lam, p)) return false;
  float s = 1.f, t = 0.f;
  if (INP) sigmoid_pair<E>(i, s, t);
  const float q = 0x1p64f * p, zs = 2.f * (0x1p64f * lam) * q;   // 2^128 (1 - a^2)
  const float r = rsqrtf(zs);
  dx = g * (0x1p-64f * (zs * r)) * s;
  di = INP ? dx * x * t : 0.f;
  dl = ag * (q * r * (INP ? s * x : x));                         // (a = 1)
  df = lam * other_side(v.k, p) * (dl - p * (ag * before));
  return true;
}
}  // namespace prism
