// ffn_math.cuh -- activations of the feed-forward operators and their derivatives, in FP32.
//
// sigmoid(z) = 1 / (1 + e) with e = exp(-z), and 1 - sigmoid(z) = e * sigmoid(z)
// without cancellation.  __expf(t) is off by about |t| 2^-24 relative: as much
// as half a spacing of its FP32 argument is worth.
//
// gelu needs Phi(z) = erfc(-z / sqrt(2)) / 2, which for z < 0 falls as exp(-z^2 /
// 2) does, so that 1 + erf would lose it.  With t = 1 / (1 + q |z|) the quotient
// erfc(|z| / sqrt(2)) / (2 exp(-z^2 / 2)) is t times a polynomial of degree 8 in
// t, fitted here for the least relative error over |z| <= 13.4 (Lawson's
// reweighted least squares): 1.7e-8, a third of FP32's half spacing.  Sixteen
// instructions; with erfcf the 8192 columns of a 4096 x 2048 activation took
// 135 us against 84 without an activation.
#pragma once
#include "ffn_internal.h"

namespace gp {

constexpr float kRsqrt2Pi = 0.39894228040143268f;        // 1 / sqrt(2 pi)
constexpr float kTanhScale = 1.59576912160573071f;       // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

struct Sigmoid {
  float s, rest;   // sigmoid and 1 - sigmoid
};
__device__ __forceinline__ Sigmoid sigmoid_of(float z) {
  const float t = z < -88.f ? 88.f : -z;     // (e stays finite and s is 0 there; a NaN stays)
  const float e = __expf(t);
  const float s = __fdividef(1.f, 1.f + e);
  return Sigmoid{s, e * s};
}

// erfc(|z| / sqrt(2)) / 2 and exp(-z^2 / 2); both 0 from |z| = 20 on, whatever lies there (a NaN stays).
struct Tail {
  float u, h, e;   // |z| up to 20
};
__device__ __forceinline__ Tail tail_of(float z) {
  float u = fabsf(z);
  u = u > 20.f ? 20.f : u;
  const float t = __fdividef(1.f, fmaf(0.26162952f, u, 1.f));
  float p = 0.030961534f;
  p = fmaf(p, t, -0.15163641f);
  p = fmaf(p, t, 0.24342063f);
  p = fmaf(p, t, -0.14265560f);
  p = fmaf(p, t, 0.15540075f);
  p = fmaf(p, t, 0.053260274f);
  p = fmaf(p, t, 0.10312700f);
  p = fmaf(p, t, 0.10371493f);
  p = fmaf(p, t, 0.10440688f);
  const float e = __expf(-0.5f * u * u);
  return Tail{u, e * (t * p), e};
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case GP_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case GP_ACT_GELU: {
      const Tail t = tail_of(z);
      return fmaxf(z, 0.f) - t.u * t.h;
    }
    case GP_ACT_GELU_TANH: return z * sigmoid_of(kTanhScale * fmaf(kTanhCube * z * z, z, z)).s;
    case GP_ACT_SILU: return z * sigmoid_of(z).s;
    case GP_ACT_SIGMOID: return sigmoid_of(z).s;
    default: return z;
  }
}

// The activation and its derivative.
struct ActSlope {
  float a, d;
};
__device__ __forceinline__ ActSlope activate_slope(float z, int act) {
  switch (act) {
    case GP_ACT_RELU: return ActSlope{z > 0.f ? z : (z != z ? z : 0.f), z > 0.f ? 1.f : (z != z ? z : 0.f)};
    case GP_ACT_GELU: {
      const Tail t = tail_of(z);
      const float phi = z > 0.f ? 1.f - t.h : t.h;
      return ActSlope{fmaxf(z, 0.f) - t.u * t.h, fmaf(copysignf(t.u, z) * kRsqrt2Pi, t.e, phi)};
    }
    case GP_ACT_GELU_TANH: {
      const Sigmoid g = sigmoid_of(kTanhScale * fmaf(kTanhCube * z * z, z, z));
      return ActSlope{z * g.s, fmaf(z * g.s * g.rest, kTanhScale * fmaf(3.f * kTanhCube * z, z, 1.f), g.s)};
    }
    case GP_ACT_SILU: {
      const Sigmoid g = sigmoid_of(z);
      return ActSlope{z * g.s, fmaf(z * g.s, g.rest, g.s)};
    }
    case GP_ACT_SIGMOID: {
      const Sigmoid g = sigmoid_of(z);
      return ActSlope{g.s, g.s * g.rest};
    }
    default: return ActSlope{z, 1.f};
  }
}

// The switch outside of the loop: N values at a time.
template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  switch (act) {
    case GP_ACT_NONE: break;
#define GP_ACT_LOOP(A)                                           \
  case A:                                                        \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = activate(v[i], A); \
    break;
    GP_ACT_LOOP(GP_ACT_RELU)
    GP_ACT_LOOP(GP_ACT_GELU)
    GP_ACT_LOOP(GP_ACT_GELU_TANH)
    GP_ACT_LOOP(GP_ACT_SILU)
    GP_ACT_LOOP(GP_ACT_SIGMOID)
#undef GP_ACT_LOOP
  }
}

}  // namespace gp
