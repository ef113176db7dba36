// ffn_math.cuh -- activations of the feed-forward operators and their derivatives, in FP32.
//
// sigmoid(z) = 1 / (1 + e) with e = exp(-z), and 1 - sigmoid(z) = e * sigmoid(z)
// without cancellation.  exp(t) as 2^(t / ln 2) by ex2.approx is off by two
// spacings and by |t| 2^-24 relative, as much as half a spacing of its FP32
// argument is worth; rcp.approx by one.  Both flush what is below 2^-126.
//
// gelu needs Phi(z) = erfc(-z / sqrt(2)) / 2, which for z < 0 falls as exp(-z^2 /
// 2) does, so that 1 + erf would lose it.  With t = 1 / (1 + q |z|) the quotient
// erfc(|z| / sqrt(2)) / (2 exp(-z^2 / 2)) is t times a polynomial of degree 8 in
// t, fitted here for the least relative error over |z| <= 13.4 (Lawson's
// reweighted least squares): 3.9e-8 with the coefficients in FP32, two thirds of
// its half spacing.  With erfcf,
// 4096 x 8192 outputs of K = 2048 took 135 us against 84 without an activation; two
// values at a time, packed, share most instructions.
#pragma once
#include "ffn_internal.h"

namespace gp {

constexpr float kRsqrt2Pi = 0.39894228040143268f;        // 1 / sqrt(2 pi)
constexpr float kTanhScale = 1.59576912160573071f;       // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

__device__ __forceinline__ float fast_exp(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// z up to `most` either way, a NaN as it is.
__device__ __forceinline__ float at_most(float z, float most) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(z), "f"(most), "f"(-most));
  return r;
}

struct Sigmoid {
  float s, rest;   // sigmoid and 1 - sigmoid
};
__device__ __forceinline__ Sigmoid sigmoid_above(float z) {   // (z above -88.7, where e is finite)
  const float e = fast_exp(-z);
  const float s = fast_rcp(1.f + e);
  return Sigmoid{s, e * s};
}
__device__ __forceinline__ Sigmoid sigmoid_of(float z) {
  float t;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(t) : "f"(z), "f"(-88.f));   // (s is 0 there; a NaN stays)
  return sigmoid_above(t);
}

// Two FP32 values in one 64-bit register: a packed FMA is one instruction, and rounds each half as a single one does.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 of_two(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_two(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// erfc(|z| / sqrt(2)) / 2 and exp(-z^2 / 2) of two values; both 0 from |z| = 20 on, whatever lies there (a NaN stays).
struct Tail {
  float2 u, h, e;   // u: |z| up to 20
};
__device__ __forceinline__ Tail tail_of(float z0, float z1) {
  float2 u = make_float2(fabsf(z0), fabsf(z1));
  u.x = u.x > 20.f ? 20.f : u.x;
  u.y = u.y > 20.f ? 20.f : u.y;
  const float2 d = of_two(fma_two(two(0.26162952f, 0.26162952f), two(u.x, u.y), two(1.f, 1.f)));
  const uint64_t t = two(fast_rcp(d.x), fast_rcp(d.y));
  uint64_t p = two(0.030961534f, 0.030961534f);
  constexpr float kC[8] = {-0.15163641f, 0.24342063f, -0.14265560f, 0.15540075f, 0.053260274f, 0.10312700f, 0.10371493f, 0.10440688f};
#pragma unroll
  for (int i = 0; i < 8; ++i) p = fma_two(p, t, two(kC[i], kC[i]));
  const float2 e = make_float2(fast_exp(-0.5f * u.x * u.x), fast_exp(-0.5f * u.y * u.y));
  return Tail{u, of_two(mul_two(two(e.x, e.y), mul_two(t, p))), e};
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case GP_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case GP_ACT_GELU: {
      const Tail t = tail_of(z, z);
      return fmaxf(z, 0.f) - t.u.x * t.h.x;
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
__device__ __forceinline__ ActSlope gelu_slope(float z, float u, float h, float e) {
  return ActSlope{fmaxf(z, 0.f) - u * h, fmaf(copysignf(u, z) * kRsqrt2Pi, e, z > 0.f ? 1.f - h : h)};
}
// In silu and gelu_tanh z is a factor of what vanishes for large |z|: it goes up to where that is 0 only, as its square, or an
// infinity, would make that NaN (values kept in FP16 are infinite where the sum was past 65504, the output beside them not).
__device__ __forceinline__ ActSlope activate_slope(float z, int act) {
  switch (act) {
    case GP_ACT_RELU: return ActSlope{z > 0.f ? z : (z != z ? z : 0.f), z > 0.f ? 1.f : (z != z ? z : 0.f)};
    case GP_ACT_GELU_TANH: {
      const float c = at_most(z, 20.f);
      const Sigmoid g = sigmoid_of(kTanhScale * fmaf(kTanhCube * c * c, c, c));
      return ActSlope{fmaxf(z, c) * g.s, fmaf(c * g.s * g.rest, kTanhScale * fmaf(3.f * kTanhCube * c, c, 1.f), g.s)};
    }
    case GP_ACT_SILU: {
      const float c = at_most(z, 88.f);
      const Sigmoid g = sigmoid_above(c);
      return ActSlope{fmaxf(z, c) * g.s, fmaf(c * g.s, g.rest, g.s)};
    }
    case GP_ACT_SIGMOID: {
      const Sigmoid g = sigmoid_of(z);
      return ActSlope{g.s, g.s * g.rest};
    }
    default: return ActSlope{z, 1.f};
  }
}
// Of N values, two at a time where that is packed.
template <int ACT, int N>
__device__ __forceinline__ void activate_slopes(ActSlope (&s)[N], const float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if (ACT == GP_ACT_GELU) {
      const Tail t = tail_of(z[i], z[i + 1]);
      s[i] = gelu_slope(z[i], t.u.x, t.h.x, t.e.x);
      s[i + 1] = gelu_slope(z[i + 1], t.u.y, t.h.y, t.e.y);
    } else {
      s[i] = activate_slope(z[i], ACT);
      s[i + 1] = activate_slope(z[i + 1], ACT);
    }
  }
}

// The switch outside of the loop: N values at a time.
template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  static_assert(N % 2 == 0, "pairs");
  switch (act) {
    case GP_ACT_NONE: break;
    case GP_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const Tail t = tail_of(v[i], v[i + 1]);
        v[i] = fmaxf(v[i], 0.f) - t.u.x * t.h.x;
        v[i + 1] = fmaxf(v[i + 1], 0.f) - t.u.y * t.h.y;
      }
      break;
#define GP_ACT_LOOP(A)                                           \
  case A:                                                        \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = activate(v[i], A); \
    break;
    GP_ACT_LOOP(GP_ACT_RELU)
    GP_ACT_LOOP(GP_ACT_GELU_TANH)
    GP_ACT_LOOP(GP_ACT_SILU)
    GP_ACT_LOOP(GP_ACT_SIGMOID)
#undef GP_ACT_LOOP
  }
}

}  // namespace gp
