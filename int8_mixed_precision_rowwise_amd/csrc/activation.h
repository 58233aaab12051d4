// Activations and their derivatives in fp32, for the epilogues and the
// backward of the linears.
//
// An activation's value is rounded to bf16 (half a step is 2^-8 of it at most) at once and sits in a GEMM's
// epilogue, where every operation shows: it takes the hardware's exponential and
// reciprocal (1 ulp each) as they are.  A derivative also goes into the bias
// gradient, which stays fp32, and into a pass that memory bounds: it carries the low
// part of the exponent's product and a Newton step for the reciprocal, so that it is
// within a few 2^-24.  The normal distribution's upper tail is
// Q(z) = exp(-z^2 / 2) t P(t), t = 1 / (1 + c z), z >= 0, with P fitted to least
// relative error over 0 .. 14 (5e-6 with 6 coefficients, 2e-8 with 9), so the far
// negative side of GELU keeps its relative accuracy.
#pragma once

#include <hip/hip_runtime.h>

namespace i8mp {
namespace {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// 1 / (1 + 2^-x)
__device__ __forceinline__ float sigmoid2(float x) { return __builtin_amdgcn_rcpf(1.0f + exp2_hw(-x)); }

__device__ __forceinline__ float normal_cdf(float z) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(z), 0.31f, 1.0f));
  float p = -0.07392736248f;
  p = __builtin_fmaf(p, t, 0.18044506100f);
  p = __builtin_fmaf(p, t, 0.01575084609f);
  p = __builtin_fmaf(p, t, 0.13342630533f);
  p = __builtin_fmaf(p, t, 0.12044223795f);
  p = __builtin_fmaf(p, t, 0.12386059923f);
  const float q = exp2_hw(z * z * -0.72134752044448170f) * (p * t);  // -log2(e) / 2
  return z < 0.0f ? q : 1.0f - q;
}

constexpr float kGeluB = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;
constexpr float kLog2eF = 1.4426950408889634f;

// (1 + tanh(b (z + c z^3))) / 2 = sigmoid(2 b (z + c z^3))
__device__ __forceinline__ float gelu_gate(float z) {
  const float u = __builtin_fmaf(z * z, 2 * kLog2eF * kGeluB * kGeluC, 2 * kLog2eF * kGeluB);
  return sigmoid2(z * u);
}

template <int ACT>
__device__ __forceinline__ float activation(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if constexpr (ACT == kActGelu) return z * normal_cdf(z);
  if constexpr (ACT == kActGeluTanh) return z * gelu_gate(z);
  if constexpr (ACT == kActSilu) return z * sigmoid2(z * kLog2eF);
  return z;
}

// exp(x) for x <= 0: 2^(x log2(e)) with the product's low part (0 where fp32 ends).
__device__ __forceinline__ float exp_full(float x) {
  x = __builtin_fmaxf(x, -150.0f);
  const float h = x * kLog2eF;
  const float l = __builtin_fmaf(x, 1.9259629911266175e-8f, __builtin_fmaf(x, kLog2eF, -h));
  const float e = exp2_hw(h);
  return __builtin_fmaf(e, l * 0.69314718055994531f, e);
}
// 1 / d for finite d >= 1.
__device__ __forceinline__ float rcp_full(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}
// 1 / (1 + exp(-x)) and 1 minus that, each to its own relative accuracy.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& c) {
  const float e = exp_full(-__builtin_fabsf(x));
  const float r = rcp_full(1.0f + e), q = e * r;
  s = x < 0.0f ? q : r;
  c = x < 0.0f ? r : q;
}

// The derivative at z (NaN at an infinity, as z times 0 in the formulas has it).
template <int ACT>
__device__ __forceinline__ float activation_grad(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
  if constexpr (ACT == kActGelu) {
    const float bell = exp_full(-0.5f * (z * z));  // exact argument: z has 8 bits
    const float t = rcp_full(__builtin_fmaf(__builtin_fabsf(z), 0.20999999344348907f, 1.0f));
    float p = -0.07165630906820297f;
    p = __builtin_fmaf(p, t, 0.28358858823776245f);
    p = __builtin_fmaf(p, t, -0.3302534222602844f);
    p = __builtin_fmaf(p, t, 0.3494010269641876f);
    p = __builtin_fmaf(p, t, -0.09392520040273666f);
    p = __builtin_fmaf(p, t, 0.12487272173166275f);
    p = __builtin_fmaf(p, t, 0.06919217109680176f);
    p = __builtin_fmaf(p, t, 0.08506885170936584f);
    p = __builtin_fmaf(p, t, 0.08371157199144363f);
    const float q = bell * (p * t);
    return __builtin_fmaf(z * 0.39894228040143268f, bell, z < 0.0f ? q : 1.0f - q);  // 1 / sqrt(2 pi)
  }
  if constexpr (ACT == kActGeluTanh) {
    const float z2 = z * z;
    float s, c;
    sigmoid_pair(z * __builtin_fmaf(z2, 2 * kGeluB * kGeluC, 2 * kGeluB), s, c);
    const float du = __builtin_fmaf(z2, 6 * kGeluB * kGeluC, 2 * kGeluB);
    const float w = s * c;  // 0 from |z| = 11 on; z du is infinite from 10^13 on
    return __builtin_fmaf(z * (w == 0.0f ? 0.0f : du), w, s);
  }
  if constexpr (ACT == kActSilu) {
    float s, c;
    sigmoid_pair(z, s, c);
    return __builtin_fmaf(z * s, c, s);
  }
  return 1.0f;
}

}  // namespace
}  // namespace i8mp
