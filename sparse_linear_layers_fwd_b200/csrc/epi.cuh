// Epilogue of the layer: bias, activation and residual on the dequantized
// product, and the activations' derivatives for the backward.
//
// "Microsoft BitNet 1.58: The Era of 1-Bit Large Language Models", section
// "The BitLinear Layer", fifth operation: the product is rescaled by the kept
// scales; a feed-forward block then adds a bias, applies its activation and
// adds the residual stream. Done on the accumulator in registers, it costs no
// pass over memory of its own. All of it is evaluated in fp32 and rounded
// once to bf16; z, when kept for the backward, is rounded to bf16 too (what a
// training program keeps of it), but the activation of the forward sees it
// unrounded.
#pragma once

#include "common.cuh"

namespace sbn {

enum : int { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActSilu = 3, kActGelu = 4, kActCount = 5 };

struct EpiParams {
  const float* bias;         // [N_out] (per expert: [E, N_out]) or NULL
  const uint16_t* residual;  // [T, N_out] bf16 or NULL (may be the output itself)
  uint16_t* z;               // [T, N_out] bf16 or NULL: the activation's argument
  int act;
};

// 2^x and 1 / x on the special-function unit, each within two steps of fp32.
SBN_DEVFN float epi_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
SBN_DEVFN float epi_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(-z): the argument's rounding is |z| half steps, so the relative error
// is about (|z| + 5) 2^-24. Infinity where it overflows, and 1 / (1 + exp(-z)) 0.
SBN_DEVFN float epi_exp_neg(float z) { return epi_ex2(-1.44269504f * z); }
SBN_DEVFN float epi_sigmoid(float z) { return epi_rcp(1.f + epi_exp_neg(z)); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2), which its
// derivative needs too: the rational approximation 7.1.26 of Abramowitz and
// Stegun's Handbook of Mathematical Functions for erfc(|z| / sqrt 2), within
// 1.5e-7 absolute (half of it in Phi); a library erfc takes four times as
// many instructions, which bound the kernels around it. Relative to Phi the
// error passes 2^-12 below z = -3.6 and half a step of bf16, 2^-9, below -5.2
// (1.6e-3 at -5, 3.6e-3 at -6), where |z Phi| < 5e-7; 0.5 (1 + erf) in fp32 is
// off by more there (4e-2 at -5).
SBN_DEVFN float epi_phi(float z, float& e) {
  const float x = fabsf(z) * 0.70710678f;
  e = epi_ex2(-0.72134752f * z * z);
  const float t = epi_rcp(fmaf(0.3275911f, x, 1.f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  q = 0.5f * q * t * e;
  return z < 0.f ? q : 1.f - q;
}

// max(z, 0) that keeps a NaN.
SBN_DEVFN float epi_relu(float z) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
  return y;
}

SBN_DEVFN float act_f(int act, float z) {
  switch (act) {
    case kActRelu: return epi_relu(z);
    case kActRelu2: { const float r = epi_relu(z); return r * r; }
    case kActSilu: return z * epi_sigmoid(z);
    case kActGelu: { float e; return z * epi_phi(z, e); }
    default: return z;
  }
}

SBN_DEVFN float act_df(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActRelu2: return 2.f * epi_relu(z);
    case kActSilu: {
      const float s = epi_sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    case kActGelu: {
      float e;
      const float phi = epi_phi(z, e);
      return fmaf(z * 0.39894228f, e, phi);
    }
    default: return 1.f;
  }
}

// The activation over a register array (one branch for all of it).
template <int N>
SBN_DEVFN void act_all(int act, float (&v)[N]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActRelu, v[i]);
      break;
    case kActRelu2:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActRelu2, v[i]);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActSilu, v[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActGelu, v[i]);
      break;
    default: break;
  }
}

SBN_DEVFN uint16_t f32_to_bf16_bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

}  // namespace sbn
