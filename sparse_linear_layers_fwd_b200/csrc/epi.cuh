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

// Phi(z), the normal distribution function; erfc keeps its relative accuracy
// for large negative z, where 1 + erf would cancel.
SBN_DEVFN float epi_phi(float z) { return 0.5f * erfcf(-0.70710678f * z); }

SBN_DEVFN float act_f(int act, float z) {
  switch (act) {
    case kActRelu: return fmaxf(z, 0.f);
    case kActRelu2: { const float r = fmaxf(z, 0.f); return r * r; }
    case kActSilu: return z / (1.f + expf(-z));
    case kActGelu: return z * epi_phi(z);
    default: return z;
  }
}

SBN_DEVFN float act_df(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActRelu2: return 2.f * fmaxf(z, 0.f);
    case kActSilu: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    case kActGelu: return epi_phi(z) + z * expf(-0.5f * z * z) * 0.39894228f;
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
