// The activations of a linear layer and their slopes, in fp32 (device side).
#pragma once

#include "fp8_device.h"
#include "muon.h"

namespace muon {

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + exp(-u)): both instructions are within 1 ulp, exp2's argument rounds
// to |u| 2^-24 more.
__device__ __forceinline__ float sigmoid(float u) {
  return rcp_fast(1.f + exp2_fast(-1.44269504f * u));
}

// The normal distribution function, and with it exp(-z^2 / 2): Abramowitz and
// Stegun 7.1.26, erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + p x) with
// x = |z| / sqrt(2), within 1.5e-7, so within 0.75e-7 of the function; a tenth of
// the instructions of the library's erfc, which an epilogue of 268 million values
// would wait for (0.4 ms beside a product of 0.8 ms).
__device__ __forceinline__ float normal_cdf(float z, float& density) {
  const float x = 0.70710678f * fabsf(z);
  const float t = rcp_fast(fmaf(0.3275911f, x, 1.f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  density = exp2_fast(-1.44269504f * (x * x));
  const float half = 0.5f * (p * t) * density;
  return z > 0.f ? 1.f - half : half;
}

// (a NaN is below nothing and stays one)
__device__ __forceinline__ float relu(float z) { return z < 0.f ? 0.f : z; }

// u of gelu_tanh: z (1 + tanh(u / 2)) / 2 = z sigmoid(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float tanh_arg(float z) {
  return z * fmaf(0.071354816f, z * z, 1.5957691f);
}

// `act` is the same for all lanes: one branch for eight values.
__device__ __forceinline__ void activate(float (&v)[8], int act) {
  if (act == MUON_ACT_RELU || act == MUON_ACT_RELU2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = relu(v[i]);
    if (act == MUON_ACT_RELU2)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= v[i];
  } else if (act == MUON_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e;
      v[i] *= normal_cdf(v[i], e);
    }
  } else if (act == MUON_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= sigmoid(tanh_arg(v[i]));
  } else if (act == MUON_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= sigmoid(v[i]);
  }
}

// d *= act'(z).  At zero relu's slope is 0.
__device__ __forceinline__ void activate_grad(float (&d)[8], const float (&z)[8], int act) {
  if (act == MUON_ACT_RELU) {
    // (a NaN in z is in the result, as it is in the forward pass's)
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = z[i] > 0.f ? d[i] : z[i] <= 0.f ? d[i] * 0.f : z[i];
  } else if (act == MUON_ACT_RELU2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= 2.f * relu(z[i]);
  } else if (act == MUON_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e;
      const float c = normal_cdf(z[i], e);
      d[i] *= fmaf(0.39894228f * z[i], e, c);
    }
  } else if (act == MUON_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(tanh_arg(z[i]));
      const float du = fmaf(0.21406445f, z[i] * z[i], 1.5957691f);
      d[i] *= fmaf(z[i] * (s - s * s), du, s);
    }
  } else if (act == MUON_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(z[i]);
      d[i] *= fmaf(z[i], s - s * s, s);
    }
  }
}

}  // namespace muon
