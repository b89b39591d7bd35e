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

// The normal distribution's tail beyond |z|, Phi(-|z|), and exp(-z^2 / 2).
//
// For results in bf16 and 8 bits Abramowitz and Stegun 7.1.26, erfc(x) = (a1 t + .. +
// a5 t^5) exp(-x^2), t = 1 / (1 + p x) with x = |z| / sqrt(2), within 1.5e-7, here
// halved; a tenth of the instructions of the library's erfc, which an epilogue of 268
// million values would wait for (0.4 ms beside a product of 0.8 ms).
//
// FINE, for results in fp32 and for the slopes, whose sum is one: of that form with a
// polynomial of three degrees more, t = 1 / (1 + 0.3 |z|), fitted here to the least
// relative error of the tail over |z| <= 14, 1.5e-7.  As evaluated the tail is within
// (1.5 z^2 + 7) 2^-24 of itself, where the shorter formula is off by 3e-6 at z = -2 and
// 5e-5 at -3.
template <bool FINE>
__device__ __forceinline__ float normal_tail(float z, float& density) {
  float p, t;
  if constexpr (FINE) {
    t = rcp_fast(fmaf(0.3f, fabsf(z), 1.f));
    p = fmaf(0.0356747620f, t, -0.157203034f);
    p = fmaf(p, t, 0.206353426f);
    p = fmaf(p, t, -0.0536835715f);
    p = fmaf(p, t, 0.128561586f);
    p = fmaf(p, t, 0.0999135002f);
    p = fmaf(p, t, 0.120753951f);
    p = fmaf(p, t, 0.119629301f);
  } else {
    t = rcp_fast(fmaf(0.23164190f, fabsf(z), 1.f));  // p / sqrt(2)
    p = fmaf(0.5307027145f, t, -0.7265760135f);
    p = fmaf(p, t, 0.7107068705f);
    p = fmaf(p, t, -0.142248368f);
    p = fmaf(p, t, 0.127414796f);
  }
  density = exp2_fast(-0.72134752f * (z * z));
  return p * t * density;
}
// z Phi(z): for z > 0 z - z tail, else z tail.  Beyond 30 the tail is zero, which an
// infinity must not meet as a factor.
template <bool FINE>
__device__ __forceinline__ float gelu(float z) {
  float e;
  const float tail = normal_tail<FINE>(z, e);
  return fmaf(-__builtin_fminf(fabsf(z), 30.f), tail, __builtin_fmaxf(z, 0.f));
}

// (a NaN is below nothing and stays one)
__device__ __forceinline__ float relu(float z) { return z < 0.f ? 0.f : z; }

// z in front of a factor that is zero far from it, where an infinity (or, in the slopes,
// a square that overflows) must not meet it.  sigmoid(u) is 0 or 1 in fp32 from |u| =
// 104 on, so a slope is 0 or 1 beyond +-128 whichever z it is taken at.  A NaN stays
// one by the other factor.
__device__ __forceinline__ float above_minus_inf(float z) {
  return __builtin_fmaxf(z, -0x1.fffffep127f);
}
__device__ __forceinline__ float near_zero(float z) {
  return __builtin_amdgcn_fmed3f(z, -128.f, 128.f);
}

// u of gelu_tanh: z (1 + tanh(u / 2)) / 2 = z sigmoid(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float tanh_arg(float z) {
  return z * fmaf(0.071354816f, z * z, 1.5957691f);
}

// `act` is the same for all lanes: one branch for all of the values.  FINE: GELU for a
// result in fp32.
template <bool FINE, int S, int N>
__device__ __forceinline__ void activate(float (&v)[S][N], int act) {
  auto each = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < N; ++i) v[s][i] = f(v[s][i]);
  };
  switch (act) {
    case MUON_ACT_RELU: each([](float z) { return relu(z); }); break;
    case MUON_ACT_RELU2: each([](float z) { return relu(z) * relu(z); }); break;
    case MUON_ACT_GELU: each([](float z) { return gelu<FINE>(z); }); break;
    case MUON_ACT_GELU_TANH: each([](float z) { return above_minus_inf(z) * sigmoid(tanh_arg(z)); }); break;
    case MUON_ACT_SILU: each([](float z) { return above_minus_inf(z) * sigmoid(z); }); break;
    default: break;
  }
}

// d *= act'(z).  At zero relu's slope is 0; at an infinity a slope is its limit there.
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
      const float tail = normal_tail<true>(z[i], e);
      const float c = z[i] > 0.f ? 1.f - tail : tail;
      d[i] *= fmaf(0.39894228f * near_zero(z[i]), e, c);
    }
  } else if (act == MUON_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(tanh_arg(z[i])), b = near_zero(z[i]);
      const float du = fmaf(0.21406445f, b * b, 1.5957691f);
      d[i] *= fmaf(b * (s - s * s), du, s);
    }
  } else if (act == MUON_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(z[i]);
      d[i] *= fmaf(near_zero(z[i]), s - s * s, s);
    }
  }
}

}  // namespace muon
