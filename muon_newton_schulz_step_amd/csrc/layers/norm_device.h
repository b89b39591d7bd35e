// Device-side helpers that the norms' kernels share.  Internal; not part of the
// C ABI.
#pragma once

#include "fp8_device.h"

namespace muon {

constexpr int kOut8 = 2;  // the 8-bit type among MUON_BF16, MUON_FP32

template <int K> struct ElemOf { using type = float; };
template <> struct ElemOf<MUON_BF16> { using type = bf16_t; };
template <> struct ElemOf<kOut8> { using type = unsigned char; };

// Sum over the team's waves of each wave's v, the same in all lanes.  `buf`
// alternates between calls, so one barrier per call is enough.
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*buf)[16], int wave, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TEAM > 1) {
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) buf[i][wave] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < TEAM; ++w) s += buf[i][w];
      v[i] = s;
    }
  }
}

}  // namespace muon
