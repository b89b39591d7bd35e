// Internal interface between the host side of a block's fused operators
// (muon_block.cpp) and their HIP kernels.  Not part of the public C ABI.
#pragma once

#include "muon_layer.h"

namespace muon {

// matmul8 with an epilogue: z = a b^T + bias, y = act(z) + residual
struct Linear8Args : Matmul8Args {
  const float* bias;        // or null
  int act;                  // muon_activation
  const void* res;          // or null
  int res_fp32;
  long long ldr;
  void* z;                  // or null; y's type, bf16 beside an 8-bit y
  long long ldz;
  unsigned char* y8;        // the 8-bit result (y is then null)
  unsigned char* s8;
  long long ld_y8, sld_y8;
};
// out: MUON_BF16, MUON_FP32, or 2 for the 8-bit result
Matmul8Plan linear8_plan(int out, int m, int n, int ld);
hipError_t launch_linear8(int out, const Linear8Args& a, const Matmul8Plan& p, hipStream_t s);

// dz = dy act'(z) in bf16 and in 8 bits, and its sum over the rows
struct Linear8BackArgs {
  const void* dy;
  long long lddy;
  const void* z;            // or null (no activation)
  long long ldz;
  int act;
  int rows, cols;
  void* dz;                 // bf16, or null
  long long lddz;
  unsigned char* q;         // the 8-bit copy, or null
  unsigned char* s;
  long long ld, sld;
  float* dbias;             // or null
  int accumulate;
  float* part;              // [groups][cols] partial sums, unused with one group
  int groups;
};
int linear8_back_groups(int rows, int cols);
// types: 0 or 1 for dy and z in bf16 or fp32
hipError_t launch_linear8_backward(int dy_fp32, int z_fp32, const Linear8BackArgs& a, hipStream_t s);

}  // namespace muon
