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
// Products of many rows: those of muon_matmul8 for a result of this type, exact ones, or
// the 8-bit instruction's.
enum Products { kMatmul8, kExact, kFast };
// out: MUON_BF16, MUON_FP32, or 2 for the 8-bit result
Matmul8Plan linear8_plan(int out, int m, int n, int ld, Products products);
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


// r = scale x + gate post(branch), h = norm(r)
struct ResidualArgs {
  const void* x;
  long long ldx;
  const void* b;            // the branch, or null
  long long ldb;
  int rows, cols;
  muon_residual_params p;
  void* r;                  // x's type, or null
  long long ldr;
  void* h;                  // or the 8-bit result
  int h_type;               // MUON_BF16, MUON_FP32, or 2 for the 8-bit result
  long long ldh;
  unsigned char* h8;
  unsigned char* s8;
  long long ld, sld;
  float* stats;             // [4][rows]: mean, rstd, and the post norm's
};
hipError_t launch_residual_norm(int x_bf16, int b_bf16, const ResidualArgs& a, hipStream_t s);

struct ResidualBackArgs {
  const void* dr;           // or null
  long long lddr;
  const void* dh;
  long long lddh;
  const void* r;
  long long ldr;
  const void* b;            // read only where the branch has a norm or a gate
  long long ldb;
  const void* x;            // read only for the scale's gradient
  long long ldx;
  int rows, cols;
  muon_residual_params p;
  const float* stats;
  void* dx;
  long long lddx;
  void* db;                 // or null
  long long lddb;
  muon_residual_grads g;
  int accumulate;
  double* part_scale;       // [groups]
  float* part;              // [groups][2 or 4][cols]
  int groups;
};
// Whether the branch's parameters have gradients: four sums per column, not two.
inline bool residual_branch(const muon_residual_params& p) { return p.post_weight || p.gate; }
int residual_back_groups(int rows, int cols, bool branch, bool b_fp32);
hipError_t launch_residual_norm_backward(int x_bf16, int b_bf16, const ResidualBackArgs& a,
                                         hipStream_t s);

}  // namespace muon
