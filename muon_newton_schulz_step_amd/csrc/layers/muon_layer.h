// Internal interface between the host side of the 8-bit linear layer and
// layer norm (muon_layer.cpp) and their HIP kernels.  Not part of the public
// C ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <type_traits>

#include "muon.h"

namespace muon {

// Columns of a block that shares one scale, and the row length of an 8-bit
// tensor in bytes and of its scales (whole blocks; whole 32-bit words).
constexpr int kBlock8 = 128;
inline long long ld8(long long cols) { return (cols + kBlock8 - 1) / kBlock8 * kBlock8; }
inline long long scale_ld8(long long cols) {
  return ((cols + kBlock8 - 1) / kBlock8 + 3) / 4 * 4;
}

struct Quant8Args {
  const void* x;
  long long ldx;
  int rows, cols;
  long long ld, sld;        // of the output
  unsigned char* q;
  unsigned char* s;
  unsigned char* qt;        // 128-row blocks: the transposed copy, or null
  unsigned char* st;
  long long ldt, sldt;
};
hipError_t launch_quantize8_rows(int x_bf16, const Quant8Args& a, hipStream_t s);
hipError_t launch_quantize8_blocks(int x_bf16, const Quant8Args& a, hipStream_t s);

struct Dequant8Args {
  const unsigned char* q;
  const unsigned char* s;
  long long ld, sld;
  int rows, cols, shift;    // shift: 0 for 1-row blocks, 7 for 128-row blocks
  void* y;
  long long ldy;
};
hipError_t launch_dequantize8(int y_bf16, const Dequant8Args& a, hipStream_t s);

// y[m][n] = sum_k a[m][k] b[n][k]
struct Matmul8Args {
  const unsigned char* a;
  const unsigned char* b;
  const unsigned char* sa;
  const unsigned char* sb;
  int m, n;
  int ld, sld;              // bytes of a row of values and of scales, both operands
  int shift_a, shift_b;     // 0 or 7, as for Dequant8Args
  void* y;
  long long ldy;
  int tiles_m, tiles_n, group_m;
};
// The kernel of a product and the bm x bn results of y that a workgroup computes.
struct Matmul8Plan {
  bool few;  // the kernel for few rows
  int bm, bn;
  bool exact = false;  // linear8's tiles: products of bf16 values
};
Matmul8Plan matmul8_plan(int y_bf16, int m, int n, int ld);
hipError_t launch_matmul8(int y_bf16, const Matmul8Args& a, const Matmul8Plan& p, hipStream_t s);

// dw[n][k] (+)= sum_t dy[t][n] x[t][k], in tiles of kTileT tokens
constexpr int kTileT = 64;
struct WeightGradArgs {
  const void* dy;           // bf16
  long long lddy;
  const unsigned char* x;
  const unsigned char* sx;
  int tokens, n, k;
  int ld, sld, shift;
  void* dw;
  int accumulate;
  float* part;              // [splits][n][k] partial sums, or null (one split)
  int splits, tiles_per_split;  // token tiles of a split
  int tiles_n, tiles_k;
};
struct WeightGradPlan {
  int kind, splits, tiles_per_split;  // tile variant; token splits, token tiles in each
  int bn, bk;
};
WeightGradPlan weight_grad_plan(int tokens, int n, int k);
hipError_t launch_weight_grad(int dw_bf16, const WeightGradArgs& a, const WeightGradPlan& p,
                              hipStream_t s);

struct NormArgs {
  const void* x;
  long long ldx;
  int rows, cols;
  const float* weight;
  const float* bias;        // or null
  float eps;
  void* y;
  long long ldy;
  unsigned char* y8;
  unsigned char* s8;
  long long ld, sld;
  float* mean;
  float* rstd;
};
// out: MUON_BF16, MUON_FP32, or 2 for the 8-bit output
hipError_t launch_layer_norm(int x_bf16, int out, const NormArgs& a, hipStream_t s);

struct NormBackArgs {
  const void* dy;
  long long lddy;
  const void* x;            // or the 8-bit tensor x8, sx8
  long long ldx;
  const unsigned char* x8;
  const unsigned char* sx8;
  long long ld, sld;
  int shift;
  int rows, cols;
  const float* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  long long lddx;
  float* dweight;
  float* dbias;             // or null
  int accumulate;
  float* part;              // [groups][2][cols], unused with one group
  int groups;
};
int norm_backward_groups(int rows, int cols);
// x: MUON_BF16, MUON_FP32, or 2 for the 8-bit tensor
hipError_t launch_layer_norm_backward(int dy_bf16, int x, const NormBackArgs& a, hipStream_t s);

// The per-launch timing log (muon_timing_enable) around one launch.
hipError_t timed_call(int kind, int m, int n, double flops, double exec_flops, double bytes,
                      hipStream_t s, hipError_t (*launch)(void*), void* arg);
template <typename F>
hipError_t timed_launch(int kind, int m, int n, double flops, double exec_flops, double bytes,
                        hipStream_t s, F&& launch) {
  return timed_call(
      kind, m, n, flops, exec_flops, bytes, s, [](void* f) { return (*static_cast<std::remove_reference_t<F>*>(f))(); },
      &launch);
}
// MUON_ERR_INVALID_ARG for a stream of another device than the current one.
int check_stream_device(hipStream_t stream);

}  // namespace muon
