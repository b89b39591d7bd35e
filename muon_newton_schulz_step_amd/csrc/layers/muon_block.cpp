// Host side of a block's fused operators: argument checks (pure host code until
// the last one, so they run on a machine without a GPU), workspace sizes and
// launches.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "muon.h"
#include "muon_block.h"
#include "muon_checks.h"

using namespace muon;

namespace {

constexpr int kOut8 = 2;
bool is_activation(int a) { return a >= MUON_ACT_NONE && a <= MUON_ACT_SILU; }
const Span kNone{nullptr, 0};
Span vec_of(const void* p, long long n) { return {p, p ? (size_t)n * 4 : 0}; }

size_t back_workspace(int rows, int cols) {
  const int groups = linear8_back_groups(rows, cols);
  return groups > 1 ? (size_t)groups * (size_t)cols * sizeof(float) : 0;
}

}  // namespace

extern "C" {

int muon_linear8(const muon_tensor8* a, const muon_tensor8* b, const float* bias, int activation,
                 const void* residual, int residual_dtype, long long ldr, void* z, long long ldz,
                 void* y, int y_dtype, long long ldy, const muon_tensor8* y8, hipStream_t stream) {
  if (!tensor8_ok(a) || !tensor8_ok(b) || a->cols != b->cols || !is_activation(activation))
    return MUON_ERR_INVALID_ARG;
  if (!aligned(bias, 4)) return MUON_ERR_INVALID_ARG;
  const int m = a->rows, n = b->rows;
  if (y8 ? !tensor8_ok(y8) || y8->rows != m || y8->cols != n || y8->block_rows != 1 || y
         : !is_dtype(y_dtype))
    return MUON_ERR_INVALID_ARG;
  if (residual && !is_dtype(residual_dtype)) return MUON_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return MUON_OK;
  const size_t ez = y8 ? 2 : size_of(y_dtype);
  if ((!y8 && !matrix_ok(y, m, n, ldy)) || (residual && !matrix_ok(residual, m, n, ldr)) ||
      (z && !matrix_ok(z, m, n, ldz)))
    return MUON_ERR_INVALID_ARG;
  const Span res = residual ? matrix(residual, m, n, ldr, size_of(residual_dtype)) : kNone;
  if (conflict({y8 ? data_of(y8) : matrix(y, m, n, ldy, ez), y8 ? scale_of(y8) : kNone,
                z ? matrix(z, m, n, ldz, ez) : kNone},
               {data_of(a), scale_of(a), data_of(b), scale_of(b), vec_of(bias, n), res}))
    return MUON_ERR_INVALID_ARG;
  // (an 8-bit result of few rows has a workgroup of 512 threads to 128 columns)
  if (!tiles_fit(m, n)) return MUON_ERR_UNSUPPORTED;
  if (int st = check_stream_device(stream)) return st;
  Linear8Args g{};
  g.a = bytes_of(a->data); g.b = bytes_of(b->data);
  g.sa = bytes_of(a->scale); g.sb = bytes_of(b->scale);
  g.m = m; g.n = n;
  g.ld = (int)ld8(a->cols); g.sld = (int)scale_ld8(a->cols);
  g.shift_a = shift_of(a); g.shift_b = shift_of(b);
  g.y = y; g.ldy = ldy;
  g.bias = bias; g.act = activation;
  g.res = residual; g.res_fp32 = residual_dtype == MUON_FP32; g.ldr = ldr;
  g.z = z; g.ldz = ldz;
  if (y8) {
    g.y8 = bytes_of(y8->data); g.s8 = bytes_of(y8->scale);
    g.ld_y8 = ld8(n); g.sld_y8 = scale_ld8(n);
  }
  const int out = y8 ? kOut8 : y_dtype;
  const Matmul8Plan plan = linear8_plan(out, m, n, g.ld);
  const double dm = m, dn = n, k = a->cols;
  const double bytes = dm * k + dn * k + dm * dn * ((y8 ? 1.0 : (double)ez) + (z ? (double)ez : 0.0) +
                                                    (residual ? (double)size_of(residual_dtype) : 0.0));
  return status_of(timed_launch(MUON_K_LINEAR8, m, n, 2 * dm * dn * k,
                                2 * padded(m, plan.bm) * padded(n, plan.bn) * g.ld, bytes, stream,
                                [&] { return launch_linear8(out, g, plan, stream); }));
}

size_t muon_linear8_backward_workspace_bytes(int rows, int cols) {
  if (rows < 1 || rows > MUON_MAX_ROWS || cols < 1 || cols > MUON_MAX_COLS8) return 0;
  return back_workspace(rows, cols);
}

int muon_linear8_backward(const void* dy, int dy_dtype, long long lddy, const void* z, int z_dtype,
                          long long ldz, int activation, int rows, int cols, void* dz,
                          long long lddz, const muon_tensor8* dz8, float* dbias, int accumulate,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!is_dtype(dy_dtype) || !is_activation(activation) || !matrix_ok(dy, rows, cols, lddy) ||
      cols > MUON_MAX_COLS8 || (accumulate != 0 && accumulate != 1))
    return MUON_ERR_INVALID_ARG;
  const bool act = activation != MUON_ACT_NONE;
  if (act && (!is_dtype(z_dtype) || !matrix_ok(z, rows, cols, ldz))) return MUON_ERR_INVALID_ARG;
  if (!dz && !dz8 && !dbias && rows > 0) return MUON_ERR_INVALID_ARG;
  if ((dz && !matrix_ok(dz, rows, cols, lddz)) || !aligned(dbias, 4)) return MUON_ERR_INVALID_ARG;
  if (dz8 && (!tensor8_ok(dz8) || dz8->rows != rows || dz8->cols != cols || dz8->block_rows != 1))
    return MUON_ERR_INVALID_ARG;
  const Span s_dy = matrix(dy, rows, cols, lddy, size_of(dy_dtype));
  const Span s_z = act ? matrix(z, rows, cols, ldz, size_of(z_dtype)) : kNone;
  const Span s_dz = dz ? matrix(dz, rows, cols, lddz, 2) : kNone;
  const Span s_q = dz8 ? data_of(dz8) : kNone, s_s = dz8 ? scale_of(dz8) : kNone;
  if (conflict({s_dz, s_q, s_s, vec_of(dbias, cols)}, {s_dy, s_z})) return MUON_ERR_INVALID_ARG;
  const size_t need = dbias ? muon_linear8_backward_workspace_bytes(rows, cols) : 0;
  if (need) {
    if (!workspace || workspace_bytes < need || !aligned(workspace, MUON_WORKSPACE_ALIGN))
      return MUON_ERR_WORKSPACE;
    if (conflict({Span{workspace, need}}, {s_dy, s_z, s_dz, s_q, s_s, vec_of(dbias, cols)}))
      return MUON_ERR_INVALID_ARG;
  }
  if (rows == 0 && (!dbias || accumulate)) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  Linear8BackArgs g{};
  g.dy = dy; g.lddy = lddy; g.z = z; g.ldz = ldz; g.act = activation;
  g.rows = rows; g.cols = cols; g.dz = dz; g.lddz = lddz;
  if (dz8) {
    g.q = bytes_of(dz8->data); g.s = bytes_of(dz8->scale);
    g.ld = ld8(cols); g.sld = scale_ld8(cols);
  }
  g.dbias = dbias; g.accumulate = accumulate;
  g.part = static_cast<float*>(workspace);
  g.groups = linear8_back_groups(rows, cols);
  const double bytes = (double)rows * cols *
                       (size_of(dy_dtype) + (act ? (double)size_of(z_dtype) : 0.0) +
                        (dz ? 2.0 : 0.0) + (dz8 ? 1.0 : 0.0));
  return status_of(timed_launch(MUON_K_LINEAR8_BACK, rows, cols, 0.0, 0.0, bytes, stream, [&] {
    return launch_linear8_backward(dy_dtype == MUON_FP32, z_dtype == MUON_FP32, g, stream);
  }));
}

}  // extern "C"
