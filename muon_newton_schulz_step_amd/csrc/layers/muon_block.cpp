// Host side of a block's fused operators: argument checks (pure host code until
// the last one, so they run on a machine without a GPU), workspace sizes and
// launches.
#include <hip/hip_runtime_api.h>

#include <algorithm>
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

// The parameters: what is there is aligned, and nothing is there without what it is for.
bool params_ok(const muon_residual_params* p) {
  if (!p || !p->weight || (p->post_bias && !p->post_weight)) return false;
  for (const float* v : {p->weight, p->bias, p->post_weight, p->post_bias, p->gate, p->scale})
    if (!aligned(v, 4)) return false;
  return std::isfinite(p->eps) && p->eps >= 0.f && (p->rms == 0 || p->rms == 1);
}
// The two element types: the branch is no wider than the stream.
int types_status(int x_dtype, int branch_dtype) {
  if (!is_dtype(x_dtype) || !is_dtype(branch_dtype)) return MUON_ERR_INVALID_ARG;
  return x_dtype == MUON_BF16 && branch_dtype == MUON_FP32 ? MUON_ERR_UNSUPPORTED : MUON_OK;
}
// The sums over the rows: groups fp64 numbers, padded to 256 bytes, and their rows.
size_t scale_parts_bytes(int groups) { return ((size_t)groups * sizeof(double) + 255) / 256 * 256; }

size_t back_workspace(int rows, int cols) {
  const int groups = linear8_back_groups(rows, cols);
  return groups > 1 ? (size_t)groups * (size_t)cols * sizeof(float) : 0;
}

}  // namespace

extern "C" {

int muon_linear8(const muon_tensor8* a, const muon_tensor8* b, const float* bias, int activation,
                 const void* residual, int residual_dtype, long long ldr, void* z, long long ldz,
                 void* y, int y_dtype, long long ldy, const muon_tensor8* y8, hipStream_t stream) {
  const int choice = activation > 0 ? activation & (MUON_EXACT | MUON_FAST) : 0;
  activation -= choice;
  if (choice == (MUON_EXACT | MUON_FAST) || (choice == MUON_FAST && !y8 && y_dtype == MUON_FP32))
    return MUON_ERR_INVALID_ARG;
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
  // what is rounded to 8 bits behind an epilogue is exact by itself
  const bool fused = bias || activation != MUON_ACT_NONE || residual || z;
  const Products products = choice == MUON_FAST                    ? kFast
                            : choice == MUON_EXACT || (y8 && fused) ? kExact
                                                                    : kMatmul8;
  const Matmul8Plan plan = linear8_plan(out, m, n, g.ld, products);
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

int muon_residual_norm(const void* x, int x_dtype, long long ldx, const void* branch,
                       int branch_dtype, long long ldb, int rows, int cols,
                       const muon_residual_params* params, void* r, long long ldr, void* h,
                       int h_dtype, long long ldh, const muon_tensor8* h8, float* stats,
                       hipStream_t stream) {
  if (!params_ok(params) || !matrix_ok(x, rows, cols, ldx)) return MUON_ERR_INVALID_ARG;
  const int types = types_status(x_dtype, branch ? branch_dtype : x_dtype);
  if (types == MUON_ERR_INVALID_ARG) return types;
  if (branch ? !matrix_ok(branch, rows, cols, ldb) : residual_branch(*params) && rows > 0)
    return MUON_ERR_INVALID_ARG;
  if (r ? !matrix_ok(r, rows, cols, ldr) : (branch || params->scale) && rows > 0)
    return MUON_ERR_INVALID_ARG;
  if ((h != nullptr) == (h8 != nullptr) && !(rows == 0 && !h8)) return MUON_ERR_INVALID_ARG;
  if (h8 ? !tensor8_ok(h8) || h8->rows != rows || h8->cols != cols || h8->block_rows != 1
         : !is_dtype(h_dtype) || !matrix_ok(h, rows, cols, ldh))
    return MUON_ERR_INVALID_ARG;
  if (rows > 0 && (!stats || !aligned(stats, 4))) return MUON_ERR_INVALID_ARG;
  const size_t ex = size_of(x_dtype);
  if (conflict({r ? matrix(r, rows, cols, ldr, ex) : kNone,
                h8 ? data_of(h8) : matrix(h, rows, cols, ldh, size_of(h_dtype)),
                h8 ? scale_of(h8) : kNone, vec_of(stats, 4LL * rows)},
               {matrix(x, rows, cols, ldx, ex),
                branch ? matrix(branch, rows, cols, ldb, size_of(branch_dtype)) : kNone,
                vec_of(params->weight, cols), vec_of(params->bias, cols),
                vec_of(params->post_weight, cols), vec_of(params->post_bias, cols),
                vec_of(params->gate, cols), vec_of(params->scale, 1)}))
    return MUON_ERR_INVALID_ARG;
  if (types != MUON_OK) return types;
  if (cols > MUON_MAX_NORM_COLS) return MUON_ERR_UNSUPPORTED;
  if (rows == 0) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  ResidualArgs a{};
  a.x = x; a.ldx = ldx; a.b = branch; a.ldb = ldb; a.rows = rows; a.cols = cols; a.p = *params;
  a.r = r; a.ldr = ldr; a.h = h; a.h_type = h8 ? kOut8 : h_dtype; a.ldh = ldh;
  if (h8) {
    a.h8 = bytes_of(h8->data); a.s8 = bytes_of(h8->scale);
    a.ld = ld8(cols); a.sld = scale_ld8(cols);
  }
  a.stats = stats;
  const int b_bf16 = branch ? branch_dtype == MUON_BF16 : x_dtype == MUON_BF16;
  const double bytes = (double)rows * cols *
                       ((r ? 2.0 : 1.0) * ex + (branch ? (double)size_of(branch_dtype) : 0.0) +
                        (h8 ? 1.0 : (double)size_of(h_dtype)));
  return status_of(timed_launch(MUON_K_RESIDUAL_NORM, rows, cols, 0.0, 0.0, bytes, stream, [&] {
    return launch_residual_norm(x_dtype == MUON_BF16, b_bf16, a, stream);
  }));
}

size_t muon_residual_norm_backward_workspace_bytes(int rows, int cols, int branch_params) {
  if (rows < 1 || rows > MUON_MAX_ROWS || cols < 1 || cols > MUON_MAX_NORM_COLS ||
      (branch_params != 0 && branch_params != 1))
    return 0;
  // (of either type, which the query does not know)
  const int groups = std::max(residual_back_groups(rows, cols, branch_params, false),
                              residual_back_groups(rows, cols, branch_params, true));
  return scale_parts_bytes(groups) +
         (size_t)groups * (branch_params ? 4 : 2) * (size_t)cols * sizeof(float);
}

int muon_residual_norm_backward(const void* dr, long long lddr, const void* dh, long long lddh,
                                const void* r, long long ldr, const void* branch, long long ldb,
                                const void* x, long long ldx, int x_dtype, int branch_dtype,
                                int rows, int cols, const muon_residual_params* params,
                                const float* stats, void* dx, long long lddx, void* dbranch,
                                long long lddb, const muon_residual_grads* grads, int accumulate,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!params_ok(params) || !grads || (accumulate != 0 && accumulate != 1))
    return MUON_ERR_INVALID_ARG;
  const int types = types_status(x_dtype, branch_dtype);
  if (types == MUON_ERR_INVALID_ARG) return types;
  const bool of_branch = residual_branch(*params);
  if ((dr && !matrix_ok(dr, rows, cols, lddr)) || !matrix_ok(dh, rows, cols, lddh) ||
      !matrix_ok(r, rows, cols, ldr) || !matrix_ok(dx, rows, cols, lddx) ||
      (of_branch && !matrix_ok(branch, rows, cols, ldb)) ||
      (grads->scale && !matrix_ok(x, rows, cols, ldx)) ||
      (dbranch && !matrix_ok(dbranch, rows, cols, lddb)))
    return MUON_ERR_INVALID_ARG;
  if ((grads->post_weight && !params->post_weight) || (grads->post_bias && !params->post_bias) ||
      (grads->gate && !params->gate) || (grads->scale && !params->scale))
    return MUON_ERR_INVALID_ARG;
  for (const float* g : {grads->weight, grads->bias, grads->post_weight, grads->post_bias,
                         grads->gate, grads->scale})
    if (!aligned(g, 4)) return MUON_ERR_INVALID_ARG;
  if (rows > 0 && (!stats || !aligned(stats, 4))) return MUON_ERR_INVALID_ARG;
  const size_t ex = size_of(x_dtype), eb = size_of(branch_dtype);
  const auto span = [&](const void* p, long long ld, size_t es) {
    return p ? matrix(p, rows, cols, ld, es) : kNone;
  };
  const size_t need =
      cols <= MUON_MAX_NORM_COLS ? muon_residual_norm_backward_workspace_bytes(rows, cols, of_branch) : 0;
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, MUON_WORKSPACE_ALIGN)))
    return MUON_ERR_WORKSPACE;
  if (conflict({span(dx, lddx, ex), span(dbranch, lddb, eb), vec_of(grads->weight, cols),
                vec_of(grads->bias, cols), vec_of(grads->post_weight, cols),
                vec_of(grads->post_bias, cols), vec_of(grads->gate, cols), vec_of(grads->scale, 1),
                Span{workspace, need}},
               {span(dr, lddr, ex), span(dh, lddh, eb), span(r, ldr, ex),
                of_branch ? span(branch, ldb, eb) : kNone, grads->scale ? span(x, ldx, ex) : kNone,
                vec_of(stats, 4LL * rows), vec_of(params->weight, cols), vec_of(params->bias, cols),
                vec_of(params->post_weight, cols), vec_of(params->post_bias, cols),
                vec_of(params->gate, cols), vec_of(params->scale, 1)}))
    return MUON_ERR_INVALID_ARG;
  if (types != MUON_OK) return types;
  if (cols > MUON_MAX_NORM_COLS) return MUON_ERR_UNSUPPORTED;
  if (rows == 0 && accumulate) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  ResidualBackArgs a{};
  a.dr = dr; a.lddr = lddr; a.dh = dh; a.lddh = lddh; a.r = r; a.ldr = ldr;
  a.b = branch; a.ldb = ldb; a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols;
  a.p = *params; a.stats = stats; a.dx = dx; a.lddx = lddx; a.db = dbranch; a.lddb = lddb;
  a.g = *grads; a.accumulate = accumulate;
  a.groups = rows > 0 ? residual_back_groups(rows, cols, of_branch, branch_dtype == MUON_FP32) : 0;
  if (need) {
    a.part_scale = static_cast<double*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + scale_parts_bytes(a.groups));
  }
  const double bytes = (double)rows * cols *
                       ((dr ? 3.0 : 2.0) * ex + eb + (of_branch ? eb : 0) + (dbranch ? eb : 0) +
                        (grads->scale ? ex : 0));
  return status_of(timed_launch(
      MUON_K_RESIDUAL_NORM_BACK, rows, cols, 0.0, 0.0, bytes, stream, [&] {
        return launch_residual_norm_backward(x_dtype == MUON_BF16, branch_dtype == MUON_BF16, a,
                                             stream);
      }));
}

}  // extern "C"
