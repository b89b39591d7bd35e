// Host side of the 8-bit linear layer and layer norm: argument checks (pure
// host code until the last one, so they run on a machine without a GPU),
// workspace sizes and launches.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "muon.h"
#include "muon_checks.h"
#include "muon_layer.h"

using namespace muon;

namespace {

size_t norm_workspace(int rows, int cols) {
  const int groups = norm_backward_groups(rows, cols);
  return groups > 1 ? (size_t)groups * 2 * (size_t)cols * sizeof(float) : 0;
}

}  // namespace

extern "C" {

size_t muon_tensor8_bytes(int rows, int cols) {
  return shape8_ok(rows, cols, 1) ? (size_t)rows * (size_t)ld8(cols) : 0;
}

size_t muon_tensor8_scale_bytes(int rows, int cols, int block_rows) {
  if (!shape8_ok(rows, cols, block_rows)) return 0;
  const size_t blocks = ((size_t)rows + (size_t)block_rows - 1) / (size_t)block_rows;
  return blocks * (size_t)scale_ld8(cols);
}

int muon_quantize8(const void* x, int x_dtype, int rows, int cols, long long ldx,
                   const muon_tensor8* out, const muon_tensor8* transposed, hipStream_t stream) {
  if (!is_dtype(x_dtype) || !matrix_ok(x, rows, cols, ldx) || !tensor8_ok(out))
    return MUON_ERR_INVALID_ARG;
  if (out->rows != rows || out->cols != cols) return MUON_ERR_INVALID_ARG;
  if (transposed) {
    // a transposed tensor of no columns does not exist
    if (rows == 0 || !tensor8_ok(transposed) || transposed->rows != cols ||
        transposed->cols != rows || transposed->block_rows != 128)
      return MUON_ERR_INVALID_ARG;
    if (out->block_rows != 128) return MUON_ERR_UNSUPPORTED;
  }
  const Span none{nullptr, 0};
  if (conflict({data_of(out), scale_of(out), transposed ? data_of(transposed) : none,
                transposed ? scale_of(transposed) : none},
               {matrix(x, rows, cols, ldx, size_of(x_dtype))}))
    return MUON_ERR_INVALID_ARG;
  if (!pieces_fit(rows, cols) || !tiles_fit(rows, cols)) return MUON_ERR_UNSUPPORTED;
  if (rows == 0) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  Quant8Args a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols;
  a.ld = ld8(cols); a.sld = scale_ld8(cols);
  a.q = bytes_of(out->data); a.s = bytes_of(out->scale);
  if (transposed) {
    a.qt = bytes_of(transposed->data); a.st = bytes_of(transposed->scale);
    a.ldt = ld8(rows); a.sldt = scale_ld8(rows);
  }
  const double bytes = (double)rows * cols * (size_of(x_dtype) + (transposed ? 2.0 : 1.0));
  return status_of(timed_launch(MUON_K_QUANT8, rows, cols, 0.0, 0.0, bytes, stream, [&] {
    return out->block_rows == 1 ? launch_quantize8_rows(x_dtype == MUON_BF16, a, stream)
                                : launch_quantize8_blocks(x_dtype == MUON_BF16, a, stream);
  }));
}

int muon_dequantize8(const muon_tensor8* t, void* y, int y_dtype, long long ldy,
                     hipStream_t stream) {
  if (!is_dtype(y_dtype) || !tensor8_ok(t) || !matrix_ok(y, t->rows, t->cols, ldy))
    return MUON_ERR_INVALID_ARG;
  if (conflict({matrix(y, t->rows, t->cols, ldy, size_of(y_dtype))}, {data_of(t), scale_of(t)}))
    return MUON_ERR_INVALID_ARG;
  if (!pieces_fit(t->rows, t->cols)) return MUON_ERR_UNSUPPORTED;
  if (t->rows == 0) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  Dequant8Args a{};
  a.q = bytes_of(t->data); a.s = bytes_of(t->scale);
  a.ld = ld8(t->cols); a.sld = scale_ld8(t->cols);
  a.rows = t->rows; a.cols = t->cols; a.shift = shift_of(t);
  a.y = y; a.ldy = ldy;
  const double bytes = (double)t->rows * t->cols * (1.0 + size_of(y_dtype));
  return status_of(timed_launch(MUON_K_QUANT8, t->rows, t->cols, 0.0, 0.0, bytes, stream,
                                [&] { return launch_dequantize8(y_dtype == MUON_BF16, a, stream); }));
}

int muon_matmul8(const muon_tensor8* a, const muon_tensor8* b, void* y, int y_dtype,
                 long long ldy, hipStream_t stream) {
  if (!is_dtype(y_dtype) || !tensor8_ok(a) || !tensor8_ok(b)) return MUON_ERR_INVALID_ARG;
  if (a->cols != b->cols || ldy < b->rows || ldy > (1LL << 31)) return MUON_ERR_INVALID_ARG;
  if (a->rows == 0 || b->rows == 0) return MUON_OK;
  if (!matrix_ok(y, a->rows, b->rows, ldy)) return MUON_ERR_INVALID_ARG;
  if (conflict({matrix(y, a->rows, b->rows, ldy, size_of(y_dtype))},
               {data_of(a), scale_of(a), data_of(b), scale_of(b)}))
    return MUON_ERR_INVALID_ARG;
  if (!tiles_fit(a->rows, b->rows)) return MUON_ERR_UNSUPPORTED;
  if (int st = check_stream_device(stream)) return st;
  Matmul8Args g{};
  g.a = bytes_of(a->data); g.b = bytes_of(b->data);
  g.sa = bytes_of(a->scale); g.sb = bytes_of(b->scale);
  g.m = a->rows; g.n = b->rows;
  g.ld = (int)ld8(a->cols); g.sld = (int)scale_ld8(a->cols);
  g.shift_a = shift_of(a); g.shift_b = shift_of(b);
  g.y = y; g.ldy = ldy;
  const Matmul8Plan plan = matmul8_plan(y_dtype == MUON_BF16, g.m, g.n, g.ld);
  const double m = g.m, n = g.n, k = a->cols;
  return status_of(timed_launch(
      MUON_K_MATMUL8, g.m, g.n, 2 * m * n * k,
      2 * padded(g.m, plan.bm) * padded(g.n, plan.bn) * g.ld,
      m * k + n * k + m * n * size_of(y_dtype), stream,
      [&] { return launch_matmul8(y_dtype == MUON_BF16, g, plan, stream); }));
}

size_t muon_weight_grad_workspace_bytes(int tokens, int n, int k) {
  if (tokens < 0 || tokens > MUON_MAX_ROWS || n < 1 || n > MUON_MAX_ROWS || k < 1 ||
      k > MUON_MAX_COLS8)
    return 0;
  const int splits = weight_grad_plan(tokens, n, k).splits;
  return splits > 1 ? (size_t)splits * (size_t)n * (size_t)k * sizeof(float) : 0;
}

int muon_weight_grad(const void* dy, int dy_dtype, long long lddy, int tokens, int n,
                     const muon_tensor8* x, void* dw, int dw_dtype, int accumulate,
                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!is_dtype(dy_dtype) || !is_dtype(dw_dtype) || (accumulate != 0 && accumulate != 1))
    return MUON_ERR_INVALID_ARG;
  if (!matrix_ok(dy, tokens, n, lddy) || !tensor8_ok(x) || x->rows != tokens ||
      !matrix_ok(dw, n, x->cols, x->cols))
    return MUON_ERR_INVALID_ARG;
  const Span out = matrix(dw, n, x->cols, x->cols, size_of(dw_dtype));
  const Span in = matrix(dy, tokens, n, lddy, size_of(dy_dtype));
  if (conflict({out}, {in, data_of(x), scale_of(x)})) return MUON_ERR_INVALID_ARG;
  // (the kernel reaches the rows of a tile with 32-bit offsets)
  if (dy_dtype != MUON_BF16 || (accumulate && dw_dtype != MUON_FP32) || !tiles_fit(n, x->cols) ||
      lddy > (1LL << 26))
    return MUON_ERR_UNSUPPORTED;
  const size_t need = muon_weight_grad_workspace_bytes(tokens, n, x->cols);
  if (need) {
    if (!workspace || workspace_bytes < need || !aligned(workspace, MUON_WORKSPACE_ALIGN))
      return MUON_ERR_WORKSPACE;
    if (conflict({Span{workspace, need}}, {in, out, data_of(x), scale_of(x)}))
      return MUON_ERR_INVALID_ARG;
  }
  if (tokens == 0 && accumulate) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  WeightGradArgs g{};
  g.dy = dy; g.lddy = lddy;
  g.x = bytes_of(x->data); g.sx = bytes_of(x->scale);
  g.tokens = tokens; g.n = n; g.k = x->cols;
  g.ld = (int)ld8(x->cols); g.sld = (int)scale_ld8(x->cols); g.shift = shift_of(x);
  g.dw = dw; g.accumulate = accumulate;
  const WeightGradPlan plan = weight_grad_plan(tokens, n, x->cols);
  g.part = need ? static_cast<float*>(workspace) : nullptr;
  const double t = tokens, k = x->cols;
  return status_of(timed_launch(
      MUON_K_WEIGHT_GRAD, n, x->cols, 2 * t * n * k,
      2 * padded(tokens, kTileT) * padded(n, plan.bn) * padded(x->cols, plan.bk),
      2 * t * n + t * k + n * k * size_of(dw_dtype) * (accumulate ? 2 : 1), stream,
      [&] { return launch_weight_grad(dw_dtype == MUON_BF16, g, plan, stream); }));
}

int muon_layer_norm(const void* x, int x_dtype, long long ldx, int rows, int cols,
                    const float* weight, const float* bias, float eps, void* y, int y_dtype,
                    long long ldy, const muon_tensor8* y8, float* mean, float* rstd,
                    hipStream_t stream) {
  if (!is_dtype(x_dtype) || !matrix_ok(x, rows, cols, ldx)) return MUON_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return MUON_ERR_INVALID_ARG;
  if (!weight || !aligned(weight, 4) || !aligned(bias, 4)) return MUON_ERR_INVALID_ARG;
  if ((y != nullptr) == (y8 != nullptr) && !(rows == 0 && !y8)) return MUON_ERR_INVALID_ARG;
  const size_t vec = (size_t)cols * 4, per_row = (size_t)(rows > 0 ? rows : 0) * 4;
  if (rows > 0 && (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)))
    return MUON_ERR_INVALID_ARG;
  Span out{nullptr, 0}, out_s{nullptr, 0};
  if (y8) {
    if (!tensor8_ok(y8) || y8->rows != rows || y8->cols != cols || y8->block_rows != 1)
      return MUON_ERR_INVALID_ARG;
    out = data_of(y8);
    out_s = scale_of(y8);
  } else {
    if (!is_dtype(y_dtype) || !matrix_ok(y, rows, cols, ldy)) return MUON_ERR_INVALID_ARG;
    out = matrix(y, rows, cols, ldy, size_of(y_dtype));
  }
  if (conflict({out, out_s, Span{mean, per_row}, Span{rstd, per_row}},
               {matrix(x, rows, cols, ldx, size_of(x_dtype)), Span{weight, vec}, Span{bias, vec}}))
    return MUON_ERR_INVALID_ARG;
  if (cols > MUON_MAX_NORM_COLS) return MUON_ERR_UNSUPPORTED;
  if (rows == 0) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  NormArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols;
  a.weight = weight; a.bias = bias; a.eps = eps;
  a.y = y; a.ldy = ldy;
  if (y8) {
    a.y8 = bytes_of(y8->data); a.s8 = bytes_of(y8->scale);
    a.ld = ld8(cols); a.sld = scale_ld8(cols);
  }
  a.mean = mean; a.rstd = rstd;
  const double bytes = (double)rows * cols * (size_of(x_dtype) + (y8 ? 1.0 : size_of(y_dtype)));
  return status_of(timed_launch(MUON_K_LAYER_NORM, rows, cols, 0.0, 0.0, bytes, stream, [&] {
    return launch_layer_norm(x_dtype == MUON_BF16, y8 ? 2 : y_dtype, a, stream);
  }));
}

size_t muon_layer_norm_backward_workspace_bytes(int rows, int cols) {
  if (rows < 1 || rows > MUON_MAX_ROWS || cols < 1 || cols > MUON_MAX_NORM_COLS) return 0;
  return norm_workspace(rows, cols);
}

int muon_layer_norm_backward(const void* dy, int dy_dtype, long long lddy, const void* x,
                             int x_dtype, long long ldx, const muon_tensor8* x8, int rows,
                             int cols, const float* weight, const float* mean,
                             const float* rstd, void* dx, long long lddx, float* dweight,
                             float* dbias, int accumulate, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  if (!is_dtype(dy_dtype) || !matrix_ok(dy, rows, cols, lddy) || !matrix_ok(dx, rows, cols, lddx))
    return MUON_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MUON_ERR_INVALID_ARG;
  if ((x != nullptr) == (x8 != nullptr) && !(rows == 0 && !x8)) return MUON_ERR_INVALID_ARG;
  if (!weight || !dweight || !aligned(weight, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
    return MUON_ERR_INVALID_ARG;
  if (rows > 0 && (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)))
    return MUON_ERR_INVALID_ARG;
  Span in{nullptr, 0}, in_s{nullptr, 0};
  if (x8) {
    if (!tensor8_ok(x8) || x8->rows != rows || x8->cols != cols) return MUON_ERR_INVALID_ARG;
    in = data_of(x8);
    in_s = scale_of(x8);
  } else {
    if (!is_dtype(x_dtype) || !matrix_ok(x, rows, cols, ldx)) return MUON_ERR_INVALID_ARG;
    in = matrix(x, rows, cols, ldx, size_of(x_dtype));
  }
  const size_t vec = (size_t)cols * 4, per_row = (size_t)rows * 4, es = size_of(dy_dtype);
  const Span s_dy = matrix(dy, rows, cols, lddy, es), s_dx = matrix(dx, rows, cols, lddx, es);
  if (conflict({s_dx, Span{dweight, vec}, Span{dbias, vec}},
               {s_dy, in, in_s, Span{weight, vec}, Span{mean, per_row}, Span{rstd, per_row}}))
    return MUON_ERR_INVALID_ARG;
  if (cols > MUON_MAX_NORM_COLS) return MUON_ERR_UNSUPPORTED;
  if (const size_t need = norm_workspace(rows, cols)) {
    if (!workspace || workspace_bytes < need || !aligned(workspace, MUON_WORKSPACE_ALIGN))
      return MUON_ERR_WORKSPACE;
    if (conflict({Span{workspace, need}},
                 {s_dy, s_dx, in, in_s, Span{weight, vec}, Span{mean, per_row}, Span{rstd, per_row},
                  Span{dweight, vec}, Span{dbias, vec}}))
      return MUON_ERR_INVALID_ARG;
  }
  if (rows == 0 && accumulate) return MUON_OK;
  if (int st = check_stream_device(stream)) return st;
  NormBackArgs a{};
  a.dy = dy; a.lddy = lddy; a.x = x; a.ldx = ldx;
  if (x8) {
    a.x8 = bytes_of(x8->data); a.sx8 = bytes_of(x8->scale);
    a.ld = ld8(cols); a.sld = scale_ld8(cols); a.shift = shift_of(x8);
  }
  a.rows = rows; a.cols = cols; a.weight = weight; a.mean = mean; a.rstd = rstd;
  a.dx = dx; a.lddx = lddx; a.dweight = dweight; a.dbias = dbias; a.accumulate = accumulate;
  a.part = static_cast<float*>(workspace);
  a.groups = norm_backward_groups(rows, cols);
  const double bytes =
      (double)rows * cols * (2.0 * es + (x8 ? 1.0 : (double)size_of(x_dtype)));
  return status_of(timed_launch(
      MUON_K_LAYER_NORM_BACK, rows, cols, 0.0, 0.0, bytes, stream, [&] {
        return launch_layer_norm_backward(dy_dtype == MUON_BF16, x8 ? 2 : x_dtype, a, stream);
      }));
}

}  // extern "C"
