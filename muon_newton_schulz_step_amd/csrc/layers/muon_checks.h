// Argument checks that the host sides of the entry points share: pure host code.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "muon.h"
#include "muon_layer.h"

namespace muon {

inline bool is_dtype(int d) { return d == MUON_BF16 || d == MUON_FP32; }
inline size_t size_of(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Span {
  const void* p;
  size_t bytes;
};
// rows of `cols` elements, `ld` apart
inline Span matrix(const void* p, int rows, int cols, long long ld, size_t es) {
  return {p, rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es : 0};
}
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}
// A written range meets another written one, or one that is read.
inline bool conflict(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (auto w = written.begin(); w != written.end(); ++w) {
    for (auto o = w + 1; o != written.end(); ++o)
      if (overlap(*w, *o)) return true;
    for (const Span& r : read)
      if (overlap(*w, r)) return true;
  }
  return false;
}

inline bool shape8_ok(int rows, int cols, int block_rows) {
  return rows >= 0 && rows <= MUON_MAX_ROWS && cols >= 1 && cols <= MUON_MAX_COLS8 && (block_rows == 1 || block_rows == 128);
}
// A matrix operand: sizes, stride, pointer.  Its rows must have a byte range
// that a signed 64-bit offset reaches, which any real allocation has.
inline bool matrix_ok(const void* p, int rows, int cols, long long ld) {
  return rows >= 0 && rows <= MUON_MAX_ROWS && cols >= 1 && cols <= MUON_MAX_ROWS && ld >= cols &&
         ld <= (1LL << 31) &&
         (rows == 0 || (p && aligned(p, MUON_PTR_ALIGN)));
}
inline bool tensor8_ok(const muon_tensor8* t) {
  return t && shape8_ok(t->rows, t->cols, t->block_rows) &&
         (t->rows == 0 ||
          (t->data && t->scale && aligned(t->data, MUON_PTR_ALIGN) && aligned(t->scale, 4)));
}
inline Span data_of(const muon_tensor8* t) { return {t->data, muon_tensor8_bytes(t->rows, t->cols)}; }
inline Span scale_of(const muon_tensor8* t) {
  return {t->scale, muon_tensor8_scale_bytes(t->rows, t->cols, t->block_rows)};
}
inline unsigned char* bytes_of(void* p) { return static_cast<unsigned char*>(p); }
inline int shift_of(const muon_tensor8* t) { return t->block_rows == 128 ? 7 : 0; }
// Pieces of 512 columns, the element-wise kernels' unit of work, have 16 threads
// each, and a launch has less than 2^32.  Tiles are counted in 32 bits.
inline bool pieces_fit(int rows, int cols) {
  return (double)rows * (double)((cols + 511LL) / 512) <= 268435440.0;
}
inline bool tiles_fit(long long rows, long long cols) {
  return (double)((rows + 63) / 64) * (double)((cols + 63) / 64) < 2147483648.0;
}
// A size in whole tiles, for the flops that a launch executes.
inline double padded(long long size, int tile) { return (double)((size + tile - 1) / tile * tile); }
inline int status_of(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_ERR_HIP; }

}  // namespace muon
