// linear8: the product with an epilogue, its choice of a kernel and a tile, and
// its launch (the kernels: matmul8_kernels.h).
#include "matmul8_kernels.h"

namespace muon {

namespace {
constexpr int kOut8 = 2;

// Whether an 8-bit result comes from exact products.  Rounding to 8 bits turns an
// error of relative size e into flips of a whole step, 2^-4, for a share e / 2^-4 of the
// values: sqrt(e 2^-4) in the norm.  The 8-bit instruction's cut leaves e near 1e-4
// where a few columns of a are 64 times the others, and more where the sum is short
// and few of them share it: an MLP's result (squared ReLU, those columns 1% of all) was
// off by 6.2e-3 of its norm for 200 rows of 128, 5.6e-3 for 60 of 520, 3 to 3.7e-3 for
// thousands of rows and 520 or more columns; with exact products by 1.7e-3, what its
// rounding to bf16 does.  Exact costs 99 us against 74 (8192 x 8192 x 512), 26 against
// 20 (8192 x 2048 x 512), 14 against 12 (512 x 5120 x 1280), but 62 against 35 at 512 x
// 16384 x 4096.
bool exact8(int m, int ld) { return ld <= 512 || (m <= 512 && ld <= 1280); }

template <int BM, int BN, int WGM, int WGN, bool EXACT, typename Y>
void tiles(Linear8Args a, hipStream_t s) {
  a.tiles_m = (a.m + BM - 1) / BM;
  a.tiles_n = (a.n + BN - 1) / BN;
  a.group_m = 6;  // as for the plain product
  const dim3 grid((unsigned)a.tiles_m * (unsigned)a.tiles_n), block(64 * WGM * WGN);
  // results larger than the last-level cache are stored past it, as there
  const double bytes = (double)a.m * a.n * (sizeof(Y) + (a.z ? sizeof(KeptOf<Y>) : 0));
  if (bytes > 256.0 * (1 << 20))
    hipLaunchKernelGGL((matmul8_tile_kernel<BM, BN, WGM, WGN, EXACT, true, Y, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((matmul8_tile_kernel<BM, BN, WGM, WGN, EXACT, false, Y, true>), grid, block, 0, s, a);
}

template <typename Y>
void go(const Linear8Args& a, const Matmul8Plan& p, hipStream_t s) {
  constexpr bool FP32 = std::is_same_v<Y, float>;
  if (p.few) {
    const dim3 grid((a.n + p.bn - 1) / p.bn), block(64 * kFewWaves);
    if constexpr (is8<Y>) {
      if (p.bm == 16)
        hipLaunchKernelGGL((matmul8_rows_kernel<1, 8, Y, true>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((matmul8_rows_kernel<2, 8, Y, true>), grid, block, 0, s, a);
    } else {
      if (p.bm == 16 && p.bn == 16)
        hipLaunchKernelGGL((matmul8_rows_kernel<1, 1, Y, true>), grid, block, 0, s, a);
      else if (p.bm == 16)
        hipLaunchKernelGGL((matmul8_rows_kernel<1, 2, Y, true>), grid, block, 0, s, a);
      else if (p.bn == 16)
        hipLaunchKernelGGL((matmul8_rows_kernel<2, 1, Y, true>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((matmul8_rows_kernel<2, 2, Y, true>), grid, block, 0, s, a);
    }
  } else if (p.bm == 64) {
    if constexpr (!is8<Y>) tiles<64, 64, 2, 1, FP32, Y>(a, s);
  } else if (is8<Y> && exact8(a.m, a.ld)) {
    if constexpr (is8<Y>) {
      if (p.bm == 128)
        tiles<128, 128, 4, 2, true, Y>(a, s);
      else
        tiles<256, 256, 4, 2, true, Y>(a, s);
    }
  } else if (p.bm == 128) {
    tiles<128, 128, FP32 ? 4 : 2, 2, FP32, Y>(a, s);
  } else {
    tiles<256, 256, 4, 2, FP32, Y>(a, s);
  }
}
}  // namespace

Matmul8Plan linear8_plan(int out, int m, int n, int ld) {
  if (out != kOut8) return matmul8_plan(out == MUON_BF16, m, n, ld);
  // An 8-bit result needs whole blocks of 128 columns in a workgroup.
  if (m <= 32) return {true, m <= 16 ? 16 : 32, 128};
  // the costs of the plain product's tiles
  auto share = [&](int b) {
    return (double)(((long long)((m + b - 1) / b) * ((n + b - 1) / b) + 255) / 256);
  };
  const double q128 = share(128), q256 = share(256), odd = (long long)q128 % 2 ? 1.0 : 0.0;
  const bool small = exact8(m, ld) ? 0.9 * q128 + 0.2 * odd < 3.3 * q256
                                : 0.44 * q128 + 0.28 * odd < 1.55 * q256;
  const int b = small ? 128 : 256;
  return {false, b, b};
}

hipError_t launch_linear8(int out, const Linear8Args& a, const Matmul8Plan& p, hipStream_t s) {
  if (out == kOut8)
    go<unsigned char>(a, p, s);
  else if (out == MUON_BF16)
    go<bf16_t>(a, p, s);
  else
    go<float>(a, p, s);
  return hipGetLastError();
}

}  // namespace muon
