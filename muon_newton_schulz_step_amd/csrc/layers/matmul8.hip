// matmul8: the choice of a kernel and a tile for a plain product, and its launch
// (the kernels: matmul8_kernels.h).
#include "matmul8_kernels.h"

namespace muon {

namespace {
template <int BM, int BN, int WGM, int WGN, typename Y>
void tiles(Matmul8Args a, hipStream_t s) {
  constexpr bool EXACT = std::is_same_v<Y, float>;
  a.tiles_m = (a.m + BM - 1) / BM;
  a.tiles_n = (a.n + BN - 1) / BN;
  // tiles of a column that run side by side on an XCD's 32 CUs
  a.group_m = 6;
  const dim3 grid((unsigned)a.tiles_m * (unsigned)a.tiles_n), block(64 * WGM * WGN);
  // A result larger than the last-level cache is stored past it, which leaves
  // the cache to the operands (16384 x 16384 x 4096, 512 MB: 911 -> 882 us); a
  // smaller one stays there for its reader (8192 x 4096, 64 MB: 108 us, 113
  // stored past).
  if ((double)a.m * a.n * sizeof(Y) > 256.0 * (1 << 20))
    hipLaunchKernelGGL((matmul8_tile_kernel<BM, BN, WGM, WGN, EXACT, true, Y>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((matmul8_tile_kernel<BM, BN, WGM, WGN, EXACT, false, Y>), grid, block, 0, s, a);
}

template <typename Y>
void go(const Matmul8Args& a, const Matmul8Plan& p, hipStream_t s) {
  constexpr bool FP32 = std::is_same_v<Y, float>;
  if (p.few) {
    const dim3 grid((a.n + p.bn - 1) / p.bn), block(64 * kFewWaves);
    if (p.bm == 16 && p.bn == 16)
      hipLaunchKernelGGL((matmul8_rows_kernel<1, 1, Y>), grid, block, 0, s, a);
    else if (p.bm == 16)
      hipLaunchKernelGGL((matmul8_rows_kernel<1, 2, Y>), grid, block, 0, s, a);
    else if (p.bn == 16)
      hipLaunchKernelGGL((matmul8_rows_kernel<2, 1, Y>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((matmul8_rows_kernel<2, 2, Y>), grid, block, 0, s, a);
  } else if (p.bm == 64) {
    tiles<64, 64, 2, 1, Y>(a, s);
  } else if (p.bm == 128) {
    tiles<128, 128, FP32 ? 4 : 2, 2, Y>(a, s);
  } else {
    tiles<256, 256, 4, 2, Y>(a, s);
  }
}
}  // namespace

Matmul8Plan matmul8_plan(int y_bf16, int m, int n, int ld) {
  // Few rows.  32 columns to a workgroup where that leaves 256 workgroups and
  // enough rows share the second half's saving (16 x 8192 x 4096: 11.1 -> 8.7 us,
  // 32 x 8192 x 4096: 16.6 -> 11.7 us; but 1 x 8192 x 8192: 13 -> 20 us, 16 x 8192
  // x 8192: 20 -> 22 us).  Past 16 rows a very wide product is faster in tiles (32
  // x 16384 x 4096: 22.8 -> 17.6 us).  A workgroup of 512 threads for 16 columns
  // reaches the 2^32 threads of a launch at 2^27 columns: tiles from there on.
  if ((m <= 16 && n <= (1 << 26)) || (m <= 32 && n < 16384)) {
    const bool two = n >= 8192 && (m > 16 || (m > 8 && ld <= 4096));
    return {true, m <= 16 ? 16 : 32, two ? 32 : 16};
  }
  // The tile by the time of the fullest CU, in us per k-tile.  Measured, for a
  // result in bf16: 256 x 256 (one per CU) 1.55; 128 x 128 0.72 alone and 0.88 for
  // two; 64 x 64 0.30 alone, and 0.2 for each of several beside 0.1.  (512 x 4096
  // x 4096: 38, 21, 18 us with the three tiles; 2048 x 2048 x 2048: 23.5, 11.6,
  // 14.9 us; 6000 x 2000 x 700: 15.1, 17.5, 21.5 us.)  In fp32: 3.3; 1.1 and 1.8;
  // 0.56, and 0.265 each beside 0.3; its 128 x 128 tiles have 8 waves, which hide
  // the conversions better (2048 x 1280 x 5120: 46.6 -> 37.2 us).  (8192 x 4096 x
  // 4096: 217, 234, 275 us; 1024 x 4096 x 4096: 83, 36.2, 37.3 us; 2048 x 1280 x
  // 1280: 31.6, 13.7, 12.7 us.)  Over 64 sizes of 48 to 16384 rows, 700 to 16384
  // columns and sums of 700 to 5120 the choice is on average within 0.3% of the
  // fastest of the three for either type (worst: 16384 x 5120 x 1280 in fp32,
  // whose stores bound it, 273 us against 232).  A fourth tile of 64 x 128, not
  // here, was faster at some middle sizes: in bf16 by up to 9% (1024 x 4096 x 4096:
  // 25.8 -> 23.7 us), in fp32 by up to 18% (1024 x 1280 x 5120: 31.1 -> 26.3 us); over
  // the 64 sizes the choice is 0.8% and 2.7% off the fastest of all four.
  const bool fp32 = !y_bf16;
  auto share = [&](int bm, int bn) {  // tiles of the fullest CU
    return (double)(((long long)((m + bm - 1) / bm) * ((n + bn - 1) / bn) + 255) / 256);
  };
  const double q256 = share(256, 256), q128 = share(128, 128), q64 = share(64, 64);
  const double odd = (long long)q128 % 2 ? 1.0 : 0.0;
  const double t256 = (fp32 ? 3.3 : 1.55) * q256;
  const double t128 = fp32 ? 0.9 * q128 + 0.2 * odd : 0.44 * q128 + 0.28 * odd;
  const double t64 = fp32 ? 0.3 + 0.265 * q64 : 0.1 + 0.2 * q64;
  const int b = t64 < t128 && t64 < t256 ? 64 : t128 < t256 ? 128 : 256;
  return {false, b, b};
}

hipError_t launch_matmul8(int y_bf16, const Matmul8Args& a, const Matmul8Plan& p, hipStream_t s) {
  if (y_bf16)
    go<bf16_t>(a, p, s);
  else
    go<float>(a, p, s);
  return hipGetLastError();
}

}  // namespace muon
