// linear8: the product with an epilogue, its choice of a kernel and a tile, and
// its launch (the kernels: matmul8_kernels.h).
#include "matmul8_kernels.h"

namespace muon {

namespace {
constexpr int kOut8 = 2;

// Rounding to 8 bits turns a product's error of relative size e into flips of a whole
// step, 2^-4, for a share e / 2^-4 of the values: sqrt(e 2^-4) in the norm.  The 8-bit
// instruction's cut leaves e near 1e-4 where a few columns of a are 64 times the others,
// and more where the sum is short and few of them share it.  A hidden layer in 8 bits was
// off from that of exact products by 1.7e-3 to 2.2e-3 of its norm with every activation
// and 2.3e-3 to 2.8e-3 with the squared ReLU, which doubles e (4096 x 1280, 600 x 700, 2000
// x 528, 1024 x 4096, those columns 1% of all), an MLP's result by 2.4e-3 to 3.7e-3
// and, of 200 rows of 128, 6.2e-3 where with exact products its rounding to bf16 leaves
// 1.7e-3.  So 8-bit results come from exact products unless their caller chose speed
// (fast): the up projection of an MLP with z kept takes 59 us instead of 44 (4096 x
// 5120 x 1280) and 1722 instead of 1004 (16384 x 16384 x 4096).
//
// A plain product in 8 bits, without bias, activation, residual and z, is muon_matmul8's
// with its result rounded once more, cut as that is, but where exact products cost
// little: 99 us against 74 (8192 x 8192 x 512), 26 against 20 (8192 x 2048 x 512), 14
// against 12 (512 x 5120 x 1280).
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
  } else if (p.exact) {
    if (p.bm == 64 && p.bn == 128)
      tiles<64, 128, 2, 2, true, Y>(a, s);
    else if (p.bm == 128)
      tiles<128, 128, 4, 2, true, Y>(a, s);
    else if (p.bm == 256)
      tiles<256, 256, 4, 2, true, Y>(a, s);
    else if constexpr (!is8<Y>)
      tiles<64, 64, 2, 1, true, Y>(a, s);
  } else if constexpr (!std::is_same_v<Y, float>) {
    if (p.bm == 128)
      tiles<128, 128, 2, 2, false, Y>(a, s);
    else if (p.bm == 256)
      tiles<256, 256, 4, 2, false, Y>(a, s);
    else if constexpr (is8<Y>)
      tiles<64, 128, 2, 2, false, Y>(a, s);
    else
      tiles<64, 64, 2, 1, false, Y>(a, s);
  }
}
}  // namespace

// The tile by the time of the fullest CU per k-tile, in us, as for the plain product,
// with one of 64 x 128 beside the others for results in fp32 and 8 bits: of those a CU
// holds three, which fill the last round of a middle-sized grid better.  Measured at
// 100 to 16384 rows, 768 to 5120 columns and sums of 700 to 5120 (in us; fp32 with a
// residual, 8 bits with z kept, of cut products):
//   fp32    4099 x 1280 x 5120 65.4 -> 57.7, 1027 x 5120 x 1280 25.2 -> 21.4, 300 x 4096
//           x 4096 27.2 -> 22.5; but 16384 x 1280 x 5120 184 against 193
//   8 bits  600 x 1280 x 5120 33.3 -> 26.5, 4099 x 768 x 3080 23.6 -> 20.2; but 2048 x
//           4096 x 4096 35.4 against 52.6.  Exact, the fastest of the three or within 3% at
//           14 sizes of 1024 to 16384 rows: 1200 x 5000 x 1300 23.8 (128: 25.7, 256: 40.2),
//           4096 x 5120 x 1280 58 (62, 78), 16384 x 16384 x 4096 1640 (1977, 1850)
// In bf16 it gains at few sizes (4099 x 768 x 3080 21.8 -> 18.7) and is not taken, but
// for exact products, whose costs are those of a result in fp32.
Matmul8Plan linear8_plan(int out, int m, int n, int ld, Products products) {
  bool exact = products == kExact;
  auto share = [&](int bm, int bn) {  // tiles of the fullest CU
    return (double)(((long long)((m + bm - 1) / bm) * ((n + bn - 1) / bn) + 255) / 256);
  };
  const double q64 = share(64, 64), q96 = share(64, 128), q128 = share(128, 128);
  const double odd = (long long)q128 % 2 ? 1.0 : 0.0;
  // exact products
  const double e64 = 0.2 + 0.25 * q64, e96 = 0.08 + 0.44 * q96;
  const double e128 = (q128 <= 2 ? 0.77 : 0.87) * q128;
  if (out != kOut8) {
    exact = exact || out == MUON_FP32;
    Matmul8Plan p = matmul8_plan(!exact, m, n, ld);
    if (exact && !p.few && p.bm <= 128 && e96 < (p.bm == 64 ? e64 : e128)) p = {false, 64, 128};
    p.exact = exact;
    return p;
  }
  // An 8-bit result needs whole blocks of 128 columns in a workgroup.
  if (m <= 32) return {true, m <= 16 ? 16 : 32, 128};
  const double q256 = share(256, 256);
  if (products == kMatmul8) exact = exact8(m, ld);
  const double t96 = exact ? e96 : 0.1 + 0.3 * q96;
  const double t128 = exact ? e128 : 0.44 * q128 + 0.28 * odd;
  const double t256 = exact ? 3.3 * q256 : 1.55 * q256;
  if (t96 < t128 && t96 < t256) return {false, 64, 128, exact};
  return t128 < t256 ? Matmul8Plan{false, 128, 128, exact} : Matmul8Plan{false, 256, 256, exact};
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
