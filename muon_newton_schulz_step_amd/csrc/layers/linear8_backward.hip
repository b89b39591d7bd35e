// The backward pass of linear8 up to its two gradient products:
//   dz = dy act'(z)  in bf16 and, with a scale per block of 1 x 128, in 8 bits,
//   dbias = sum over the rows of dz.
// One pass over dy and z, bound by HBM: 8192 x 5120 squared ReLU 51.5 us with the
// reduction (5.7 TB/s, some of it from the last-level cache), 60 + 5 us traced with
// cold inputs; GELU 58 us.  A wave has one row in work and one on its way: two or four
// at a time took 54.5 and 59.6 us.
//
// A workgroup of 8 waves has a strip of 512 columns, 8 to a lane, as the
// conversion to 8 bits does (16 lanes hold a block), and a share of the rows: the
// columns' sums stay in registers, are joined in LDS and leave as one partial row
// per workgroup, which a second launch adds in order.
#include "activation.h"
#include "muon_block.h"

namespace muon {

constexpr int kBackWaves = 8;

template <typename D, typename Z>
__global__ __launch_bounds__(64 * kBackWaves) void linear8_back_kernel(Linear8BackArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int piece = blockIdx.x, c = piece * 512 + lane * 8;
  const long long step = (long long)gridDim.y * kBackWaves;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  Raw8<D> rd;
  Raw8<Z> rz;
  auto fetch = [&](long long row) __attribute__((always_inline)) {
    rd.load(static_cast<const D*>(a.dy) + row * a.lddy + c, a.cols - c);
    if (a.act != MUON_ACT_NONE)
      rz.load(static_cast<const Z*>(a.z) + row * a.ldz + c, a.cols - c);
  };
  long long row = (long long)blockIdx.y * kBackWaves + wave;
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += step) {
    float d[8], z[8];
    rd.get(d);
    if (a.act != MUON_ACT_NONE) rz.get(z);
    if (row + step < a.rows) fetch(row + step);
    if (a.act != MUON_ACT_NONE) activate_grad(d, z, a.act);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += d[i];
    if (a.dz) store8_edge(static_cast<bf16_t*>(a.dz) + row * a.lddz + c, a.cols - c, d);
    if (a.q) {
      const int byte = block_units(d, d);
      if (c < a.ld) *reinterpret_cast<u32x2_t*>(a.q + row * a.ld + c) = to_e4m3(d);
      const unsigned word = pack_scales(byte);
      if (lane == 0) *reinterpret_cast<unsigned*>(a.s + row * a.sld + 4 * piece) = word;
    }
  }
  if (!a.dbias) return;
  // column c of the strip: element c % 8 of lane c / 8, rows of 64 padded by one
  constexpr int ROW = 65, PER = 8 * ROW;
  __shared__ float acc[kBackWaves * PER];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[wave * PER + i * ROW + lane] = sum[i];
  __syncthreads();
  const int col = piece * 512 + (int)threadIdx.x;
  if (col >= a.cols) return;
  const int at = (threadIdx.x & 7) * ROW + (threadIdx.x >> 3);
  float s = acc[at];
#pragma unroll
  for (int w = 1; w < kBackWaves; ++w) s += acc[w * PER + at];
  if (a.groups > 1)
    a.part[(long long)blockIdx.y * a.cols + col] = s;
  else
    a.dbias[col] = a.accumulate ? a.dbias[col] + s : s;
}

// dbias from the partial sums, in their order: 32 columns per workgroup, 32
// threads to a column.
__global__ __launch_bounds__(1024) void bias_reduce_kernel(const float* part, int groups, int cols,
                                                           float* dbias, int accumulate) {
  __shared__ float acc[32][33];
  const int x = threadIdx.x & 31, g0 = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + x;
  float s = 0.f;
  if (c < cols)
#pragma unroll 8
    for (int g = g0; g < groups; g += 32) s += part[(long long)g * cols + c];
  acc[g0][x] = s;
  __syncthreads();
  if (g0 == 0 && c < cols) {
    s = 0.f;
#pragma unroll
    for (int g = 0; g < 32; ++g) s += acc[g][x];
    dbias[c] = accumulate ? dbias[c] + s : s;
  }
}

// Workgroups along the rows: at most 512 in all, which the chip holds at once, as few
// as give no wave more rows than that many would, and at least two rows to a wave.
int linear8_back_groups(int rows, int cols) {
  const long long strips = (cols + 511LL) / 512;
  const long long most = strips < 512 ? 512 / strips : 1;
  const long long all = ((long long)rows + kBackWaves - 1) / kBackWaves;  // rows of a wave
  const long long each = (all + most - 1) / most;
  return (int)((all + (each < 2 ? 2 : each) - 1) / (each < 2 ? 2 : each));
}

hipError_t launch_linear8_backward(int dy_fp32, int z_fp32, const Linear8BackArgs& a,
                                   hipStream_t s) {
  if (a.rows > 0) {
    const dim3 grid((a.cols + 511) / 512, a.groups), block(64 * kBackWaves);
    if (dy_fp32) {
      if (z_fp32)
        hipLaunchKernelGGL((linear8_back_kernel<float, float>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((linear8_back_kernel<float, bf16_t>), grid, block, 0, s, a);
    } else {
      if (z_fp32)
        hipLaunchKernelGGL((linear8_back_kernel<bf16_t, float>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((linear8_back_kernel<bf16_t, bf16_t>), grid, block, 0, s, a);
    }
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !a.dbias || a.groups == 1) return err;
  hipLaunchKernelGGL(bias_reduce_kernel, dim3((a.cols + 31) / 32), dim3(1024), 0, s, a.part,
                     a.groups, a.cols, a.dbias, a.accumulate);
  return hipGetLastError();
}

}  // namespace muon
