// 8-bit tensors: e4m3 values with one power-of-two scale per block of
// 1 x 128 or 128 x 128, written from and read back as bf16 or fp32.
// All three kernels move each byte once and are bound by HBM: 8192 x 5120 bf16
// to 8 bits in 26.6 us and back in 19.8 us (4.7 and 6.3 TB/s, the latter's input
// partly from the last-level cache; a 1 GiB copy runs at 5.2); with the transposed
// copy 4096 x 16384 bf16 in 55.6 us and fp32 in 83.6 us (4.8 TB/s).  Small weights
// are short of that: 1280 x 5120 has 400 blocks and takes 11 us in either type.
#include "fp8_device.h"
#include "muon_layer.h"

namespace muon {

// Blocks of one row: a wave takes 512 columns of a row, 8 per lane, so the
// 16 lanes of a DPP row hold one block and the wave's four scales are one
// aligned word.  Each wave does kItems such pieces, loaded together.
constexpr int kItems = 4;

template <typename T>
__global__ __launch_bounds__(256) void quantize8_rows_kernel(Quant8Args a, unsigned pieces,
                                                             unsigned per_row) {
  const int lane = threadIdx.x & 63;
  const unsigned first =
      (unsigned)__builtin_amdgcn_readfirstlane((blockIdx.x * 4 + (threadIdx.x >> 6)) * kItems);
  float v[kItems][8];
  static_for<kItems>([&](auto u) {
    const unsigned p = first + u;
    if (p < pieces) {
      const unsigned row = p / per_row;
      const int c = (int)(p - row * per_row) * 512 + lane * 8;
      load8_edge(static_cast<const T*>(a.x) + (long long)row * a.ldx + c, a.cols - c, v[u]);
    }
  });
  static_for<kItems>([&](auto u) {
    const unsigned p = first + u;
    if (p < pieces) {
      const unsigned row = p / per_row, piece = p - row * per_row;
      const int c = (int)piece * 512 + lane * 8;
      unsigned top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned f = finite_bits(v[u][i]);
        top = top > f ? top : f;
      }
      const int byte = scale_byte(max16(top));
      float w[8];
      to_units(v[u], byte, w);
      if (c < a.ld) *reinterpret_cast<u32x2_t*>(a.q + (long long)row * a.ld + c) = to_e4m3(w);
      const unsigned word = pack_scales(byte);
      if (lane == 0)
        *reinterpret_cast<unsigned*>(a.s + (long long)row * a.sld + 4 * piece) = word;
    }
  });
}

// Blocks of 128 x 128: one workgroup each, thread t holding rows
// 8 (t / 16) + i and columns 8 (t % 16) + j.  The transposed copy has the same
// values and scales with the two axes exchanged; it goes through LDS so that
// both copies are written in whole 128-byte rows.
template <typename T, bool TRANS>
__global__ __launch_bounds__(256) void quantize8_blocks_kernel(Quant8Args a, int blocks_c) {
  __shared__ unsigned tops[4];
  __shared__ __attribute__((aligned(16))) unsigned char tile[TRANS ? 128 * 144 : 16];
  const int tid = threadIdx.x;
  const int rb = (int)(blockIdx.x / (unsigned)blocks_c), cb = (int)(blockIdx.x % (unsigned)blocks_c);
  const int r0 = rb * 128 + (tid >> 4) * 8, c0 = cb * 128 + (tid & 15) * 8;
  float v[8][8];
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8_edge(static_cast<const T*>(a.x) + (long long)(r0 + i) * a.ldx + c0,
               r0 + i < a.rows ? a.cols - c0 : 0, v[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned f = finite_bits(v[i][j]);
      top = top > f ? top : f;
    }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const unsigned o = (unsigned)__shfl_xor((int)top, d);
    top = top > o ? top : o;
  }
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  top = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = top > tops[w] ? top : tops[w];
  const int byte = scale_byte(top);
  unsigned q[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float w[8];
    to_units(v[i], byte, w);
    const u32x2_t o = to_e4m3(w);
    q[i][0] = o[0];
    q[i][1] = o[1];
    if (r0 + i < a.rows)
      *reinterpret_cast<u32x2_t*>(a.q + (long long)(r0 + i) * a.ld + c0) = o;
  }
  // the last block of a row of scales also writes its padding (as blocks of
  // zeros, like the other kernel), so that equal tensors are equal byte by byte
  auto put = [](unsigned char* row, int i, int blocks, long long sld, int v) {
    row[i] = (unsigned char)v;
    if (i == blocks - 1)
      for (int j = blocks; j < sld; ++j) row[j] = (unsigned char)scale_byte(0u);
  };
  if (tid == 0) put(a.s + (long long)rb * a.sld, cb, blocks_c, a.sld, byte);
  if constexpr (TRANS) {
    if (tid == 0) put(a.st + (long long)cb * a.sldt, rb, (a.rows + 127) / 128, a.sldt, byte);
    // column j of the thread's 8 x 8 bytes: 8 rows, one LDS word pair
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u32x2_t col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unsigned w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= ((q[4 * h + i][j >> 2] >> (8 * (j & 3))) & 0xffu) << (8 * i);
        col[h] = w;
      }
      *reinterpret_cast<u32x2_t*>(tile + ((tid & 15) * 8 + j) * 144 + (tid >> 4) * 8) = col;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int u = tid + 256 * s, c = u >> 3, ch = u & 7;
      if (cb * 128 + c < a.cols)
        *reinterpret_cast<u32x4_t*>(a.qt + (long long)(cb * 128 + c) * a.ldt + rb * 128 + ch * 16) =
            *reinterpret_cast<const u32x4_t*>(tile + c * 144 + ch * 16);
    }
  }
}

// Back to bf16 or fp32 (every value is exact in both): 8 elements per lane.
template <typename T>
__global__ __launch_bounds__(256) void dequantize8_kernel(Dequant8Args a, unsigned pieces,
                                                          unsigned per_row) {
  const int lane = threadIdx.x & 63;
  const unsigned first =
      (unsigned)__builtin_amdgcn_readfirstlane((blockIdx.x * 4 + (threadIdx.x >> 6)) * kItems);
  u32x2_t q[kItems];
  int byte[kItems];
  static_for<kItems>([&](auto u) {
    const unsigned p = first + u;
    q[u] = u32x2_t{0u, 0u};
    byte[u] = 127;
    if (p < pieces) {
      const unsigned row = p / per_row;
      const int c = (int)(p - row * per_row) * 512 + lane * 8;
      if (c < a.ld) {
        q[u] = *reinterpret_cast<const u32x2_t*>(a.q + (long long)row * a.ld + c);
        byte[u] = a.s[(long long)(row >> a.shift) * a.sld + (c >> 7)];
      }
    }
  });
  static_for<kItems>([&](auto u) {
    const unsigned p = first + u;
    if (p < pieces) {
      const unsigned row = p / per_row;
      const int c = (int)(p - row * per_row) * 512 + lane * 8;
      float v[8];
      from_e4m3(q[u], scale_of(byte[u]), v);
      store8_edge(static_cast<T*>(a.y) + (long long)row * a.ldy + c, a.cols - c, v);
    }
  });
}

namespace {
// Pieces of 512 columns; the host checks that their number fits 32 bits.
unsigned pieces_of(int rows, long long ld, unsigned* per_row) {
  *per_row = (unsigned)((ld + 511) / 512);
  return (unsigned)rows * *per_row;
}
dim3 piece_grid(unsigned pieces) { return dim3((pieces + 4 * kItems - 1) / (4 * kItems)); }
}  // namespace

hipError_t launch_quantize8_rows(int x_bf16, const Quant8Args& a, hipStream_t s) {
  unsigned per_row;
  const unsigned pieces = pieces_of(a.rows, a.ld, &per_row);
  if (x_bf16)
    hipLaunchKernelGGL(quantize8_rows_kernel<bf16_t>, piece_grid(pieces), dim3(256), 0, s, a,
                       pieces, per_row);
  else
    hipLaunchKernelGGL(quantize8_rows_kernel<float>, piece_grid(pieces), dim3(256), 0, s, a,
                       pieces, per_row);
  return hipGetLastError();
}

hipError_t launch_quantize8_blocks(int x_bf16, const Quant8Args& a, hipStream_t s) {
  const int bc = (a.cols + 127) / 128, br = (a.rows + 127) / 128;
  const dim3 grid((unsigned)bc * (unsigned)br), block(256);
  if (x_bf16) {
    if (a.qt)
      hipLaunchKernelGGL((quantize8_blocks_kernel<bf16_t, true>), grid, block, 0, s, a, bc);
    else
      hipLaunchKernelGGL((quantize8_blocks_kernel<bf16_t, false>), grid, block, 0, s, a, bc);
  } else {
    if (a.qt)
      hipLaunchKernelGGL((quantize8_blocks_kernel<float, true>), grid, block, 0, s, a, bc);
    else
      hipLaunchKernelGGL((quantize8_blocks_kernel<float, false>), grid, block, 0, s, a, bc);
  }
  return hipGetLastError();
}

hipError_t launch_dequantize8(int y_bf16, const Dequant8Args& a, hipStream_t s) {
  unsigned per_row;
  const unsigned pieces = pieces_of(a.rows, a.ld, &per_row);
  if (y_bf16)
    hipLaunchKernelGGL(dequantize8_kernel<bf16_t>, piece_grid(pieces), dim3(256), 0, s, a, pieces,
                       per_row);
  else
    hipLaunchKernelGGL(dequantize8_kernel<float>, piece_grid(pieces), dim3(256), 0, s, a, pieces,
                       per_row);
  return hipGetLastError();
}

}  // namespace muon
