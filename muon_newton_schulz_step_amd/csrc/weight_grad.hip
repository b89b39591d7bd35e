// The weight gradient of a linear layer from the 8-bit activation that the
// forward pass kept:
//   dw[n][k] (+)= sum_t dy[t][n] x[t][k],   x = q 2^e(t, k / 128)
// x is brought back to bf16 on its way into LDS, which is exact (4 significant
// bits and a power of two), and the product runs on the bf16 MFMA with fp32
// sums.  dy stays bf16: the result goes into Newton-Schulz, which raises a
// gradient's small singular values, and with them the noise that rounding dy
// to 8 bits would spread over all directions.
//
// Both operands hold the summed axis t in rows, so both are read from LDS with
// the transposing read.  Few output tiles and many tokens (a small matrix)
// are split over the tokens; the parts are added in their order by a second
// kernel, so the result does not change from run to run.
#include "muon_gemm.h"

#include "fp8_device.h"
#include "muon_layer.h"

namespace muon {

constexpr int kTileT = 64;  // tokens per LDS tile

template <int BN, int BK, int WGN, int WGK, typename W>
__global__ __launch_bounds__(64 * WGN * WGK) void weight_grad_kernel(WeightGradArgs g) {
  constexpr int NT = 64 * WGN * WGK;
  constexpr int WTN = BN / WGN, WTK = BK / WGK;
  constexpr int FN = WTN / 32, FK = WTK / 32;
  constexpr int UN = BN / 8, UK = BK / 8;          // chunks of 8 per token row
  constexpr int PN = kTileT * UN / NT, PK = kTileT * UK / NT;
  static_assert(PN * NT == kTileT * UN && PK * NT == kTileT * UK, "chunks split over the threads");
  __shared__ u32x4_t lds[2][kTileT * (UN + UK)];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave / WGK, wk = wave % WGK;
  const int L = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int tiles = g.tiles_n * g.tiles_k;
  const int split = L / tiles, tile = L - split * tiles;
  const int n0 = tile / g.tiles_k * BN, k0 = tile % g.tiles_k * BK;
  const int t_first = split * g.tiles_per_split;
  const int t_all = (g.tokens + kTileT - 1) / kTileT;
  const int t_end = t_first + g.tiles_per_split < t_all ? t_first + g.tiles_per_split : t_all;

  u32x4_t rd[PN];
  u32x2_t rx[PK];
  int sx[PK];
  auto gload = [&](int kt) {
#pragma unroll
    for (int i = 0; i < PN; ++i) {
      const int q = tid + NT * i, t = kt * kTileT + q / UN, n = n0 + q % UN * 8;
      const bf16_t* p = static_cast<const bf16_t*>(g.dy) + (long long)t * g.lddy + n;
      rd[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (t < g.tokens) {
        if (n + 8 <= g.n) {
          __builtin_memcpy(&rd[i], p, 16);
        } else {
          float v[8];
          load8_edge(p, g.n - n, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) rd[i][e] = pack_bf16(v[2 * e], v[2 * e + 1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const int q = tid + NT * i, t = kt * kTileT + q / UK, k = k0 + q % UK * 8;
      rx[i] = u32x2_t{0u, 0u};
      sx[i] = 127;
      if (t < g.tokens && k < g.ld) {
        rx[i] = *reinterpret_cast<const u32x2_t*>(g.x + (long long)t * g.ld + k);
        sx[i] = g.sx[(long long)(t >> g.shift) * g.sld + (k >> 7)];
      }
    }
  };
  auto lstore = [&](u32x4_t* St) {
#pragma unroll
    for (int i = 0; i < PN; ++i) {
      const int q = tid + NT * i, t = q / UN;
      St[t * UN + qrow_unit<BN / 32>(t, q % UN)] = rd[i];
    }
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const int q = tid + NT * i, t = q / UK;
      St[kTileT * UN + t * UK + qrow_unit<BK / 32>(t, q % UK)] =
          bf16_of_e4m3(rx[i][0], rx[i][1], scale_of(sx[i]));
    }
  };

  f32x16_t acc[FN][FK];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FK; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // transposing reads, as for the row-major operand of the step's update
  const int hsel = lane >> 5;
  const int tr_k = 8 * hsel + ((lane & 15) >> 2);
  const int tr_j = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  auto frag = [&](const u32x4_t* P, auto units, int kk, int j) __attribute__((always_inline)) {
    constexpr int U = decltype(units)::value;
    u32x2_t h[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = 16 * kk + tr_k + 4 * s;
      h[s] = lds_read_tr16(reinterpret_cast<const unsigned char*>(P) +
                           (k * U + qrow_unit<U / 4>(k, j >> 3)) * 16 + (j & 7) * 2);
    }
    return u32x4_t{h[0][0], h[0][1], h[1][0], h[1][1]};
  };
  auto compute = [&](const u32x4_t* St) {
#pragma unroll
    for (int kk = 0; kk < kTileT / 16; ++kk) {
      u32x4_t fn[FN], fk[FK];
#pragma unroll
      for (int i = 0; i < FN; ++i)
        fn[i] = frag(St, std::integral_constant<int, UN>{}, kk, wn * WTN + 32 * i + tr_j);
#pragma unroll
      for (int j = 0; j < FK; ++j)
        fk[j] = frag(St + kTileT * UN, std::integral_constant<int, UK>{}, kk,
                     wk * WTK + 32 * j + tr_j);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FK; ++j) mma<bf16_t>(acc[i][j], fn[i], fk[j]);
    }
  };
  if (t_first < t_end) {
    gload(t_first);
    lstore(lds[0]);
    __syncthreads();
    for (int kt = t_first; kt < t_end; ++kt) {
      const int cur = (kt - t_first) & 1;
      if (kt + 1 < t_end) gload(kt + 1);
      compute(lds[cur]);
      if (kt + 1 < t_end) lstore(lds[cur ^ 1]);
      __syncthreads();
    }
  }

  // lane: column k, 4 consecutive rows n per quad; 32 lanes write one row run
  W* dw = static_cast<W*>(g.dw);
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FK; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int n = n0 + wn * WTN + 32 * i + 8 * (r / 4) + 4 * hsel + r % 4;
        const int k = k0 + wk * WTK + 32 * j + (lane & 31);
        if (n < g.n && k < g.k) {
          const long long o = (long long)n * g.k + k;
          if (g.part)
            g.part[(long long)split * g.n * g.k + o] = acc[i][j][r];
          else if (g.accumulate)
            dw[o] = from_f32<W>(to_f32(dw[o]) + acc[i][j][r]);
          else
            dw[o] = from_f32<W>(acc[i][j][r]);
        }
      }
}

// dw (+)= the parts, in their order; 4 elements per thread.
template <typename W>
__global__ __launch_bounds__(256) void weight_grad_join_kernel(const float* part, int splits,
                                                               long long elems, void* dw,
                                                               int accumulate) {
  const long long o = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (o >= elems) return;
  W* w = static_cast<W*>(dw) + o;
  const int n = elems - o < 4 ? (int)(elems - o) : 4;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (n == 4) {
#pragma unroll 4
    for (int p = 0; p < splits; ++p) {
      f32x4_t v;
      __builtin_memcpy(&v, part + p * elems + o, 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
  } else {
    for (int p = 0; p < splits; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) s[e] += part[p * elems + o + e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) w[e] = from_f32<W>(accumulate ? to_f32(w[e]) + s[e] : s[e]);
}

// Token splits: enough workgroups for two per CU, and at least four token
// tiles in each.
int weight_grad_splits(int tokens, int n, int k, int* tiles_per_split) {
  const long long tiles = (long long)((n + 127) / 128) * ((k + 127) / 128);
  const int tt = (tokens + kTileT - 1) / kTileT;
  long long want = 512 / tiles;
  if (want > tt / 4) want = tt / 4;
  if (want < 1) want = 1;
  const int per = tt > 0 ? (int)((tt + want - 1) / want) : 1;
  *tiles_per_split = per;
  return tt > 0 ? (tt + per - 1) / per : 1;
}

namespace {
template <typename W>
void go(const WeightGradArgs& in, hipStream_t s) {
  WeightGradArgs a = in;
  a.tiles_n = (a.n + 127) / 128;
  a.tiles_k = (a.k + 127) / 128;
  hipLaunchKernelGGL((weight_grad_kernel<128, 128, 2, 2, W>),
                     dim3((unsigned)(a.tiles_n * a.tiles_k * a.splits)), dim3(256), 0, s, a);
  if (a.part) {
    const long long elems = (long long)a.n * a.k;
    hipLaunchKernelGGL(weight_grad_join_kernel<W>, dim3((unsigned)((elems + 1023) / 1024)),
                       dim3(256), 0, s, a.part, a.splits, elems, a.dw, a.accumulate);
  }
}
}  // namespace

hipError_t launch_weight_grad(int dw_bf16, const WeightGradArgs& a, hipStream_t s) {
  if (dw_bf16)
    go<bf16_t>(a, s);
  else
    go<float>(a, s);
  return hipGetLastError();
}

}  // namespace muon
