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

constexpr int kGroupN = 4;

// Wait until this wave has no LDS operation in flight (lgkmcnt(0), the other
// counters untouched: loads into registers stay in flight).
__device__ __forceinline__ void wait_lgkm0() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_s_waitcnt(0xc07f);
#endif
}

// A workgroup computes a BN x BK tile of dw in WGN x WGK waves of 32x32 MFMA
// tiles.  A token tile of both operands lies in LDS as bf16 rows [t][column]
// (64-byte segments permuted by t % 4 as for the step's row-major operand, so
// that the 4 rows of a transposing read fall on 4 quarters of the bank line),
// two stages.  Loads go through registers, because x changes its type on the
// way and because rows of any stride and a ragged last tile then go the same
// way.  While token tile kt is multiplied, kt + 1 goes from registers to the
// other stage in the first of the four substeps of 16 tokens, and the loads of
// kt + 2 follow at once: they have three quarters of a tile and its barrier to
// arrive.  The waves meet before the last substep, whose operands are in
// registers by then, and read the next tile's first ones during it.  After each
// MFMA comes its share of the substep's LDS reads and writes.
// Token tiles below the ragged edges are loaded without a branch, in line with
// the MFMAs.
//   8192 tokens, 4096 x 4096, 256 x 256 tiles: 220 to 236 us by box, 1.16 to
//   1.25 PFLOP/s (393 us with 128 x 128 tiles on 4 waves, everything loaded and
//   stored at the tile's ends, and no order pinned; 234 us with a branch around
//   each load; a library's plain bf16 product of 8192^3 runs at 1.36 to 1.41).
//   The MFMAs are busy 59% of the cycles, at 1.96 GHz, the LDS a third; neither
//   reading operands two substeps ahead nor loading two token tiles ahead
//   changed that.

template <int BN, int BK, int WGN, int WGK, typename W>
__global__ __launch_bounds__(64 * WGN * WGK) void weight_grad_kernel(WeightGradArgs g) {
  constexpr int NT = 64 * WGN * WGK;
  constexpr int WTN = BN / WGN, WTK = BK / WGK;
  constexpr int FN = WTN / 32, FK = WTK / 32;
  constexpr int UN = BN / 8, UK = BK / 8;          // chunks of 8 per token row
  constexpr int PN = kTileT * UN / NT, PK = kTileT * UK / NT;
  static_assert(PN * NT == kTileT * UN && PK * NT == kTileT * UK, "chunks split over the threads");
  static_assert(NT % UN == 0 && NT % UK == 0, "a thread keeps its columns");
  constexpr int SN = kTileT * UN, SK = kTileT * UK;
  __shared__ u32x4_t Ln[2 * SN], Lk[2 * SK];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave / WGK, wk = wave % WGK;
  const int L = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int tiles = g.tiles_n * g.tiles_k;
  const int split = L / tiles, tile = L - split * tiles;
  // Tiles go in groups of kGroupN tile rows, column by column: an XCD's 32 CUs
  // then share 4 panels of dy and 8 of x, not 2 and 16 (16384 tokens, 4096 x
  // 16384: 1805 -> 1782 us; 8192 tokens, 4096 x 4096: 231 -> 230).
  const int group = tile / (kGroupN * g.tiles_k), first = group * kGroupN;
  const int rows = g.tiles_n - first < kGroupN ? g.tiles_n - first : kGroupN;
  const int place = tile - first * g.tiles_k;
  const int n0 = (first + place % rows) * BN, k0 = place / rows * BK;
  const int t_first = split * g.tiles_per_split;
  const int t_all = (g.tokens + kTileT - 1) / kTileT;
  const int t_end = t_first + g.tiles_per_split < t_all ? t_first + g.tiles_per_split : t_all;

  // the thread's chunks: columns cn (of dy) and ck (of x), rows tn + i NT / UN
  // and tk + i NT / UK
  const int tn = tid / UN, cn = tid % UN, tk = tid / UK, ck = tid % UK;
  const int n = n0 + 8 * cn, k = k0 + 8 * ck;
  const bool k_in = k < g.ld, n_all = n0 + BN <= g.n;
  const unsigned dy_off = (unsigned)tn * (unsigned)g.lddy + (n < g.n ? 8 * cn : 0);
  const unsigned x_off = (unsigned)tk * (unsigned)g.ld + (k_in ? 8 * ck : 0);
  const unsigned s_off = (g.shift ? 0u : (unsigned)tk * (unsigned)g.sld) + (k_in ? ck >> 4 : 0);
  u32x4_t rd[PN];
  u32x2_t rx[PK];
  int sx[PK];
  // A chunk past dy's or x's last column reads the tile's first one, and one
  // across dy's last column reads up to 7 elements behind it, of the rows that
  // follow: what comes of them is not stored.  The last row has none that follow
  // (nor, where rows are shorter than 7, have the last 7), and rows past it
  // must be zero: from token tile `safe` on, loads look at each chunk.
  const int short_rows = n_all ? 0 : g.lddy < 7 ? 7 : 1;
  const int safe = g.tokens > short_rows ? (g.tokens - short_rows) / kTileT : 0;
  auto gload = [&](int kt, auto plain) __attribute__((always_inline)) {
    const int t0 = kt * kTileT;
    const bf16_t* dyb = static_cast<const bf16_t*>(g.dy) + (long long)t0 * g.lddy + n0;
    const unsigned char* xb = g.x + (long long)t0 * g.ld + k0;
    const unsigned char* sb = g.sx + (long long)(t0 >> g.shift) * g.sld + (k0 >> 7);
#pragma unroll
    for (int i = 0; i < PN; ++i) {
      const bf16_t* p = dyb + (long long)(NT / UN * i) * g.lddy + dy_off;
      if constexpr (decltype(plain)::value) {
        __builtin_memcpy(&rd[i], p, 16);
      } else {
        float v[8];
        load8_edge(p, t0 + tn + NT / UN * i < g.tokens ? g.n - n : 0, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) rd[i][e] = pack_bf16(v[2 * e], v[2 * e + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const unsigned char* p = xb + (long long)(NT / UK * i) * g.ld + x_off;
      const unsigned char* s = sb + (g.shift ? 0 : (long long)(NT / UK * i) * g.sld) + s_off;
      if (decltype(plain)::value || t0 + tk + NT / UK * i < g.tokens) {
        rx[i] = *reinterpret_cast<const u32x2_t*>(p);
        sx[i] = *s;
      } else {
        rx[i] = u32x2_t{0u, 0u};
        sx[i] = 127;
      }
    }
  };
  auto gload_any = [&](int kt) __attribute__((always_inline)) {
    if (kt < safe)
      gload(kt, std::true_type{});
    else
      gload(kt, std::false_type{});
  };
  auto lstore = [&](int st) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PN; ++i) {
      const int t = tn + NT / UN * i;
      Ln[st * SN + t * UN + qrow_unit<4>(t, cn)] = rd[i];
    }
#pragma unroll
    for (int i = 0; i < PK; ++i) {
      const int t = tk + NT / UK * i;
      Lk[st * SK + t * UK + qrow_unit<4>(t, ck)] =
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
  u32x4_t fn[2][FN], fk[2][FK];
  auto frag = [&](const u32x4_t* P, auto units, int kk, int j) __attribute__((always_inline)) {
    constexpr int U = decltype(units)::value;
    u32x2_t h[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int kr = 16 * kk + tr_k + 4 * s;
      h[s] = lds_read_tr16(reinterpret_cast<const unsigned char*>(P) +
                           (kr * U + qrow_unit<4>(kr, j >> 3)) * 16 + (j & 7) * 2);
    }
    return u32x4_t{h[0][0], h[0][1], h[1][0], h[1][1]};
  };
  auto fload = [&](int st, int kk, int slot) __attribute__((always_inline)) {
    auto rn = [&](int i) __attribute__((always_inline)) {
      fn[slot][i] = frag(Ln + st * SN, std::integral_constant<int, UN>{}, kk, wn * WTN + 32 * i + tr_j);
    };
    rn(0);
#pragma unroll
    for (int j = 0; j < FK; ++j)
      fk[slot][j] = frag(Lk + st * SK, std::integral_constant<int, UK>{}, kk,
                         wk * WTK + 32 * j + tr_j);
#pragma unroll
    for (int i = 1; i < FN; ++i) rn(i);
  };
  auto mfmas = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FK; ++j) mma<bf16_t>(acc[i][j], fn[slot][i], fk[slot][j]);
  };
  // one substep's order: after each MFMA its share of the LDS reads, of WR LDS
  // writes and of LD loads
  auto pins = [&](auto wr, auto ld) __attribute__((always_inline)) {
    constexpr int WR = decltype(wr)::value, LD = decltype(ld)::value;
    constexpr int NR = 2 * (FN + FK), NM = FN * FK;
    static_for<NM>([&](auto x) {
      constexpr int i = decltype(x)::value;
      constexpr int rd_ = NR * (i + 1) / NM - NR * i / NM, w_ = WR * (i + 1) / NM - WR * i / NM,
                    l_ = LD * (i + 1) / NM - LD * i / NM;
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if constexpr (rd_ > 0) __builtin_amdgcn_sched_group_barrier(0x100, rd_, 0);
      if constexpr (w_ > 0) __builtin_amdgcn_sched_group_barrier(0x200, w_, 0);
      if constexpr (l_ > 0) __builtin_amdgcn_sched_group_barrier(0x020, l_, 0);
    });
  };
  using Z = std::integral_constant<int, 0>;
  // token tile kt from stage cur; the registers hold tile kt + 1, which goes to
  // stage nxt, and then take tile kt + 2 (`plain`: it is there and below safe)
  auto ttile = [&](int kt, int cur, int nxt, auto plain) __attribute__((always_inline)) {
    lstore(nxt);
    fload(cur, 1, 1);
    mfmas(0);
    pins(std::integral_constant<int, PN + PK>{}, Z{});
    if constexpr (decltype(plain)::value) {
      gload(kt + 2, plain);
      fload(cur, 2, 0);
      mfmas(1);
      pins(Z{}, std::integral_constant<int, PN + 2 * PK>{});
    } else {
      if (kt + 2 < t_end) gload_any(kt + 2);
      fload(cur, 2, 0);
      mfmas(1);
      pins(Z{}, Z{});
    }
    fload(cur, 3, 1);
    mfmas(0);
    pins(Z{}, Z{});
    __builtin_amdgcn_s_setprio(0);
    wait_lgkm0();
    barrier_no_fence();
    __builtin_amdgcn_s_setprio(1);
    fload(nxt, 0, 0);
    mfmas(1);
    pins(Z{}, Z{});
  };
  if (t_first < t_end) {
    gload_any(t_first);
    lstore(0);
    if (t_first + 1 < t_end) gload_any(t_first + 1);
    wait_lgkm0();
    barrier_no_fence();
    fload(0, 0, 0);
    int kt = t_first;
    for (; kt + 3 < t_end && kt + 3 < safe; kt += 2) {
      ttile(kt, 0, 1, std::true_type{});
      ttile(kt + 1, 1, 0, std::true_type{});
    }
    for (; kt < t_end; kt += 2) {
      ttile(kt, 0, 1, std::false_type{});
      if (kt + 1 < t_end) ttile(kt + 1, 1, 0, std::false_type{});
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

// The tile and the number of token splits.  A CU holds one workgroup of 256 x
// 256 or 256 x 128 tiles, or two of 128 x 128 ones, all of 8 waves.  Per token
// tile: 1.7 us (256 x 256), 1.05 us (256 x 128), and for 128 x 128 0.7 us alone
// on its CU, 1.3 us for two.  The result and its parts move at 6 TB/s, written
// and read, and a second launch costs 5 us.  The plan takes the smallest sum.
// The constants are fitted to every tile and up to 32 parts at 33 sizes of 2048 to
// 16384 tokens and 500 x 500 to 4096 x 4096: the plan's choice is within 5.3% of
// the fastest at each and 0.4% on average.  (16384 tokens, 2048 x 2048: 143 us in
// 4 parts of 256 x 256, 155 in 2 of 256 x 128, 158 with 128 x 128; 16384 tokens, 768
// x 1003: 40.8 us in 10 parts of 256 x 128, 42.9 in 5 of 128 x 128; 2048 tokens,
// 2048 x 2048: 26.9 us with 128 x 128, 34.1 with 256 x 128.)
WeightGradPlan weight_grad_plan(int tokens, int n, int k) {
  struct Kind {
    int bn, bk, per_cu;
    double one, full;  // us per token tile: alone on its CU, all places taken
  };
  static const Kind kinds[3] = {
      {256, 256, 1, 1.7, 1.7}, {256, 128, 1, 1.05, 1.05}, {128, 128, 2, 0.7, 1.3}};
  const int tt = (int)(((long long)tokens + kTileT - 1) / kTileT);
  WeightGradPlan best{};
  double least = 0.0;
  for (int i = 0; i < 3; ++i) {
    const Kind& c = kinds[i];
    const long long tiles = (long long)((n + c.bn - 1) / c.bn) * ((k + c.bk - 1) / c.bk);
    for (int want = 1; want <= 64; ++want) {
      // at least four token tiles in a part, and no more parts than fill the chip
      if (want > 1 && (want > tt / 4 || tiles * (want - 1) >= 256 * c.per_cu)) break;
      const int per = tt > 0 ? (tt + want - 1) / want : 1;
      const int splits = tt > 0 ? (tt + per - 1) / per : 1;
      const long long wgs = tiles * splits;
      const double us_tile = wgs <= 256 ? c.one : c.full;
      const double rounds = (double)((wgs + 256 * c.per_cu - 1) / (256 * c.per_cu));
      double us = rounds * per * us_tile;
      if (splits > 1) us += 5.0 + 2.0 * splits * 4.0 * n * k / 6e6;
      if (best.splits == 0 || us < least) {
        least = us;
        best = WeightGradPlan{i, splits, per, c.bn, c.bk};
      }
    }
  }
  return best;
}

namespace {
template <typename W>
void go(const WeightGradArgs& in, const WeightGradPlan& p, hipStream_t s) {
  WeightGradArgs a = in;
  a.splits = p.splits;
  a.tiles_per_split = p.tiles_per_split;
  a.tiles_n = (a.n + p.bn - 1) / p.bn;
  a.tiles_k = (a.k + p.bk - 1) / p.bk;
  const dim3 grid((unsigned)a.tiles_n * (unsigned)a.tiles_k * (unsigned)a.splits), block(512);
  if (p.kind == 0)
    hipLaunchKernelGGL((weight_grad_kernel<256, 256, 2, 4, W>), grid, block, 0, s, a);
  else if (p.kind == 1)
    hipLaunchKernelGGL((weight_grad_kernel<256, 128, 4, 2, W>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((weight_grad_kernel<128, 128, 2, 4, W>), grid, block, 0, s, a);
  if (a.part) {
    const long long elems = (long long)a.n * a.k;
    hipLaunchKernelGGL(weight_grad_join_kernel<W>, dim3((unsigned)((elems + 1023) / 1024)),
                       dim3(256), 0, s, a.part, a.splits, elems, a.dw, a.accumulate);
  }
}
}  // namespace

hipError_t launch_weight_grad(int dw_bf16, const WeightGradArgs& a, const WeightGradPlan& p,
                              hipStream_t s) {
  if (dw_bf16)
    go<bf16_t>(a, p, s);
  else
    go<float>(a, p, s);
  return hipGetLastError();
}

}  // namespace muon
