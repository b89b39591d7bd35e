// y = a b^T of two 8-bit tensors (e4m3, a power-of-two scale per block of 128
// along the sum):
//   y[m][n] = sum_k a[m][k] b[n][k],  a = qa 2^ea(m, k / 128), b likewise.
// A bf16 result of many rows comes from v_mfma_scale_f32_32x32x64_f8f6f4, which
// multiplies by both scales inside the instruction, so that the block scales
// cost no vector work: a lane hands over the scale byte of its own row next to
// its operand.  The instruction adds products in groups of 8 consecutive k in
// fixed point, 13 bits below the group's largest exponent, the rest cut off
// (measured: one product of 2^16 and one of m 2^(16 - j) in a group come out with
// m cut to 13 - j fraction bits, and 0 from j = 14 on; the groups' sums and the
// accumulator keep all 24 bits).  A result is thus off by less than
// 7 * 2^-13 * sum of the groups' largest products; on Gaussian operands of any
// length by 1.5e-5 of the result's norm, 1/110 of what rounding it to bf16 does
// (1.7e-3).  A result in fp32 keeps more than that, so it comes from bf16 MFMAs
// at half the rate, to whose operands the values are converted exactly
// (EXACT; 1e-7 of the norm); and so does one that an epilogue rounds to 8 bits
// (linear8.hip).
//
// Two kernels:
//   tiles   both operands through LDS, for many rows of a: bound by the MFMAs;
//   rows    few rows of a (up to 32): bound by reading b once, so always exact.
// Both with an epilogue too (EPI, for linear8): z = y + bias, kept where it is
// asked for, and act(z) + residual in bf16, fp32 or 8 bits.  What that costs a product
// of 16384 x 16384 x 4096 (815 us on the same card): bias 15 us, squared ReLU 20, GELU
// 110, a bf16 residual 90 (512 MB), an 8-bit result 58, and all of GELU, z kept and 8
// bits 180; one of 4096 x 5120 x 1280 (38 us): 1, 2, 5, 6, 2 and 11 (products of the
// 8-bit instruction in all).
#pragma once

#include "muon_gemm.h"

#include "activation.h"
#include "muon_block.h"

namespace muon {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t frag8(const u32x4_t& lo, const u32x4_t& hi) {
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// The type of z, and the arguments with and without an epilogue.
template <typename Y> using KeptOf = std::conditional_t<std::is_same_v<Y, float>, float, bf16_t>;
template <bool EPI> using ProductArgs = std::conditional_t<EPI, Linear8Args, Matmul8Args>;
template <typename Y> constexpr bool is8 = std::is_same_v<Y, unsigned char>;

// What lies behind the last block in a row of scales: blocks of zeros, so that equal
// tensors are equal byte by byte.
__device__ __forceinline__ void pad_scales(const Linear8Args& g, int m) {
  for (long long j = g.ld_y8 >> 7; j < g.sld_y8; ++j)
    g.s8[(long long)m * g.sld_y8 + j] = (unsigned char)scale_byte(0u);
}
// The residual of an epilogue: none, of one of the types, or (RES_ANY) of the type
// that the arguments say, for tiles at an edge.
enum Res { RES_NONE, RES_BF16, RES_FP32, RES_ANY };
// Eight elements of a residual row, as they lie in memory where the type is known.
template <int R>
struct RawRes {
  typename std::conditional_t<R == RES_BF16, Raw8<bf16_t>, Raw8<float>> raw;
  __device__ __forceinline__ void load(const void* p, bool fp32, int left) {
    if constexpr (R == RES_BF16) {
      raw.load(static_cast<const bf16_t*>(p), left);
    } else if constexpr (R == RES_FP32) {
      raw.load(static_cast<const float*>(p), left);
    } else if (fp32) {
      load8_edge(static_cast<const float*>(p), left, raw.w);
    } else {
      load8_edge(static_cast<const bf16_t*>(p), left, raw.w);
    }
  }
  __device__ __forceinline__ void add(float (&v)[8]) const {
    float r[8];
    raw.get(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
};
template <bool FULL, bool STRM, typename T>
__device__ __forceinline__ void store_run(T* p, int left, const float (&v)[8]) {
  if constexpr (FULL)
    store8<STRM>(p, v);
  else
    store8_edge<STRM>(p, left, v);
}
// A lane's place in the matrices of the epilogue: its pointers at the lane's first row
// and column of the tile, from which every run is a number of rows and columns away
// that all lanes share, so that a run's address costs the vector unit one addition.
struct Places {
  const char* res;
  char *y, *z, *s;          // y: of the 8-bit result too; s: its scale bytes
  int m, n;                 // of the first run
};
__device__ __forceinline__ long long bytes_away(int rows, int cols, long long ld, int es) {
  return ((long long)rows * ld + cols) * es;
}
// COUNT runs of eight columns of the epilogue, `rows` and `cols` away from the lane's
// first, from the sums v to the results; nothing is rounded on the way but for the z
// that is kept.  Each step is done for all runs, so that its branches (the same for
// all lanes) stand around independent work.  FULL: no row or column lies past the
// last one.
template <bool FULL, bool STRM, typename Y, int R, int COUNT>
__device__ __forceinline__ void epilogue_runs(const Linear8Args& g, const Places& at,
                                              const int (&rows)[COUNT], int cols,
                                              const float (&bias)[8],
                                              const RawRes<R> (&res)[COUNT],
                                              float (&v)[COUNT][8]) {
  using Z = KeptOf<Y>;
  const int left = g.n - at.n - cols;
  // for an 8-bit result a run past the last column pads the last block
  auto in = [&](int s) {
    return FULL || ((is8<Y> ? at.n + cols < g.ld_y8 : left > 0) && at.m + rows[s] < g.m);
  };
#pragma unroll
  for (int s = 0; s < COUNT; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[s][e] += bias[e];
  if (g.z) {
#pragma unroll
    for (int s = 0; s < COUNT; ++s)
      if (in(s))
        store_run<FULL, STRM>(
            reinterpret_cast<Z*>(at.z + bytes_away(rows[s], cols, g.ldz, sizeof(Z))), left, v[s]);
  }
  activate<std::is_same_v<Y, float>>(v, g.act);
  if (R != RES_NONE && g.res) {
#pragma unroll
    for (int s = 0; s < COUNT; ++s) res[s].add(v[s]);
  }
  if constexpr (is8<Y>) {
#pragma unroll
    for (int s = 0; s < COUNT; ++s) {
      if (!FULL) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[s][e] = e < left ? v[s][e] : 0.f;
      }
      const int byte = block_units(v[s], v[s]);
      if (in(s)) {
        *reinterpret_cast<u32x2_t*>(at.y + bytes_away(rows[s], cols, g.ld_y8, 1)) = to_e4m3(v[s]);
        if (((at.n + cols) & 127) == 0)
          *reinterpret_cast<unsigned char*>(at.s + bytes_away(rows[s], cols >> 7, g.sld_y8, 1)) =
              (unsigned char)byte;
      }
    }
  } else {
#pragma unroll
    for (int s = 0; s < COUNT; ++s)
      if (in(s))
        store_run<FULL, STRM>(
            reinterpret_cast<Y*>(at.y + bytes_away(rows[s], cols, g.ldy, sizeof(Y))), left, v[s]);
  }
}
// The same for four columns; any of them may lie past the last one.
template <typename Y>
__device__ __forceinline__ void epilogue4(const Linear8Args& g, int m, int n, f32x4_t& s) {
  float v[1][4] = {{s[0], s[1], s[2], s[3]}};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (g.bias && n + e < g.n) v[0][e] += g.bias[n + e];
    if (g.z && n + e < g.n)
      static_cast<KeptOf<Y>*>(g.z)[(long long)m * g.ldz + n + e] = from_f32<KeptOf<Y>>(v[0][e]);
  }
  activate<std::is_same_v<Y, float>>(v, g.act);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (g.res && n + e < g.n) {
      const long long at = (long long)m * g.ldr + n + e;
      v[0][e] += g.res_fp32 ? static_cast<const float*>(g.res)[at]
                            : to_f32(static_cast<const bf16_t*>(g.res)[at]);
    }
    s[e] = v[0][e];
  }
}
// ---------------------------------------------------------------- tiles
// A workgroup computes BN columns n (the MFMA's rows, operand b) by BM rows m
// (its columns, operand a) of y.  k advances by one block of 128 per k-tile:
// 128-byte operand rows of 8 chunks in LDS (swz), BN rows of b, then BM of a,
// loaded straight into LDS, two stages.  A substep is 64 k, one 32x32x64
// MFMA or (EXACT) four 32x32x16: lane (r, h) = (lane % 32, lane / 32) reads
// chunks 4 kk + 2 h and the one after it of its row, for both operands the
// same, so the order of k does not matter.  Rows past the last one read the
// last one again and are not stored.
//
// The scales go through LDS as well, a word of four k-tiles per row, so that
// no load into registers is in flight in the main loop: the compiler's wait
// for such a load would wait for the LDS loads too (8192 x 4096 x 4096: 114 ->
// 108 us).  Four k-tiles are written out, because the byte of the word that an
// MFMA takes is part of the instruction.
//
// The order of MFMAs, LDS reads and loads is pinned: each MFMA of a substep is
// followed by two reads of the next one's operands, and after the barrier by
// one load.  Between the barrier and the next wait the wave has priority over
// its neighbour, so that the two waves of a SIMD fall out of step and one's
// MFMAs cover the other's waits (16384 x 16384 x 4096: 874 -> 822 us).
//   256 x 256 tiles on 8 waves, inputs in the caches: 8192 x 4096 x 4096 103 to
//   110 us by box (2.5 to 2.67 PFLOP/s), 16384 x 16384 x 4096 788 to 798 us (2.75
//   to 2.80), to fp32 216 and 1766 us (1.25).  They take all 256 registers and
//   spill 5 (24 bytes a lane; exact ones 2, with an epilogue 6 to 8).
//   A library's product with one scale per tensor runs at 2.72 to 2.80.  At the
//   larger size the MFMAs are busy 70% of the cycles and the chip runs at 1.68
//   GHz: it is bound by power.  Without the stores of y it would take 752 us.
//   4 waves of 128 x 128, 512 registers each: 110 us; 4 stages of 64 k: 116 us.
template <int BM, int BN, int WGM, int WGN, bool EXACT, bool STRM, typename Y, bool EPI = false>
__global__ __launch_bounds__(64 * WGM * WGN, WGM * WGN == 8 && BM == 128 ? 4 : 1) void
matmul8_tile_kernel(ProductArgs<EPI> g) {
  constexpr int NW = WGM * WGN;
  constexpr int WTM = BM / WGM, WTN = BN / WGN;
  constexpr int FM = WTM / 32, FN = WTN / 32;
  constexpr int CPR = 8;
  constexpr int B_CHUNKS = BN * CPR, STAGE = (BM + BN) * CPR;
  constexpr int DPW = STAGE / 64 / NW;      // loads of a wave per k-tile
  // and of 64 scale words per four; where there are more waves than those, the
  // others load the same again
  constexpr int SG = (BM + BN) / 64, SPW = SG > NW ? SG / NW : 1;
  // a wave's loads are of one operand, or (MIXED) each is of one, told by its place
  constexpr bool MIXED = B_CHUNKS % (DPW * 64) != 0;
  static_assert(DPW * 64 * NW == STAGE && B_CHUNKS % 64 == 0, "whole loads");
  static_assert((SG % NW == 0 || SG < NW) && BN % (SPW * 64) == 0, "one operand's scales per wave");
  static_assert(FN % 2 == 0, "halves of a wave's columns are staged");
  __shared__ u32x4_t S0[STAGE], S1[STAGE];
  __shared__ __attribute__((aligned(16))) unsigned C0[BM + BN];
  __shared__ unsigned C1[BM + BN];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WGN, wn = wave % WGN;
  const int L = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int span = g.group_m * g.tiles_n;
  const int grp = L / span, first = grp * g.group_m;
  const int gm = g.tiles_m - first < g.group_m ? g.tiles_m - first : g.group_m;
  const int idx = L - grp * span;
  const int m0 = (first + idx % gm) * BM, n0 = (idx / gm) * BN;

  const int wave_s = __builtin_amdgcn_readfirstlane(wave);
  auto of_b = [&](int d) { return (wave_s * DPW + (MIXED ? d : 0)) * 64 < B_CHUNKS; };
  auto base_of = [&](int d) __attribute__((always_inline)) {
    return of_b(d) ? g.b + (long long)n0 * g.ld : g.a + (long long)m0 * g.ld;
  };
  const unsigned char* base = base_of(0);
  unsigned voff[DPW];
#pragma unroll
  for (int d = 0; d < DPW; ++d) {
    const bool is_b = of_b(d);
    const int last_row = is_b ? g.n - 1 - n0 : g.m - 1 - m0;
    const int q = (wave * DPW + d) * 64 + lane;
    const int r = q / CPR, rl = is_b ? r : r - BN;
    voff[d] = (unsigned)(rl < last_row ? rl : last_row) * (unsigned)g.ld + swz(q % CPR, r) * 16;
  }
  const int nk = g.ld / 128, last_word = (nk - 1) / 4;
  auto issue = [&](int kt, u32x4_t* St) __attribute__((always_inline)) {
    if constexpr (MIXED) {
#pragma unroll
      for (int d = 0; d < DPW; ++d)
        buffer_load_lds16(buffer_rsrc(base_of(d) + (long long)kt * 128), voff[d],
                          St + (wave_s * DPW + d) * 64);
    } else {
      const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(base + (long long)kt * 128);
#pragma unroll
      for (int d = 0; d < DPW; ++d) buffer_load_lds16(rs, voff[d], St + (wave_s * DPW + d) * 64);
    }
  };
  // word w of the scales of the tile's rows: b's, then a's
  const int sg = SG < NW ? wave_s % SG : wave_s * SPW;
  const bool sc_b = sg * 64 < BN;
  const int s_first = sc_b ? n0 : m0, s_last = sc_b ? g.n - 1 : g.m - 1;
  const int s_shift = sc_b ? g.shift_b : g.shift_a;
  const unsigned char* sbase = (sc_b ? g.sb : g.sa) + (long long)(s_first >> s_shift) * g.sld;
  unsigned soff[SPW];
#pragma unroll
  for (int d = 0; d < SPW; ++d) {
    const int i = ((SG < NW ? wave % SG : wave * SPW) + d) * 64 + lane;
    const int r = s_first + (sc_b ? i : i - BN);
    soff[d] = (unsigned)(((r < s_last ? r : s_last) >> s_shift) - (s_first >> s_shift)) *
              (unsigned)g.sld;
  }
  auto issue_scales = [&](int w, unsigned* C) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(sbase + 4 * (w < last_word ? w : last_word));
#pragma unroll
    for (int d = 0; d < SPW; ++d) buffer_load_lds4(rs, soff[d], C + (sg + d) * 64);
  };

  f32x16_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int brow = wn * WTN + (lane & 31), arow = BN + wm * WTM + (lane & 31);
  const int hsel = lane >> 5;
  i32x8_t fb[2][FN], fa[2][FM];
  int sc[FN + FM];
  auto fload = [&](const u32x4_t* St, int kk, int slot) __attribute__((always_inline)) {
    const int ch = 4 * kk + 2 * hsel;
    auto row = [&](int r) __attribute__((always_inline)) {
      return frag8(St[r * CPR + swz(ch, r)], St[r * CPR + swz(ch + 1, r)]);
    };
    fb[slot][0] = row(brow);
#pragma unroll
    for (int f = 0; f < FM; ++f) fa[slot][f] = row(arow + f * 32);
#pragma unroll
    for (int f = 1; f < FN; ++f) fb[slot][f] = row(brow + f * 32);
  };
  auto sload = [&](const unsigned* C) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < FN; ++f) sc[f] = (int)C[brow + f * 32];
#pragma unroll
    for (int f = 0; f < FM; ++f) sc[FN + f] = (int)C[arow + f * 32];
  };
  auto mfmas = [&](int slot, auto byte) __attribute__((always_inline)) {
    constexpr int B = decltype(byte)::value;
    if constexpr (EXACT) {
      float sf[FN + FM];
#pragma unroll
      for (int f = 0; f < FN + FM; ++f) sf[f] = scale_of((sc[f] >> (8 * B)) & 0xff);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        u32x4_t wb[FN], wa[FM];
#pragma unroll
        for (int i = 0; i < FN; ++i)
          wb[i] = bf16_of_e4m3((unsigned)fb[slot][i][e], (unsigned)fb[slot][i][e + 1], sf[i]);
#pragma unroll
        for (int j = 0; j < FM; ++j)
          wa[j] = bf16_of_e4m3((unsigned)fa[slot][j][e], (unsigned)fa[slot][j][e + 1], sf[FN + j]);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) mma<bf16_t>(acc[i][j], wb[i], wa[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fb[slot][i], fa[slot][j], acc[i][j], 0, 0, B, sc[i], B, sc[FN + j]);
    }
  };
  // the order of one substep: per MFMA two LDS reads and LD / NM loads
  auto pin = [&](auto loads) __attribute__((always_inline)) {
    constexpr int LD = decltype(loads)::value, NR = 2 * (FN + FM), NM = FN * FM;
    if constexpr (!EXACT)
      static_for<NM>([&](auto x) {
        constexpr int i = decltype(x)::value;
        constexpr int r0 = 2 * i < NR ? 2 * i : NR, r = i == NM - 1 ? NR : 2 * i + 2;
        constexpr int reads = (r < NR ? r : NR) - r0, lds = LD * (i + 1) / NM - LD * i / NM;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
        if constexpr (lds > 0) __builtin_amdgcn_sched_group_barrier(0x020, lds, 0);
      });
  };
  // k-tile kt, its scales in byte kt % 4.  The waves meet once the second
  // substep's operands are in registers; the k-tile after next then goes into
  // the stage just finished.
  auto ktile = [&](int kt, u32x4_t* cur, const u32x4_t* nxt, auto byte)
                   __attribute__((always_inline)) {
    fload(cur, 1, 1);
    mfmas(0, byte);
    pin(std::integral_constant<int, 0>{});
    __builtin_amdgcn_s_setprio(0);
    wait_vm_lgkm0();
    barrier_no_fence();
    __builtin_amdgcn_s_setprio(1);
    issue(kt + 2 < nk ? kt + 2 : nk - 1, cur);
    fload(nxt, 0, 0);
    mfmas(1, byte);
    pin(std::integral_constant<int, DPW>{});
  };
  // k-tiles 4 w .. 4 w + count - 1; the next four's scales go to Cn.  They
  // are read after the waits of at least one k-tile's barrier.
  auto four = [&](int w, int count, const unsigned* C, unsigned* Cn)
                  __attribute__((always_inline)) {
    sload(C);
    issue_scales(w + 1, Cn);
    ktile(4 * w, S0, S1, std::integral_constant<int, 0>{});
    if (count > 1) ktile(4 * w + 1, S1, S0, std::integral_constant<int, 1>{});
    if (count > 2) ktile(4 * w + 2, S0, S1, std::integral_constant<int, 2>{});
    if (count > 3) ktile(4 * w + 3, S1, S0, std::integral_constant<int, 3>{});
  };
  issue_scales(0, C0);
  issue(0, S0);
  wait_vmcnt<0>();
  barrier_no_fence();
  issue(nk > 1 ? 1 : 0, S1);
  fload(S0, 0, 0);
  int w = 0;
  for (; 4 * w + 8 <= nk; w += 2) {
    four(w, 4, C0, C1);
    four(w + 1, 4, C1, C0);
  }
  const int left = nk - 4 * w;  // 0 .. 7
  if (left > 0) four(w, left, C0, C1);
  if (left > 4) four(w + 1, left - 4, C1, C0);
  wait_vmcnt<0>();
  __syncthreads();

  // Epilogue: acc holds, per lane, one row m and 4 consecutive columns n per
  // register quad.  Each wave stages 32 rows m of half its columns as fp32 in
  // its own part of the LDS (16-byte units, exchanged by row) and stores runs
  // of 8 columns, neighbouring lanes neighbouring runs.  For an 8-bit result 32
  // rows of a whole block of 128 columns are staged, by the one or two waves that
  // have them, so that 16 lanes hold a block and find its scale.
  constexpr int HC = is8<Y> ? 128 : WTN / 2;  // columns of a staged row
  constexpr int UPR = HC / 4, RPR = HC / 8;   // units, runs per staged row
  constexpr int WPG = is8<Y> ? 128 / WTN : 1; // waves that share a part
  constexpr int PARTS = NW / WPG, PER = STAGE * 16 / (32 * HC * 4);  // parts, in a stage
  static_assert(BN % 128 == 0 || !is8<Y>, "whole blocks");
  static_assert(PARTS <= 2 * PER, "staging fits");
  const int part = wave_s / WPG, sub = wave_s % WPG;
  float* T = reinterpret_cast<float*>(PARTS <= PER || part < PER ? S0 : S1) + part % PER * 32 * HC;
  auto unit = [](int r, int u) __attribute__((always_inline)) {
    return 4 * (r * UPR + (u ^ (r & (UPR - 1))));
  };
  // only this wave touches its part, and a wave's LDS accesses execute in
  // order: a compiler barrier orders them; two waves meet
  auto staged = [] __attribute__((always_inline)) {
    if constexpr (WPG > 1)
      __syncthreads();
    else
      asm volatile("" ::: "memory");
  };
  constexpr int HALVES = is8<Y> ? 1 : 2, FH = FN / HALVES;
  constexpr int RUNS = 32 * RPR / 64 / WPG;  // of a lane, per staged part
  const int n_part = n0 + (is8<Y> ? wn / WPG * 128 : wn * WTN);
  auto stage = [&](int j, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FH; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16_t& c = acc[h * FH + i][j];
        *reinterpret_cast<f32x4_t*>(T + unit(lane & 31, sub * (WTN / 4) + 8 * i + 2 * q + hsel)) =
            f32x4_t{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
    staged();
  };
  // run s of the lane: its row and column of the part, and its sums
  auto row_of = [&](int s) { return (lane + 64 * (s * WPG + sub)) / RPR; };
  const int c_run = 8 * (lane % RPR);
  auto take = [&](int s, float (&v)[8]) __attribute__((always_inline)) {
    const int rr = row_of(s);
    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(T + unit(rr, c_run / 4));
    const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(T + unit(rr, c_run / 4 + 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = lo[e];
      v[4 + e] = hi[e];
    }
  };
  if constexpr (!EPI) {
    Y* y = static_cast<Y*>(g.y);
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        stage(j, h);
#pragma unroll
        for (int s = 0; s < RUNS; ++s) {
          float v[8];
          take(s, v);
          const int m = m0 + wm * WTM + j * 32 + row_of(s), n = n_part + h * HC + c_run;
          if (m < g.m) store8_edge<STRM>(y + (long long)m * g.ldy + n, g.n - n, v);
        }
        staged();
      }
  } else {
    // The bias of the tile's columns, in LDS: a load from memory behind the stores
    // of a run would wait for them.
    float* Cb = reinterpret_cast<float*>(C0);
    for (int i = tid; i < BN; i += 64 * NW)
      Cb[i] = g.bias && n0 + i < g.n ? g.bias[n0 + i] : 0.f;
    __syncthreads();
    Places at;
    at.m = m0 + wm * WTM + row_of(0);
    at.n = n_part + c_run;
    at.res = static_cast<const char*>(g.res) + bytes_away(at.m, at.n, g.ldr, g.res_fp32 ? 4 : 2);
    at.z = static_cast<char*>(g.z) + bytes_away(at.m, at.n, g.ldz, sizeof(KeptOf<Y>));
    at.y = is8<Y> ? reinterpret_cast<char*>(g.y8) + bytes_away(at.m, at.n, g.ld_y8, 1)
                  : static_cast<char*>(g.y) + bytes_away(at.m, at.n, g.ldy, sizeof(Y));
    at.s = reinterpret_cast<char*>(g.s8) + bytes_away(at.m, at.n >> 7, g.sld_y8, 1);
    // One copy of the code for all parts (only the staging names accumulators), but for
    // whole tiles without a residual, whose steps are written out: 2% of a product of
    // 16384 x 16384 x 4096 to 8 bits.  With everything written out the compiler spills
    // hundreds of registers.
    constexpr int COUNT = 2, STEPS = FM * HALVES * RUNS / COUNT;
    static_assert(RUNS % COUNT == 0 && STEPS % 2 == 0, "pairs of steps");
    auto finish = [&](auto full, auto res_kind) __attribute__((always_inline)) {
      constexpr bool FULL = decltype(full)::value;
      constexpr int R = decltype(res_kind)::value;
      constexpr bool AHEAD = R == RES_BF16 || R == RES_FP32;
      // The residual of the lane's runs t, t + 1, .. is on its way a step before it is
      // used, in one of two sets of registers: a copy from one to the other would wait
      // for it, and for the stores of the step before.
      RawRes<R> even[COUNT], odd[COUNT];
      // run s of part p: rows and columns from the lane's first run on
      auto rows_of = [&](int p, int s) { return p / HALVES * 32 + s * WPG * (64 / RPR); };
      auto fetch = [&](int t, RawRes<R>(&res)[COUNT]) __attribute__((always_inline)) {
        const int p = t / RUNS, cols = p % HALVES * HC;
#pragma unroll
        for (int s = 0; s < COUNT; ++s) {
          const int rows = rows_of(p, t % RUNS + s);
          if (FULL || (at.m + rows < g.m && at.n + cols < g.n))
            res[s].load(at.res + bytes_away(rows, cols, g.ldr, g.res_fp32 ? 4 : 2), g.res_fp32,
                        FULL ? 8 : g.n - at.n - cols);
        }
      };
      auto step = [&](int t, RawRes<R>(&res)[COUNT]) __attribute__((always_inline)) {
        const int p = t / RUNS, b = t % RUNS, cols = p % HALVES * HC;
        if (R == RES_ANY && g.res) fetch(t, res);
        float bias[8];
        const f32x4_t* bl = reinterpret_cast<const f32x4_t*>(Cb + (at.n + cols - n0));
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = bl[e / 4][e % 4];
        if (b == 0) {
          if (t > 0) staged();
          static_for<FM * HALVES>([&](auto q) {
            if (p == q) stage(decltype(q)::value / HALVES, decltype(q)::value % HALVES);
          });
        }
        int rows[COUNT];
        float v[COUNT][8];
#pragma unroll
        for (int s = 0; s < COUNT; ++s) {
          rows[s] = rows_of(p, b + s);
          take(b + s, v[s]);
        }
        epilogue_runs<FULL, STRM, Y, R>(g, at, rows, cols, bias, res, v);
      };
      if constexpr (AHEAD) {
        fetch(0, even);
#pragma unroll 1
        for (int t = 0; t < STEPS * COUNT; t += 2 * COUNT) {
          fetch(t + COUNT, odd);
          step(t, even);
          // (after the last pair the first runs again, unused)
          fetch(t + 2 * COUNT < STEPS * COUNT ? t + 2 * COUNT : 0, even);
          step(t + COUNT, odd);
        }
      } else if constexpr (FULL) {
        static_for<STEPS>([&](auto t) { step(decltype(t)::value * COUNT, even); });
      } else {
#pragma unroll 1
        for (int t = 0; t < STEPS * COUNT; t += COUNT) step(t, even);
      }
    };
    using Whole = std::true_type;
    if (m0 + BM > g.m || n0 + BN > g.n)
      finish(std::false_type{}, std::integral_constant<int, RES_ANY>{});
    else if (!g.res)
      finish(Whole{}, std::integral_constant<int, RES_NONE>{});
    else if (g.res_fp32)
      finish(Whole{}, std::integral_constant<int, RES_FP32>{});
    else
      finish(Whole{}, std::integral_constant<int, RES_BF16>{});
    // the rows of scales, by the workgroups that have the last block
    if constexpr (is8<Y>) {
      if (n0 < g.ld_y8 && n0 + BN >= g.ld_y8 && g.sld_y8 > g.ld_y8 >> 7 && tid < BM && m0 + tid < g.m)
        pad_scales(g, m0 + tid);
    }
  }
}

// ---------------------------------------------------------------- rows
// Up to 16 MF rows m.  A workgroup takes 16 NF columns n and its 8 waves share
// the blocks of k between them; operands come straight from memory (each row of
// b is used once) and go to bf16 in registers: four v_mfma_f32_16x16x32_bf16 per
// block and 16 x 16 results.  The waves' sums are added in their order through
// LDS.  NF = 2 reads a half as often, once there are workgroups enough.
constexpr int kFewWaves = 8;

template <int MF, int NF, typename Y, bool EPI = false>
__global__ __launch_bounds__(64 * kFewWaves) void matmul8_rows_kernel(ProductArgs<EPI> g) {
  __shared__ f32x4_t sums[kFewWaves][MF * NF][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = (int)blockIdx.x * 16 * NF;
  const int r = lane & 15, grp = lane >> 4;
  const int nb = g.ld / 128;
  const unsigned char *pb[NF], *psb[NF], *pa[MF], *psa[MF];
  f32x4_t acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    const int n = n0 + 16 * i + r < g.n ? n0 + 16 * i + r : g.n - 1;
    pb[i] = g.b + (long long)n * g.ld + grp * 16;
    psb[i] = g.sb + (long long)(n >> g.shift_b) * g.sld;
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int m = 16 * f + r < g.m ? 16 * f + r : g.m - 1;
    pa[f] = g.a + (long long)m * g.ld + grp * 16;
    psa[f] = g.sa + (long long)(m >> g.shift_a) * g.sld;
#pragma unroll
    for (int i = 0; i < NF; ++i) acc[i][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  // chunks grp and grp + 4 of the block's eight: each load of a wave takes 64
  // consecutive bytes of 16 rows
  struct Frag {
    u32x4_t lo, hi;
    float scale;
  };
  auto load = [](const unsigned char* p, const unsigned char* s, int kb)
                  __attribute__((always_inline)) {
    return Frag{*reinterpret_cast<const u32x4_t*>(p + kb * 128),
                *reinterpret_cast<const u32x4_t*>(p + kb * 128 + 64), scale_of(s[kb])};
  };
  auto bf16 = [](const Frag& f, int e) __attribute__((always_inline)) {
    const u32x4_t& c = e < 2 ? f.lo : f.hi;
    return __builtin_bit_cast(bf16x8_t,
                              bf16_of_e4m3(c[2 * (e & 1)], c[2 * (e & 1) + 1], f.scale));
  };
  for (int kb = wave; kb < nb; kb += kFewWaves) {
    Frag fb[NF], fa[MF];
#pragma unroll
    for (int i = 0; i < NF; ++i) fb[i] = load(pb[i], psb[i], kb);
#pragma unroll
    for (int f = 0; f < MF; ++f) fa[f] = load(pa[f], psa[f], kb);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bf16x8_t wb[NF];
#pragma unroll
      for (int i = 0; i < NF; ++i) wb[i] = bf16(fb[i], e);
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const bf16x8_t wa = bf16(fa[f], e);
#pragma unroll
        for (int i = 0; i < NF; ++i)
          acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[i], wa, acc[i][f], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int f = 0; f < MF; ++f) sums[wave][i * MF + f][lane] = acc[i][f];
  __syncthreads();
  // acc[i][f]: row m = 16 f + lane % 16, columns n0 + 16 i + 4 (lane / 16) + 0 .. 3
  auto take = [&](int t, f32x4_t& s) __attribute__((always_inline)) {
    s = sums[0][t][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += sums[w][t][lane];
  };
  if constexpr (is8<Y>) {
    // wave w has the columns 16 w .. 16 w + 15 of the block, of MF times 16 rows
    static_assert(NF == kFewWaves, "a block of columns to a workgroup");
    __shared__ unsigned tops[MF][kFewWaves][16];
    f32x4_t v[MF];
    const int c = n0 + 16 * wave + 4 * grp;
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      take(wave * MF + f, v[f]);
      const int m = 16 * f + r;
      unsigned top = 0;
      if (m < g.m) {
        epilogue4<Y>(g, m, c, v[f]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (c + e >= g.n) v[f][e] = 0.f;
          const unsigned u = finite_bits(v[f][e]);
          top = top > u ? top : u;
        }
      }
#pragma unroll
      for (int d = 16; d <= 32; d <<= 1) {
        const unsigned o = (unsigned)__shfl_xor((int)top, d);
        top = top > o ? top : o;
      }
      if (grp == 0) tops[f][wave][r] = top;
    }
    __syncthreads();
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = 16 * f + r;
      unsigned top = 0;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) top = top > tops[f][w][r] ? top : tops[f][w][r];
      if (m < g.m) {
        const int byte = scale_byte(top);
        float q[8] = {v[f][0], v[f][1], v[f][2], v[f][3], 0.f, 0.f, 0.f, 0.f};
        to_units(q, byte, q);
        *reinterpret_cast<unsigned*>(g.y8 + (long long)m * g.ld_y8 + c) = to_e4m3(q)[0];
        if (wave == 0 && grp == 0) {
          g.s8[(long long)m * g.sld_y8 + (n0 >> 7)] = (unsigned char)byte;
          if (n0 + 128 >= g.ld_y8) pad_scales(g, m);
        }
      }
    }
  } else {
    for (int t = wave; t < MF * NF; t += kFewWaves) {
      f32x4_t s;
      take(t, s);
      const int m = 16 * (t % MF) + r, c = n0 + 16 * (t / MF) + 4 * grp;
      if (m < g.m) {
        if constexpr (EPI) epilogue4<Y>(g, m, c, s);
        Y* y = static_cast<Y*>(g.y) + (long long)m * g.ldy + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < g.n) y[e] = from_f32<Y>(s[e]);
      }
    }
  }
}

}  // namespace muon
