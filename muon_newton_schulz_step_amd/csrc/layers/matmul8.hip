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
// (EXACT; 1e-7 of the norm).
//
// Two kernels:
//   tiles   both operands through LDS, for many rows of a: bound by the MFMAs;
//   rows    few rows of a (up to 32): bound by reading b once, so always exact.
#include "muon_gemm.h"

#include "fp8_device.h"
#include "muon_layer.h"

namespace muon {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t frag8(const u32x4_t& lo, const u32x4_t& hi) {
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
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
//   spill 8 (28 bytes a lane; to fp32 2).
//   A library's product with one scale per tensor runs at 2.72 to 2.80.  At the
//   larger size the MFMAs are busy 70% of the cycles and the chip runs at 1.68
//   GHz: it is bound by power.  Without the stores of y it would take 752 us.
//   4 waves of 128 x 128, 512 registers each: 110 us; 4 stages of 64 k: 116 us.
template <int BM, int BN, int WGM, int WGN, bool EXACT, bool STRM, typename Y>
__global__ __launch_bounds__(64 * WGM * WGN) void matmul8_tile_kernel(Matmul8Args g) {
  constexpr int NW = WGM * WGN;
  constexpr int WTM = BM / WGM, WTN = BN / WGN;
  constexpr int FM = WTM / 32, FN = WTN / 32;
  constexpr int CPR = 8;
  constexpr int B_CHUNKS = BN * CPR, STAGE = (BM + BN) * CPR;
  constexpr int DPW = STAGE / 64 / NW;      // loads of a wave per k-tile
  // and of 64 scale words per four; where there are more waves than those, the
  // others load the same again
  constexpr int SG = (BM + BN) / 64, SPW = SG > NW ? SG / NW : 1;
  static_assert(DPW * 64 * NW == STAGE && B_CHUNKS % (DPW * 64) == 0, "one operand per wave");
  static_assert((SG % NW == 0 || NW % SG == 0) && BN % (SPW * 64) == 0,
                "one operand's scales per wave");
  // the epilogue's staging: 32 rows m of half the wave's columns, per wave
  static_assert(FN % 2 == 0 && NW * 32 * (WTN / 2) * 4 <= STAGE * 16, "staging fits");
  __shared__ u32x4_t S0[STAGE], S1[STAGE];
  __shared__ unsigned C0[BM + BN], C1[BM + BN];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WGN, wn = wave % WGN;
  const int L = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int span = g.group_m * g.tiles_n;
  const int grp = L / span, first = grp * g.group_m;
  const int gm = g.tiles_m - first < g.group_m ? g.tiles_m - first : g.group_m;
  const int idx = L - grp * span;
  const int m0 = (first + idx % gm) * BM, n0 = (idx / gm) * BN;

  const int wave_s = __builtin_amdgcn_readfirstlane(wave);
  const bool is_b = wave_s * DPW * 64 < B_CHUNKS;
  const unsigned char* base = is_b ? g.b + (long long)n0 * g.ld : g.a + (long long)m0 * g.ld;
  const int last_row = is_b ? g.n - 1 - n0 : g.m - 1 - m0;
  unsigned voff[DPW];
#pragma unroll
  for (int d = 0; d < DPW; ++d) {
    const int q = (wave * DPW + d) * 64 + lane;
    const int r = q / CPR, rl = is_b ? r : r - BN;
    voff[d] = (unsigned)(rl < last_row ? rl : last_row) * (unsigned)g.ld + swz(q % CPR, r) * 16;
  }
  const int nk = g.ld / 128, last_word = (nk - 1) / 4;
  auto issue = [&](int kt, u32x4_t* St) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(base + (long long)kt * 128);
#pragma unroll
    for (int d = 0; d < DPW; ++d) buffer_load_lds16(rs, voff[d], St + (wave_s * DPW + d) * 64);
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
  // of 8 columns, neighbouring lanes neighbouring runs.
  constexpr int HC = WTN / 2, UPR = HC / 4, RPR = HC / 8;  // units, runs per staged row
  float* T = reinterpret_cast<float*>(S0) + wave * 32 * HC;
  auto unit = [](int r, int u) __attribute__((always_inline)) {
    return 4 * (r * UPR + (u ^ (r & (UPR - 1))));
  };
  Y* y = static_cast<Y*>(g.y);
#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < FN / 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16_t& c = acc[h * (FN / 2) + i][j];
          *reinterpret_cast<f32x4_t*>(T + unit(lane & 31, 8 * i + 2 * q + hsel)) =
              f32x4_t{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
        }
      // only this wave touches its part, and a wave's LDS accesses execute in
      // order: a compiler barrier orders them
      asm volatile("" ::: "memory");
#pragma unroll
      for (int s = 0; s < 32 * RPR / 64; ++s) {
        const int t = lane + 64 * s, rr = t / RPR, c = t % RPR;
        float v[8];
        const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(T + unit(rr, 2 * c));
        const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(T + unit(rr, 2 * c + 1));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = lo[e];
          v[4 + e] = hi[e];
        }
        const int m = m0 + wm * WTM + j * 32 + rr, n = n0 + wn * WTN + h * HC + 8 * c;
        if (m < g.m) store8_edge<STRM>(y + (long long)m * g.ldy + n, g.n - n, v);
      }
      asm volatile("" ::: "memory");
    }
}

// ---------------------------------------------------------------- rows
// Up to 16 MF rows m.  A workgroup takes 16 NF columns n and its 8 waves share
// the blocks of k between them; operands come straight from memory (each row of
// b is used once) and go to bf16 in registers: four v_mfma_f32_16x16x32_bf16 per
// block and 16 x 16 results.  The waves' sums are added in their order through
// LDS.  NF = 2 reads a half as often, once there are workgroups enough.
constexpr int kFewWaves = 8;

template <int MF, int NF, typename Y>
__global__ __launch_bounds__(64 * kFewWaves) void matmul8_rows_kernel(Matmul8Args g) {
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
  for (int t = wave; t < MF * NF; t += kFewWaves) {
    f32x4_t s = sums[0][t][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += sums[w][t][lane];
    const int m = 16 * (t % MF) + r, c = n0 + 16 * (t / MF) + 4 * grp;
    if (m < g.m) {
      Y* y = static_cast<Y*>(g.y) + (long long)m * g.ldy + c;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < g.n) y[e] = from_f32<Y>(s[e]);
    }
  }
}

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
