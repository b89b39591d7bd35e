// The norms after and before a block, fused with the block's gate and the
// residual stream's scale:
//   p = N(branch) pw + pb  (or the branch itself),  r = s x + gate p,
//   h = N(r) w + b,        N(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps)
// or, for RMS norms, the same with a mean of zero; and backward, with
// vh = N's result before its weight, for g = dh w, d the gradient of r:
//   d = dr + rstd (g - mean(g) - rh mean(g rh))          (RMS: without mean(g))
//   dx = s d,  ds = sum(d x),  dw = sum over rows of dh rh,  db of dh
//   e = d gate pw,  dbranch = post rstd (e - mean(e) - bh mean(e bh))
// With S1 = sum over rows of d bh and S0 of d, the branch's parameters are
//   dpw = gate S1,  dpb = gate S0,  dgate = pw S1 + pb S0,
// so that four sums per column serve five gradients.
// h comes from r in fp32, before r is rounded to the stream's type.  All sums are
// fp32, ds fp64 over pairs in fp32: it has rows x cols terms of either sign.  Whole
// lanes of a row in fp32 were 1.1 to 1.7 times as far off (4096 x 1280 by 1.9 against
// 1.1 times 2^-24 sqrt(terms)) for 0 to 3% less time (16384 columns -8 to 9%); with
// every term in fp64 it is off by 1.0 and costs up to 14% (16384 x 1280 fp32, bf16
// branch: 104, 105 and 118 us, before rh, d and bh were made zeros past the last column,
// which costs 2 us more there).
//
// Both passes read each element once and are bound by HBM:
//   16384 x 1280 fp32, bf16 branch, gate and scale, to 8 bits 46 to 48 us (4.9 TB/s; a
//   copy runs at 5.2); 8192 x 4096 bf16 with everything 57 to 60 us (4.6); backward 96 to
//   98 us (4.8) and 6 for the sums' reduction, 4096 x 8192 107 and 8, and of the RMS norm
//   and residual sum alone 55 and 5 us (8192 x 4096).
// As in layer norm a team of waves holds a row in registers, 8 consecutive columns
// per lane (a chunk: 512 columns per wave), stays for many rows, and has its next row
// on its way.  One chunk to a lane up to 8192 columns, in the backward pass up to 4096:
// with two or three the vectors and sums left room for half the waves (1280 columns
// forward 61 us instead of 55, backward 118 instead of 82, 4096 columns backward 182
// instead of 105).  Where rows are short of whole chunks (640, 1280) and both norms are
// there, the vector unit bounds: 16384 x 1280 bf16 with everything 55 us forward, 91 and 5
// backward (floors 32 and 57).
#include "muon_block.h"
#include "norm_device.h"

namespace muon {

// Columns of a row that wave w of a team has.
template <int TEAM, int NCH>
__device__ __forceinline__ float columns_of(int w, int cols) {
  int c = 0;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int left = cols - (k * TEAM + w) * 512;
    c += left < 0 ? 0 : left < 512 ? left : 512;
  }
  return (float)c;
}

// Zeros past the last column, of which `left` are in front: a finite mean times a finite
// 1 / sqrt(variance + eps) may be an infinity there, which a weight of zero turns into
// NaN.  Every row is longer than all of a lane's chunks but the last (with_shape).
__device__ __forceinline__ void zero_past(float (&v)[8], int left) {
  if (left < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? v[i] : 0.f;
  }
}

// A row's mean and 1 / sqrt(variance + eps); x becomes the deviations.  Each wave
// takes the mean of its own columns and the squared deviations from that, corrected
// by the sum of the deviations (which are the mean's rounding), and the team joins
// them behind one barrier: with c_w columns, mean m_w and sum M_w of wave w
//   mean = m_0 + sum c_w (m_w - m_0) / n,  sum = sum M_w + c_w (m_w - mean)^2,
// so that a row of equal values has that value as its mean, exactly.  Lane l of each
// row of 16 takes wave l's part (`share`: its columns).  `buf` alternates between calls.
// past: what lies past the last column is used, and becomes zeros.
template <int TEAM, int NCH>
__device__ __forceinline__ void row_norm(float (&x)[NCH][8], const int (&col)[NCH], int cols, bool rms,
                                         float eps, float (*buf)[16], int tw, int lane, float own,
                                         float share, bool past, float& mu, float& rstd) {
  const float n = (float)cols;
  float t[2] = {0.f, 0.f};
  mu = 0.f;
  if (rms) {
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[0] = fmaf(x[k][i], x[k][i], t[0]);
    float q[1] = {t[0]};
    team_sum<TEAM>(q, buf, tw, lane);
    rstd = 1.f / sqrtf(q[0] / n + eps);
    return;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[k][i];
  const float inv = own > 0.f ? 1.f / own : 0.f;
  float m = wave_sum(s) * inv;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int left = cols - col[k];
    if (left >= 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = x[k][i] - m;
        t[0] = fmaf(d, d, t[0]);
        t[1] += d;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < left ? x[k][i] - m : 0.f;
        t[0] = fmaf(d, d, t[0]);
        t[1] += d;
      }
    }
  }
  t[0] = wave_sum(t[0]);
  t[1] = wave_sum(t[1]);
  const float off = t[1] * inv, better = m + off;
  m = better == better ? better : m;  // (an infinite mean stays one)
  t[0] = fmaf(-t[1], off, t[0]);
  t[0] = t[0] < 0.f ? 0.f : t[0];
  mu = m;
  float sum = t[0];
  if constexpr (TEAM > 1) {
    if (lane == 0) {
      buf[0][tw] = m;
      buf[1][tw] = t[0];
    }
    __syncthreads();
    const int l = lane & 15;
    const float m0 = buf[0][0], ml = buf[0][l < TEAM ? l : 0], ql = buf[1][l < TEAM ? l : 0];
    mu = m0 + sum16(l < TEAM ? share * (ml - m0) : 0.f) / n;
    if (mu != mu) mu = sum16(l < TEAM ? share * ml : 0.f) / n;  // an infinite mean, as the formula has it
    const float e = ml - mu;
    sum = sum16(l < TEAM ? fmaf(share * e, e, ql) : 0.f);
  }
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[k][i] -= mu;
    if (past && k == NCH - 1) zero_past(x[k], cols - col[k]);
  }
  rstd = 1.f / sqrtf(sum / n + eps);
}

constexpr int forward_waves(int team) { return team > 1 ? team : 4; }

template <int XT, int BT, int TEAM, int NCH>
__global__ __launch_bounds__(64 * forward_waves(TEAM)) void residual_norm_kernel(ResidualArgs a) {
  using X = typename ElemOf<XT>::type;
  using B = typename ElemOf<BT>::type;
  constexpr int TEAMS = forward_waves(TEAM) / TEAM;
  __shared__ float buf[2][2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tw = wave % TEAM;
  const long long step = (long long)gridDim.x * TEAMS;
  const bool post = a.p.post_weight, rms = a.p.rms;
  const float s = a.p.scale ? *a.p.scale : 1.f;
  const float own = columns_of<TEAM, NCH>(tw, a.cols), share = columns_of<TEAM, NCH>(lane & 15, a.cols);
  // rows too long for the registers have their vectors read again for each row
  constexpr bool LEAN = TEAM * NCH > 16;
  int col[NCH];
  float w[LEAN ? 1 : NCH][8], b[LEAN ? 1 : NCH][8];
  float pw[LEAN ? 1 : NCH][8], pb[LEAN ? 1 : NCH][8];  // times the gate
  // columns past the last one have zeros everywhere: nothing below asks for them
  auto vec = [&](const float* p, int c, float otherwise, float (&v)[8]) __attribute__((always_inline)) {
    if (p) {
      load8_edge(p + c, a.cols - c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < a.cols ? otherwise : 0.f;
    }
  };
  auto vectors_in = [&](int c, float (&w)[8], float (&b)[8]) __attribute__((always_inline)) {
    vec(a.p.weight, c, 1.f, w);
    vec(a.p.bias, c, 0.f, b);
  };
  auto vectors_post = [&](int c, float (&pw)[8], float (&pb)[8]) __attribute__((always_inline)) {
    float gate[8];
    vec(a.p.gate, c, 1.f, gate);
    vec(a.p.post_weight, c, 1.f, pw);
    vec(a.p.post_bias, c, 0.f, pb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pw[i] *= gate[i];
      pb[i] *= gate[i];
    }
  };
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = ((k * TEAM + tw) * 64 + lane) * 8;
    if constexpr (!LEAN) {
      vectors_in(col[k], w[k], b[k]);
      vectors_post(col[k], pw[k], pb[k]);
    }
  }
  Raw8<X> rx[NCH];
  Raw8<B> rb[NCH];
  auto fetch = [&](long long row) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      rx[k].load(static_cast<const X*>(a.x) + row * a.ldx + col[k], a.cols - col[k]);
      if (a.b) rb[k].load(static_cast<const B*>(a.b) + row * a.ldb + col[k], a.cols - col[k]);
    }
  };
  int turn = 0;
  long long row = (long long)blockIdx.x * TEAMS + wave / TEAM;
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += step) {
    float x[NCH][8], v[NCH][8];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      rx[k].get(x[k]);
      if (a.b) {
        rb[k].get(v[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
      }
    }
    if (row + step < a.rows) fetch(row + step);
    float pmu = 0.f, prstd = 1.f;
    if (post)
      row_norm<TEAM>(v, col, a.cols, rms, a.p.eps, buf[0], tw, lane, own, share, true, pmu,
                     prstd);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      constexpr int ONE = LEAN ? 0 : 1;
      if constexpr (LEAN) vectors_post(col[k], pw[0], pb[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[k][i] = fmaf(s, x[k][i], fmaf(v[k][i] * prstd, pw[k * ONE][i], pb[k * ONE][i]));
      if (a.r) store8_edge(static_cast<X*>(a.r) + row * a.ldr + col[k], a.cols - col[k], v[k]);
    }
    float mu, rstd;
    row_norm<TEAM>(v, col, a.cols, rms, a.p.eps, buf[post ? 1 : turn], tw, lane, own, share, false,
                   mu, rstd);
    turn ^= 1;
    if (tw == 0 && lane == 0) {
      a.stats[row] = mu;
      a.stats[a.rows + row] = rstd;
      a.stats[2LL * a.rows + row] = post ? pmu : 0.f;
      a.stats[3LL * a.rows + row] = post ? prstd : 0.f;
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float y[8];
      constexpr int ONE = LEAN ? 0 : 1;
      if constexpr (LEAN) vectors_in(col[k], w[0], b[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(v[k][i] * rstd, w[k * ONE][i], b[k * ONE][i]);
      if (a.h_type == kOut8) {
        if (a.cols - col[k] < 8) {  // (a row that is not finite has NaN there)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = col[k] + i < a.cols ? y[i] : 0.f;
        }
        const int byte = block_units(y, y);
        if (col[k] < a.ld) *reinterpret_cast<u32x2_t*>(a.h8 + row * a.ld + col[k]) = to_e4m3(y);
        const unsigned word = pack_scales(byte);
        const int piece = k * TEAM + tw;
        if (lane == 0 && 4 * piece < a.sld)
          *reinterpret_cast<unsigned*>(a.s8 + row * a.sld + 4 * piece) = word;
      } else if (a.h_type == MUON_BF16) {
        store8_edge(static_cast<bf16_t*>(a.h) + row * a.ldh + col[k], a.cols - col[k], y);
      } else {
        store8_edge(static_cast<float*>(a.h) + row * a.ldh + col[k], a.cols - col[k], y);
      }
    }
  }
}

// Waves of a backward workgroup, of which a CU holds one: whole teams, as many as
// the registers allow (up to 170 a lane for 12, 128 for 16).
constexpr int back_waves(int team, bool branch, bool fp32) {
  const int most = !branch ? 16 : fp32 ? 8 : 12;
  return team >= 8 ? team : most / team * team;
}
// Where a lane has 16 columns their sums do not fit its registers: as many of them
// as there is room for are kept in LDS.
constexpr int back_lds(int team, int nch, bool branch) {
  return nch == 1 ? 0 : team == 16 ? 2 : branch ? 4 : 0;
}

// A team without a row left still takes part in the workgroup's barriers.
template <int XT, int BT, int TEAM, int NCH, bool BRANCH>
__global__ __launch_bounds__(64 * back_waves(TEAM, BRANCH, BT == MUON_FP32)) void
residual_back_kernel(ResidualBackArgs a) {
  using X = typename ElemOf<XT>::type;
  using B = typename ElemOf<BT>::type;
  constexpr int WAVES = back_waves(TEAM, BRANCH, BT == MUON_FP32), TEAMS = WAVES / TEAM;
  constexpr int K = BRANCH ? 4 : 2, LDS = back_lds(TEAM, NCH, BRANCH);
  // rows too long for the registers have their vectors read again for each row, and
  // their next one, as fp32 rows of several chunks, when its turn comes
  constexpr bool LEAN = TEAM * NCH > 16;
  constexpr bool EARLY = NCH == 1 || (XT == MUON_BF16 && !LEAN);
  // Chunks that zero_past is asked about: the last one.  Rows too long for the registers
  // spill less with its branch in both (2048 x 16384, branch parameters: 337 us and 459).
  constexpr auto EDGE = [](int k) { return LEAN || k == NCH - 1; };
  __shared__ float buf[2][TEAMS][2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tw = wave % TEAM, team = wave / TEAM;
  const long long step = (long long)gridDim.x * TEAMS;
  const bool post = a.p.post_weight;
  const float s = a.p.scale ? *a.p.scale : 1.f, n = (float)a.cols, centre = a.p.rms ? 0.f : 1.f / n;
  int col[NCH];
  float w[LEAN ? 1 : NCH][8], wp[BRANCH && !LEAN ? NCH : 1][8];  // wp: post weight times gate
  // sums of dh rh, dh, d bh, d: in registers or, four columns of a lane side by side
  // with its neighbours', in LDS
  float reg_sum[LDS < K ? K - LDS : 1][NCH][8];
  __shared__ f32x4_t lds_sum[LDS ? LDS * NCH * 2 * 64 * WAVES : 1];
  f32x4_t* own = lds_sum + threadIdx.x;
  auto add = [&](auto j, auto k, const float (&v)[8]) __attribute__((always_inline)) {
    constexpr int J = decltype(j)::value, C = decltype(k)::value;
    if constexpr (J < LDS) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        f32x4_t& s = own[((J * NCH + C) * 2 + q) * 64 * WAVES];
        f32x4_t t = s;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] += v[4 * q + e];
        s = t;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) reg_sum[J - LDS][C][i] += v[i];
    }
  };
  double dscale = 0.0;
  auto branch_weight = [&](int c, float (&v)[8]) __attribute__((always_inline)) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = g[i] = c + i < a.cols ? 1.f : 0.f;
    if (a.p.gate) load8_edge(a.p.gate + c, a.cols - c, g);
    if (post) load8_edge(a.p.post_weight + c, a.cols - c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= g[i];
  };
  static_for<NCH>([&](auto kk) {
    constexpr int k = decltype(kk)::value;
    col[k] = ((k * TEAM + tw) * 64 + lane) * 8;
    static_for<K>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      if constexpr (j < LDS) {
        own[((j * NCH + k) * 2) * 64 * WAVES] = own[((j * NCH + k) * 2 + 1) * 64 * WAVES] = f32x4_t{};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) reg_sum[j - LDS][k][i] = 0.f;
      }
    });
    if constexpr (!LEAN) {
      load8_edge(a.p.weight + col[k], a.cols - col[k], w[k]);
      if constexpr (BRANCH) branch_weight(col[k], wp[k]);
    }
  });
  Raw8<X> rr[NCH], rdr[NCH], rx[NCH];
  Raw8<B> rdh[NCH], rb[NCH];
  float st[4] = {0.f, 0.f, 0.f, 0.f};
  auto fetch = [&](long long row) __attribute__((always_inline)) {
    st[0] = a.stats[row];
    st[1] = a.stats[a.rows + row];
    if (BRANCH && post) {
      st[2] = a.stats[2LL * a.rows + row];
      st[3] = a.stats[3LL * a.rows + row];
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int left = a.cols - col[k];
      rr[k].load(static_cast<const X*>(a.r) + row * a.ldr + col[k], left);
      rdh[k].load(static_cast<const B*>(a.dh) + row * a.lddh + col[k], left);
    }
  };
  // what is not used before the first sums are known
  auto fetch_late = [&](long long row) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int left = a.cols - col[k];
      if (a.dr) rdr[k].load(static_cast<const X*>(a.dr) + row * a.lddr + col[k], left);
      if (BRANCH) rb[k].load(static_cast<const B*>(a.b) + row * a.ldb + col[k], left);
      if (a.g.scale) rx[k].load(static_cast<const X*>(a.x) + row * a.ldx + col[k], left);
    }
  };
  int turn = 0;
  long long first = (long long)blockIdx.x * TEAMS;  // of the workgroup's teams
  if (EARLY && first + team < a.rows) {
    fetch(first + team);
    fetch_late(first + team);
  }
  for (; first < a.rows; first += step) {
    const long long row = first + team;
    const bool in = row < a.rows;
    if (!EARLY && in) {
      fetch(row);
      if (!LEAN) fetch_late(row);
    }
    const float mu = st[0], r = st[1], pmu = st[2], pr = post ? st[3] : 1.f;
    float x[NCH][8], d[NCH][8], bh[BRANCH ? NCH : 1][8];
    float c[2] = {0.f, 0.f};
    if (in) {
      static_for<NCH>([&](auto kk) {
        constexpr int k = decltype(kk)::value;
        rr[k].get(x[k]);
        rdh[k].get(d[k]);
        float p[8];
        add(std::integral_constant<int, 1>{}, kk, d[k]);
        constexpr int kw = LEAN ? 0 : k;
        if constexpr (LEAN) load8_edge(a.p.weight + col[k], a.cols - col[k], w[0]);
        // past the last column dh, x and the weights are zeros, and rh, d and bh are
        // made so: no sum over the row gets anything from it
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = (x[k][i] - mu) * r;
        if constexpr (EDGE(k)) zero_past(x[k], a.cols - col[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float rh = x[k][i];
          p[i] = d[k][i] * rh;
          const float g = d[k][i] * w[kw][i];
          c[0] += g;
          c[1] = fmaf(g, rh, c[1]);
          d[k][i] = g;
        }
        add(std::integral_constant<int, 0>{}, kk, p);
      });
    }
    team_sum<TEAM>(c, buf[turn][team], tw, lane);
    turn ^= 1;
    float e[2] = {0.f, 0.f};
    if (in) {
      const float c0 = c[0] * centre, c1 = c[1] / n;
      if (LEAN) fetch_late(row);
      static_for<NCH>([&](auto kk) {
        constexpr int k = decltype(kk)::value;
        float xs[8], p[8];
        constexpr int kw = LEAN || !BRANCH ? 0 : k;
        if constexpr (LEAN && BRANCH) branch_weight(col[k], wp[0]);
        if (a.g.scale) rx[k].get(xs);
        float dr[8];
        if (a.dr) {
          rdr[k].get(dr);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dr[i] = 0.f;
        }
        if constexpr (BRANCH) {
          rb[k].get(bh[k]);
#pragma unroll
          for (int i = 0; i < 8; ++i) bh[k][i] = (bh[k][i] - pmu) * pr;
          if constexpr (EDGE(k)) zero_past(bh[k], a.cols - col[k]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) d[k][i] = fmaf(r, d[k][i] - c0 - x[k][i] * c1, dr[i]);
        if constexpr (EDGE(k)) zero_past(d[k], a.cols - col[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = d[k][i];
          if (a.g.scale && i % 2) dscale += (double)fmaf(v, xs[i], d[k][i - 1] * xs[i - 1]);
          if constexpr (BRANCH) {
            const float h = bh[k][i];
            p[i] = v * h;
            const float g = v * wp[kw][i];
            e[0] += g;
            e[1] = fmaf(g, h, e[1]);
          }
        }
        if constexpr (BRANCH) {
          add(std::integral_constant<int, 2>{}, kk, p);
          add(std::integral_constant<int, 3>{}, kk, d[k]);
        }
      });
      if (EARLY && row + step < a.rows) {
        fetch(row + step);
        fetch_late(row + step);
      }
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = s * d[k][i];
        store8_edge(static_cast<X*>(a.dx) + row * a.lddx + col[k], a.cols - col[k], o);
      }
    }
    if (BRANCH && post) {
      team_sum<TEAM>(e, buf[turn][team], tw, lane);
      turn ^= 1;
    }
    if (in && a.db) {
      const float e0 = e[0] * centre, e1 = e[1] / n;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float o[8];
        constexpr int ONE = LEAN ? 0 : 1;
        if constexpr (LEAN && BRANCH) branch_weight(col[k], wp[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (BRANCH) {
            const float g = d[k][i] * wp[k * ONE][i];
            o[i] = post ? pr * (g - e0 - bh[k][i] * e1) : g;
          } else {
            o[i] = d[k][i];
          }
        }
        store8_edge(static_cast<B*>(a.db) + row * a.lddb + col[k], a.cols - col[k], o);
      }
    }
  }
  // The workgroup's sums.  Those of several teams go to LDS one after the other
  // (element i of a chunk's lanes side by side, the rows of 64 padded by one) and are
  // added in the teams' order; a single team's are what it has.
  float* part = a.part + (long long)blockIdx.x * K * a.cols;
  if constexpr (TEAMS == 1) {
    static_for<K>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      static_for<NCH>([&](auto kk) {
        constexpr int k = decltype(kk)::value;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (j < LDS)
            v[i] = own[((j * NCH + k) * 2 + i / 4) * 64 * WAVES][i % 4];
          else
            v[i] = reg_sum[j - LDS][k][i];
        }
        store8_edge(part + (long long)j * a.cols + col[k], a.cols - col[k], v);
      });
    });
  } else {
    constexpr int ROW = 65, PER = NCH * TEAM * 8 * ROW;
    __shared__ float acc[TEAMS * PER];
    static_for<K>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[team * PER + ((k * TEAM + tw) * 8 + i) * ROW + lane] = reg_sum[j][k][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += 64 * WAVES) {
        const int at = ((c >> 9) * 8 + (c & 7)) * ROW + ((c >> 3) & 63);
        float v = acc[at];
#pragma unroll
        for (int t = 1; t < TEAMS; ++t) v += acc[t * PER + at];
        part[(long long)j * a.cols + c] = v;
      }
      __syncthreads();
    });
  }
  if (a.g.scale) {
    __shared__ double dbuf[16];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) dscale += __shfl_xor(dscale, o);
    if (lane == 0) dbuf[wave] = dscale;
    __syncthreads();
    if (threadIdx.x == 0) {
      double v = 0.0;
      for (int k = 0; k < WAVES; ++k) v += dbuf[k];
      a.part_scale[blockIdx.x] = v;
    }
  }
}

// The parameters' gradients from the workgroups' sums, in their order: 32 columns
// per workgroup, 32 threads to a column, two of the sums each: the norm's weight and
// bias (blockIdx.y 0), or the branch's parameters (1).  One workgroup more adds the
// scale's.
__global__ __launch_bounds__(1024) void residual_reduce_kernel(ResidualBackArgs a, int k, int ystart) {
  __shared__ float acc[2][32][33];
  __shared__ double dacc[16];
  const int y = (int)blockIdx.y + ystart;
  auto put = [&](float* out, int c, float v) __attribute__((always_inline)) {
    if (out) out[c] = a.accumulate ? out[c] + v : v;
  };
  if (y == 2) {
    if (blockIdx.x > 0) return;
    double v = 0.0;
    for (int g = threadIdx.x; g < a.groups; g += 1024) v += a.part_scale[g];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) dacc[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      v = 0.0;
      for (int i = 0; i < 16; ++i) v += dacc[i];
      put(a.g.scale, 0, (float)v);
    }
    return;
  }
  const int x = threadIdx.x & 31, g0 = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float s[2] = {0.f, 0.f};
  if (c < a.cols) {
    const float* p = a.part + (long long)2 * y * a.cols + c;
#pragma unroll 4
    for (int g = g0; g < a.groups; g += 32) {
      s[0] += p[(long long)g * k * a.cols];
      s[1] += p[((long long)g * k + 1) * a.cols];
    }
  }
  acc[0][g0][x] = s[0];
  acc[1][g0][x] = s[1];
  __syncthreads();
  if (g0 > 0 || c >= a.cols) return;
  s[0] = s[1] = 0.f;
#pragma unroll
  for (int g = 0; g < 32; ++g) {
    s[0] += acc[0][g][x];
    s[1] += acc[1][g][x];
  }
  if (y == 0) {
    put(a.g.weight, c, s[0]);
    put(a.g.bias, c, s[1]);
  } else {
    const float gate = a.p.gate ? a.p.gate[c] : 1.f;
    put(a.g.post_weight, c, gate * s[0]);
    put(a.g.post_bias, c, gate * s[1]);
    const float pw = a.p.post_weight ? a.p.post_weight[c] : 1.f;
    const float pb = a.p.post_bias ? a.p.post_bias[c] : 0.f;
    put(a.g.gate, c, fmaf(pw, s[0], pb * s[1]));
  }
}

namespace {
// Team and chunks for a row of `cols` columns: few enough chunks for the weights
// and, in the backward pass, the columns' sums to stay in registers.
template <bool BACK, typename F>
void with_shape(int cols, F&& f) {
#define MUON_SHAPE(T, N) f(std::integral_constant<int, T>{}, std::integral_constant<int, N>{})
  if constexpr (BACK) {
    if (cols <= 512) MUON_SHAPE(1, 1);
    else if (cols <= 1024) MUON_SHAPE(2, 1);
    else if (cols <= 1536) MUON_SHAPE(3, 1);
    else if (cols <= 2048) MUON_SHAPE(4, 1);
    else if (cols <= 4096) MUON_SHAPE(8, 1);
    else if (cols <= 8192) MUON_SHAPE(8, 2);
    else MUON_SHAPE(16, 2);
  } else {
    if (cols <= 512) MUON_SHAPE(1, 1);
    else if (cols <= 1024) MUON_SHAPE(2, 1);
    else if (cols <= 1536) MUON_SHAPE(3, 1);
    else if (cols <= 2048) MUON_SHAPE(4, 1);
    else if (cols <= 4096) MUON_SHAPE(8, 1);
    else if (cols <= 8192) MUON_SHAPE(16, 1);
    else MUON_SHAPE(16, 2);
  }
#undef MUON_SHAPE
}
// Workgroups for `rows` rows, `teams` to a workgroup, at most `most`, which are what the
// chip holds at once: as few as give none of them more rows than that many would.
int groups_for(int rows, int teams, int most) {
  const long long all = ((long long)rows + teams - 1) / teams;  // rows of a team
  const long long each = (all + most - 1) / most;
  return each > 0 ? (int)((all + each - 1) / each) : 0;
}
using Bf16 = std::integral_constant<int, MUON_BF16>;
using Fp32 = std::integral_constant<int, MUON_FP32>;
template <typename F>
void with_types(int x_bf16, int b_bf16, F&& f) {
  if (x_bf16) f(Bf16{}, Bf16{});
  else if (b_bf16) f(Fp32{}, Bf16{});
  else f(Fp32{}, Fp32{});
}
}  // namespace

// Workgroups of the backward pass, each with its partial sums: one per CU.  A branch in
// fp32 has fewer waves to a workgroup, and so more of these for a short batch: 2048 rows
// of 512 columns in one pass of 256 workgroups instead of two of 171, 14.5 us instead of
// 15.3 (1500 rows 14.0 instead of 15.2).
int residual_back_groups(int rows, int cols, bool branch, bool b_fp32) {
  int g = 0;
  with_shape<true>(cols, [&](auto team, auto) {
    constexpr int T = decltype(team)::value;
    g = groups_for(rows, back_waves(T, branch, b_fp32) / T, 256);
  });
  return g;
}

hipError_t launch_residual_norm(int x_bf16, int b_bf16, const ResidualArgs& a, hipStream_t s) {
  with_types(x_bf16, b_bf16, [&](auto xt, auto bt) {
    with_shape<false>(a.cols, [&](auto team, auto nch) {
      constexpr int T = decltype(team)::value, N = decltype(nch)::value;
      constexpr int waves = forward_waves(T);
      // 16 waves to a CU
      const dim3 grid(groups_for(a.rows, waves / T, 256 * (16 / waves))), block(64 * waves);
      hipLaunchKernelGGL((residual_norm_kernel<decltype(xt)::value, decltype(bt)::value, T, N>), grid,
                         block, 0, s, a);
    });
  });
  return hipGetLastError();
}

hipError_t launch_residual_norm_backward(int x_bf16, int b_bf16, const ResidualBackArgs& a,
                                         hipStream_t s) {
  const bool branch = residual_branch(a.p);
  if (a.groups > 0)
    with_types(x_bf16, b_bf16, [&](auto xt, auto bt) {
      with_shape<true>(a.cols, [&](auto team, auto nch) {
        constexpr int T = decltype(team)::value, N = decltype(nch)::value;
        constexpr int X = decltype(xt)::value, B = decltype(bt)::value;
        const dim3 grid(a.groups), block(64 * back_waves(T, branch, B == MUON_FP32));
        if (branch)
          hipLaunchKernelGGL((residual_back_kernel<X, B, T, N, true>), grid, block, 0, s, a);
        else
          hipLaunchKernelGGL((residual_back_kernel<X, B, T, N, false>), grid, block, 0, s, a);
      });
    });
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 cols((a.cols + 31) / 32, branch ? 2 : 1), block(1024);
  hipLaunchKernelGGL(residual_reduce_kernel, dim3(cols.x, cols.y + (a.g.scale && branch ? 1 : 0)),
                     block, 0, s, a, branch ? 4 : 2, 0);
  if (a.g.scale && !branch)
    hipLaunchKernelGGL(residual_reduce_kernel, dim3(1, 1), block, 0, s, a, 2, 2);
  return hipGetLastError();
}

}  // namespace muon
