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
// fp32, ds fp64 (it has rows x cols terms of either sign).
//
// Both passes read each element once and are bound by HBM.  As in layer norm a
// team of waves holds a row in registers, 8 consecutive columns per lane and
// chunk, stays for many rows, and has its next row on its way.
#include "muon_block.h"
#include "norm_device.h"

namespace muon {

// The sums over a row that two norms take one after the other: each call uses the
// other of two buffers, so one barrier per call is enough.
template <int TEAM, int N>
struct TeamSums {
  float (*buf)[N][16];
  int turn;
  template <int M>
  __device__ __forceinline__ void operator()(float (&v)[M], int tw, int lane) {
    static_assert(M <= N, "buffer");
    team_sum<TEAM>(v, buf[turn], tw, lane);
    turn ^= 1;
  }
};

// A row's mean and 1 / sqrt(variance + eps); x becomes the deviations.  The mean's
// own rounding is taken out by the sum of the deviations, as layer norm of fp32
// rows does it.
template <int NCH, typename Sums>
__device__ __forceinline__ void row_norm(float (&x)[NCH][8], const int (&col)[NCH], int cols, float n,
                                         bool rms, float eps, Sums& sums, int tw, int lane, float& mu,
                                         float& rstd) {
  mu = 0.f;
  if (!rms) {
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[k][i];
    sums(s, tw, lane);
    mu = s[0] / n;
  }
  float t[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = col[k] + i < cols ? x[k][i] - mu : 0.f;
      t[0] = fmaf(d, d, t[0]);
      t[1] += d;
    }
  sums(t, tw, lane);
  float var = t[0] / n;
  if (!rms) {
    const float off = t[1] / n, better = mu + off;
    mu = better == better ? better : mu;  // (an infinite mean stays one)
    var -= off * off;
    var = var < 0.f ? 0.f : var;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] -= mu;
  }
  rstd = 1.f / sqrtf(var + eps);
}

constexpr int forward_waves(int team) { return team > 1 ? team : 4; }

template <int XT, int BT, int TEAM, int NCH>
__global__ __launch_bounds__(64 * forward_waves(TEAM)) void residual_norm_kernel(ResidualArgs a) {
  using X = typename ElemOf<XT>::type;
  using B = typename ElemOf<BT>::type;
  constexpr int TEAMS = forward_waves(TEAM) / TEAM;
  __shared__ float buf[2][2][16];
  TeamSums<TEAM, 2> sums{buf, 0};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tw = wave % TEAM;
  const long long step = (long long)gridDim.x * TEAMS;
  const bool post = a.p.post_weight, rms = a.p.rms;
  const float s = a.p.scale ? *a.p.scale : 1.f, n = (float)a.cols;
  int col[NCH];
  float w[NCH][8], b[NCH][8], pw[NCH][8], pb[NCH][8];  // pw, pb times the gate
  auto vec = [&](const float* p, int c, float otherwise, float (&v)[8]) __attribute__((always_inline)) {
    if (p) {
      load8_edge(p + c, a.cols - c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = otherwise;
    }
  };
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = ((k * TEAM + tw) * 64 + lane) * 8;
    float gate[8];
    vec(a.p.weight, col[k], 1.f, w[k]);
    vec(a.p.bias, col[k], 0.f, b[k]);
    vec(a.p.gate, col[k], 1.f, gate);
    vec(a.p.post_weight, col[k], 1.f, pw[k]);
    vec(a.p.post_bias, col[k], 0.f, pb[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pw[k][i] *= gate[i];
      pb[k][i] *= gate[i];
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
    if (post) row_norm(v, col, a.cols, n, rms, a.p.eps, sums, tw, lane, pmu, prstd);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = fmaf(v[k][i] * prstd, pw[k][i], pb[k][i]);
        v[k][i] = col[k] + i < a.cols ? fmaf(s, x[k][i], p) : 0.f;
      }
      if (a.r) store8_edge(static_cast<X*>(a.r) + row * a.ldr + col[k], a.cols - col[k], v[k]);
    }
    float mu, rstd;
    row_norm(v, col, a.cols, n, rms, a.p.eps, sums, tw, lane, mu, rstd);
    if (tw == 0 && lane == 0) {
      a.stats[row] = mu;
      a.stats[a.rows + row] = rstd;
      a.stats[2LL * a.rows + row] = post ? pmu : 0.f;
      a.stats[3LL * a.rows + row] = post ? prstd : 0.f;
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(v[k][i] * rstd, w[k][i], b[k][i]);
      if (a.h_type == kOut8) {
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col[k] + i >= a.cols) y[i] = 0.f;
          const unsigned f = finite_bits(y[i]);
          top = top > f ? top : f;
        }
        const int byte = scale_byte(max16(top));
        to_units(y, byte, y);
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

// Waves of a backward workgroup: whole teams, about eight.
constexpr int back_waves(int team) { return team > 8 ? team : 8 / team * team; }

// A team without a row left still takes part in the workgroup's barriers.
template <int XT, int BT, int TEAM, int NCH, bool BRANCH>
__global__ __launch_bounds__(64 * back_waves(TEAM)) void residual_back_kernel(ResidualBackArgs a) {
  using X = typename ElemOf<XT>::type;
  using B = typename ElemOf<BT>::type;
  constexpr int WAVES = back_waves(TEAM), TEAMS = WAVES / TEAM, K = BRANCH ? 4 : 2;
  // fp32 rows of several chunks leave no room for the next one
  constexpr bool EARLY = XT == MUON_BF16 || NCH == 1;
  __shared__ float buf[2][TEAMS][2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tw = wave % TEAM, team = wave / TEAM;
  const long long step = (long long)gridDim.x * TEAMS;
  const bool post = a.p.post_weight;
  const float s = a.p.scale ? *a.p.scale : 1.f, n = (float)a.cols, centre = a.p.rms ? 0.f : 1.f / n;
  int col[NCH];
  float w[NCH][8], wp[BRANCH ? NCH : 1][8];  // wp: post weight times gate
  float sum[K][NCH][8];                      // dh rh, dh, d bh, d
  double dscale = 0.0;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = ((k * TEAM + tw) * 64 + lane) * 8;
    load8_edge(a.p.weight + col[k], a.cols - col[k], w[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < K; ++j) sum[j][k][i] = 0.f;
    if constexpr (BRANCH) {
      float g[8], p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = p[i] = col[k] + i < a.cols ? 1.f : 0.f;
      if (a.p.gate) load8_edge(a.p.gate + col[k], a.cols - col[k], g);
      if (post) load8_edge(a.p.post_weight + col[k], a.cols - col[k], p);
#pragma unroll
      for (int i = 0; i < 8; ++i) wp[k][i] = g[i] * p[i];
    }
  }
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
      if (a.dr) rdr[k].load(static_cast<const X*>(a.dr) + row * a.lddr + col[k], left);
      if (BRANCH) rb[k].load(static_cast<const B*>(a.b) + row * a.ldb + col[k], left);
      if (a.g.scale) rx[k].load(static_cast<const X*>(a.x) + row * a.ldx + col[k], left);
    }
  };
  int turn = 0;
  long long first = (long long)blockIdx.x * TEAMS;  // of the workgroup's teams
  if (EARLY && first + team < a.rows) fetch(first + team);
  for (; first < a.rows; first += step) {
    const long long row = first + team;
    const bool in = row < a.rows;
    if (!EARLY && in) fetch(row);
    const float mu = st[0], r = st[1], pmu = st[2], pr = post ? st[3] : 1.f;
    float x[NCH][8], d[NCH][8], dr[NCH][8], bh[BRANCH ? NCH : 1][8];
    float c[2] = {0.f, 0.f};
    float ds = 0.f;
    if (in) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        rr[k].get(x[k]);
        rdh[k].get(d[k]);
        if (a.dr) {
          rdr[k].get(dr[k]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dr[k][i] = 0.f;
        }
        if constexpr (BRANCH) rb[k].get(bh[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float rh = col[k] + i < a.cols ? (x[k][i] - mu) * r : 0.f;
          sum[0][k][i] = fmaf(d[k][i], rh, sum[0][k][i]);
          sum[1][k][i] += d[k][i];
          const float g = d[k][i] * w[k][i];
          c[0] += g;
          c[1] = fmaf(g, rh, c[1]);
          x[k][i] = rh;
          d[k][i] = g;
        }
      }
    }
    team_sum<TEAM>(c, buf[turn][team], tw, lane);
    turn ^= 1;
    float e[2] = {0.f, 0.f};
    if (in) {
      const float c0 = c[0] * centre, c1 = c[1] / n;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float xs[8];
        if (a.g.scale) rx[k].get(xs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = fmaf(r, d[k][i] - c0 - x[k][i] * c1, dr[k][i]);
          if (a.g.scale) ds = fmaf(v, xs[i], ds);
          d[k][i] = v;
          if constexpr (BRANCH) {
            const float h = col[k] + i < a.cols ? (bh[k][i] - pmu) * pr : 0.f;
            sum[2][k][i] = fmaf(v, h, sum[2][k][i]);
            sum[3][k][i] += v;
            const float g = v * wp[k][i];
            e[0] += g;
            e[1] = fmaf(g, h, e[1]);
            bh[k][i] = h;
          }
        }
      }
      dscale += (double)ds;
      if (EARLY && row + step < a.rows) fetch(row + step);
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
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (BRANCH) {
            const float g = d[k][i] * wp[k][i];
            o[i] = post ? pr * (g - e0 - bh[k][i] * e1) : g;
          } else {
            o[i] = d[k][i];
          }
        }
        store8_edge(static_cast<B*>(a.db) + row * a.lddb + col[k], a.cols - col[k], o);
      }
    }
  }
  // The workgroup's sums: every team's go to LDS (element i of a chunk's lanes side
  // by side, the rows of 64 padded by one) and are added in the teams' order.
  constexpr int ROW = 65, PER = NCH * TEAM * 8 * ROW;
  __shared__ float acc[TEAMS * PER];
  float* part = a.part + (long long)blockIdx.x * K * a.cols;
#pragma unroll
  for (int j = 0; j < K; ++j) {
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[team * PER + ((k * TEAM + tw) * 8 + i) * ROW + lane] = sum[j][k][i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += 64 * WAVES) {
      const int at = ((c >> 9) * 8 + (c & 7)) * ROW + ((c >> 3) & 63);
      float v = acc[at];
#pragma unroll
      for (int t = 1; t < TEAMS; ++t) v += acc[t * PER + at];
      part[(long long)j * a.cols + c] = v;
    }
    __syncthreads();
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
void with_shape(int cols, bool branch, F&& f) {
#define MUON_SHAPE(T, N) f(std::integral_constant<int, T>{}, std::integral_constant<int, N>{})
  if (cols <= 512) MUON_SHAPE(1, 1);
  else if (cols <= 1024) MUON_SHAPE(1, 2);
  else if (cols <= 1536) MUON_SHAPE(BACK ? 3 : 1, BACK ? 1 : 3);
  else if (cols <= 2048) MUON_SHAPE(2, 2);
  else if (cols <= 4096) MUON_SHAPE(4, 2);
  else if (cols <= 8192) MUON_SHAPE(8, 2);
  else MUON_SHAPE(16, 2);
#undef MUON_SHAPE
}
int groups_for(int rows, int teams, int most) {
  const long long g = ((long long)rows + teams - 1) / teams;
  return (int)(g < most ? g : most);
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

// Workgroups of the backward pass, each with its partial sums: one per CU.
int residual_back_groups(int rows, int cols, bool branch) {
  int g = 0;
  with_shape<true>(cols, branch, [&](auto team, auto) {
    constexpr int T = decltype(team)::value;
    g = groups_for(rows, back_waves(T) / T, 256);
  });
  return g;
}

hipError_t launch_residual_norm(int x_bf16, int b_bf16, const ResidualArgs& a, hipStream_t s) {
  with_types(x_bf16, b_bf16, [&](auto xt, auto bt) {
    with_shape<false>(a.cols, false, [&](auto team, auto nch) {
      constexpr int T = decltype(team)::value, N = decltype(nch)::value;
      constexpr int waves = forward_waves(T);
      const dim3 grid(groups_for(a.rows, waves / T, 8192 / waves)), block(64 * waves);
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
      with_shape<true>(a.cols, branch, [&](auto team, auto nch) {
        constexpr int T = decltype(team)::value, N = decltype(nch)::value;
        constexpr int X = decltype(xt)::value, B = decltype(bt)::value;
        const dim3 grid(a.groups), block(64 * back_waves(T));
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
