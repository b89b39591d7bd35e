// Layer norm over the last axis, forward and backward.
//   forward   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//             y = (x - mu) r w + b, mu and r kept for the backward pass
//   backward  xh = (x - mu) r, g = dy w:
//             dx = r (g - mean(g) - xh mean(g xh)),
//             dw = sum over rows of dy xh, db = sum over rows of dy
// All sums are fp32.  Both passes read each row once and are bound by HBM.
//
//   16384 x 1280 fp32 to bf16 23.8 us (5.3 TB/s), 8192 x 4096 bf16 24.4 us
//   (5.5 TB/s); backward 8192 x 4096 bf16 39.8 us (5.1 TB/s) and 4.3 us for the
//   reduction of 256 partial sums.  A 1 GiB copy runs at 5.2.  Short of that:
//   to 8 bits 16384 x 1280 21 us (3.0 TB/s), backward 4099 x 1280 from 8 bits
//   12.5 + 3.1 us (two rows to a wave, a join and a second launch).
// While a row is worked on, the team's next one is on its way (without: 30 us
// forward and 64 us backward of 8192 x 4096).
//
// A team of TEAM waves holds a row in registers, 8 consecutive columns per
// lane and chunk (a chunk: 512 columns per wave), so the mean and the sum of
// squared deviations are two passes over registers, not over memory.  Teams
// stay for many rows: the weights, and in the backward pass the columns'
// gradient sums, are in registers all along.
#include "muon_layer.h"
#include "norm_device.h"

namespace muon {

template <int XT, int OUT, int TEAM, int NCH>
__global__ __launch_bounds__(TEAM > 4 ? 64 * TEAM : 256) void layer_norm_kernel(NormArgs a) {
  using X = typename ElemOf<XT>::type;
  using Y = typename ElemOf<OUT>::type;
  constexpr int WAVES = TEAM > 4 ? TEAM : 4, TEAMS = WAVES / TEAM;
  __shared__ float sums[2][2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tw = wave % TEAM;
  const long long step = (long long)gridDim.x * TEAMS;
  int col[NCH];
  float w[NCH][8], b[NCH][8];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = ((k * TEAM + tw) * 64 + lane) * 8;
    load8_edge(a.weight + col[k], a.cols - col[k], w[k]);
    load8_edge(a.bias ? a.bias + col[k] : nullptr, a.bias ? a.cols - col[k] : 0, b[k]);
  }
  const float n = (float)a.cols;
  Raw8<X> raw[NCH];
  auto fetch = [&](long long row) __attribute__((always_inline)) {
    const X* xr = static_cast<const X*>(a.x) + row * a.ldx;
#pragma unroll
    for (int k = 0; k < NCH; ++k) raw[k].load(xr + col[k], a.cols - col[k]);
  };
  long long row = (long long)blockIdx.x * TEAMS + wave / TEAM;
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += step) {
    float x[NCH][8];
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      raw[k].get(x[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[k][i];
    }
    if (row + step < a.rows) fetch(row + step);
    team_sum<TEAM>(s, sums[0], tw, lane);
    // The sum's rounding leaves the mean off by a few steps of the row's average
    // magnitude, which in an fp32 row of little variance is much.  There the pass
    // that sums the squared deviations sums the deviations as well and corrects it:
    // in a row of equal values the mean is then that value, and y the bias (16384 x
    // 1280 23.0 -> 23.4 us).  bf16 values within a factor of two of each other are
    // at most 2^9 steps of one size, and 16384 of them add up without rounding;
    // where they spread further, so does their variance.
    constexpr bool CORRECT = XT == MUON_FP32;
    float mu = s[0] / n;
    float t[1 + CORRECT] = {};
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = col[k] + i < a.cols ? x[k][i] - mu : 0.f;
        t[0] = fmaf(d, d, t[0]);
        if constexpr (CORRECT)
          t[1] += d;
        else
          x[k][i] = d;
      }
    team_sum<TEAM>(t, sums[1], tw, lane);
    float var = t[0] / n;
    if constexpr (CORRECT) {
      const float off = t[1] / n, better = mu + off;
      mu = better == better ? better : mu;  // (an infinite mean stays one)
      var -= off * off;
      var = var < 0.f ? 0.f : var;
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] -= mu;
    }
    const float r = 1.f / sqrtf(var + a.eps);
    if (tw == 0 && lane == 0) {
      a.mean[row] = mu;
      a.rstd[row] = r;
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(x[k][i] * r, w[k][i], b[k][i]);
      if constexpr (OUT == kOut8) {
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col[k] + i >= a.cols) y[i] = 0.f;
          const unsigned f = finite_bits(y[i]);
          top = top > f ? top : f;
        }
        const int byte = scale_byte(max16(top));
        to_units(y, byte, y);
        if (col[k] < a.ld) *reinterpret_cast<u32x2_t*>(a.y8 + row * a.ld + col[k]) = to_e4m3(y);
        const unsigned word = pack_scales(byte);
        const int piece = k * TEAM + tw;
        if (lane == 0 && 4 * piece < a.sld)
          *reinterpret_cast<unsigned*>(a.s8 + row * a.sld + 4 * piece) = word;
      } else {
        store8_edge(static_cast<Y*>(a.y) + row * a.ldy + col[k], a.cols - col[k], y);
      }
    }
  }
}

// The input of the backward pass: eight elements of a row of x, from memory
// or from the 8-bit tensor.
template <int XT>
struct RawX {
  Raw8<typename ElemOf<XT>::type> r;
  __device__ __forceinline__ void load(const NormBackArgs& a, long long row, int col) {
    r.load(static_cast<const typename ElemOf<XT>::type*>(a.x) + row * a.ldx + col, a.cols - col);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { r.get(v); }
};
template <>
struct RawX<kOut8> {
  u32x2_t q;
  int byte;
  __device__ __forceinline__ void load(const NormBackArgs& a, long long row, int col) {
    q = u32x2_t{0u, 0u};
    byte = 127;
    if (col < a.ld) {
      q = *reinterpret_cast<const u32x2_t*>(a.x8 + row * a.ld + col);
      byte = a.sx8[(row >> a.shift) * a.sld + (col >> 7)];
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { from_e4m3(q, scale_of(byte), v); }
};

constexpr int back_waves(int team) { return team > 8 ? team : 8; }

// A team without a row left still takes part in the workgroup's barriers.
template <int DT, int XT, int TEAM, int NCH>
__global__ __launch_bounds__(64 * back_waves(TEAM)) void layer_norm_back_kernel(NormBackArgs a) {
  using D = typename ElemOf<DT>::type;
  constexpr int WAVES = back_waves(TEAM), TEAMS = WAVES / TEAM;
  // the next row does not fit the registers beside four chunks of fp32
  constexpr bool EARLY = NCH < 4 || (DT != MUON_FP32 && XT != MUON_FP32);
  __shared__ float sums[2][TEAMS][2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tw = wave % TEAM, team = wave / TEAM;
  const long long step = (long long)gridDim.x * TEAMS;
  int col[NCH];
  float w[NCH][8], dw[NCH][8], db[NCH][8];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    col[k] = ((k * TEAM + tw) * 64 + lane) * 8;
    load8_edge(a.weight + col[k], a.cols - col[k], w[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.f;
  }
  const float n = (float)a.cols;
  RawX<XT> rx[NCH];
  Raw8<D> rd[NCH];
  float mu_next = 0.f, r_next = 0.f;
  auto fetch = [&](long long row) __attribute__((always_inline)) {
    mu_next = a.mean[row];
    r_next = a.rstd[row];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      rx[k].load(a, row, col[k]);
      rd[k].load(static_cast<const D*>(a.dy) + row * a.lddy + col[k], a.cols - col[k]);
    }
  };
  int turn = 0;
  long long first = (long long)blockIdx.x * TEAMS;  // of the workgroup's teams
  if (EARLY && first + team < a.rows) fetch(first + team);
  for (; first < a.rows; first += step) {
    const long long row = first + team;
    const bool in = row < a.rows;
    float x[NCH][8], d[NCH][8];
    if (!EARLY && in) fetch(row);
    const float mu = mu_next, r = r_next;
    float s[2] = {0.f, 0.f};
    if (in) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        rx[k].get(x[k]);
        rd[k].get(d[k]);
      }
      if (EARLY && row + step < a.rows) fetch(row + step);
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // beyond the last column dy and w are zero, and x has no part
          const float xh = col[k] + i < a.cols ? (x[k][i] - mu) * r : 0.f;
          db[k][i] += d[k][i];
          dw[k][i] = fmaf(d[k][i], xh, dw[k][i]);
          const float g = d[k][i] * w[k][i];
          s[0] += g;
          s[1] = fmaf(g, xh, s[1]);
          x[k][i] = xh;
          d[k][i] = g;
        }
    }
    team_sum<TEAM>(s, sums[turn][team], tw, lane);
    turn ^= 1;
    const float c0 = s[0] / n, c1 = s[1] / n;
    if (in) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * (d[k][i] - c0 - x[k][i] * c1);
        store8_edge(static_cast<D*>(a.dx) + row * a.lddx + col[k], a.cols - col[k], o);
      }
    }
  }
  // the workgroup's sums: every team's go to LDS (element i of a chunk's lanes
  // side by side, the rows of 64 padded by one, so that neither the writes nor
  // the reads meet in a bank) and are added in the teams' order.  A single
  // workgroup's are the result, others are partial sums.
  const bool last = gridDim.x == 1;
  float* part = a.part + (long long)blockIdx.x * 2 * a.cols;
  auto put = [&](float* out, float* sums_of, int c, float s) __attribute__((always_inline)) {
    if (!last)
      sums_of[c] = s;
    else if (out)
      out[c] = a.accumulate ? out[c] + s : s;
  };
  if constexpr (TEAMS > 1) {
    constexpr int ROW = 65, PER = NCH * TEAM * 8 * ROW;
    __shared__ float acc[TEAMS * PER];
    auto join = [&](const float (&v)[NCH][8], float* out, float* sums_of)
                    __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < NCH; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[team * PER + ((k * TEAM + tw) * 8 + i) * ROW + lane] = v[k][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += 64 * WAVES) {
        const int at = ((c >> 9) * 8 + (c & 7)) * ROW + ((c >> 3) & 63);
        float s = acc[at];
#pragma unroll
        for (int t = 1; t < TEAMS; ++t) s += acc[t * PER + at];
        put(out, sums_of, c, s);
      }
      __syncthreads();
    };
    join(dw, a.dweight, part);
    join(db, a.dbias, part + a.cols);
  } else {
    auto store = [&](float (&v)[8], float* out, float* sums_of, int c)
                     __attribute__((always_inline)) {
      if (!last) {
        store8_edge(sums_of + c, a.cols - c, v);
      } else if (out) {
        float old[8];
        load8_edge(out + c, a.accumulate ? a.cols - c : 0, old);
        if (a.accumulate)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = old[i] + v[i];
        store8_edge(out + c, a.cols - c, v);
      }
    };
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      store(dw[k], a.dweight, part, col[k]);
      store(db[k], a.dbias, part + a.cols, col[k]);
    }
  }
}

// dw and db from the workgroups' partial sums, in their order: 32 columns per
// workgroup, 32 threads to a column, so that each thread's loads (8 of 256
// partial rows) are all on their way at once; joined in LDS.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* part, int groups, int cols,
                                                           float* dw, float* db, int accumulate) {
  __shared__ float acc[32][33];
  const int x = threadIdx.x & 31, g0 = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + x;
  float* out = blockIdx.y ? db : dw;
  const float* p = part + (blockIdx.y ? cols : 0) + c;
  float s = 0.f;
  if (c < cols)
#pragma unroll 8
    for (int g = g0; g < groups; g += 32) s += p[(long long)g * 2 * cols];
  acc[g0][x] = s;
  __syncthreads();
  if (g0 == 0 && c < cols) {
    s = 0.f;
#pragma unroll
    for (int g = 0; g < 32; ++g) s += acc[g][x];
    out[c] = accumulate ? out[c] + s : s;
  }
}

namespace {
// Team and chunks for a row of `cols` columns.  Forward: one wave up to 2048,
// four up to 8192, eight up to 16384; the fewest chunks that hold the row.
// Backward: up to 8192 columns at most three chunks to a lane, with a larger
// team where that takes one, since four fill the registers with their gradient
// sums: 16000 x 8192, eight waves of two chunks against four of four, 292 and 316
// us with dy and x in fp32, 238 and 264 (x bf16), 215 and 239 (x 8 bits), 190 and
// 204 (dy bf16, x fp32); with dy in bf16 and x in bf16 or 8 bits the eight cost
// more, 156 and 153, 139 and 129.  12289 to 16384 columns take four chunks on
// eight waves and spill 1 to 10 registers, 54 with dy and x in fp32 (16000 x
// 16384: 285 us all bf16, 602 all fp32).
template <bool BACK, typename F>
void with_shape(int cols, F&& f) {
#define MUON_SHAPE(T, N) f(std::integral_constant<int, T>{}, std::integral_constant<int, N>{})
  if (cols <= 512) MUON_SHAPE(1, 1);
  else if (cols <= 1024) MUON_SHAPE(1, 2);
  else if (cols <= 1536) MUON_SHAPE(1, 3);
  else if (cols <= 2048) MUON_SHAPE(BACK ? 2 : 1, BACK ? 2 : 4);
  else if (cols <= 4096) MUON_SHAPE(4, 2);
  else if (cols <= 6144) MUON_SHAPE(4, 3);
  else if (cols <= 8192) MUON_SHAPE(BACK ? 8 : 4, BACK ? 2 : 4);
  else if (cols <= 12288) MUON_SHAPE(8, 3);
  else MUON_SHAPE(8, 4);
#undef MUON_SHAPE
}
// Workgroups for `rows` rows, `teams` to a workgroup, at most `most`.
int groups_for(int rows, int teams, int most) {
  const long long g = ((long long)rows + teams - 1) / teams;
  return (int)(g < most ? g : most);
}
}  // namespace

// Workgroups of the backward pass, each with one partial sum: one per CU, which
// holds a CU's share of the registers and keeps the partial sums few.  Up to two
// rows to a team one workgroup does it all, without partial sums and a second
// launch.
int norm_backward_groups(int rows, int cols) {
  int g = 0;
  with_shape<true>(cols, [&](auto team, auto) {
    constexpr int T = decltype(team)::value;
    constexpr int teams = back_waves(T) / T;
    g = rows > 0 && rows <= 2 * teams ? 1 : groups_for(rows, teams, 256);
  });
  return g;
}

hipError_t launch_layer_norm(int x_bf16, int out, const NormArgs& a, hipStream_t s) {
  with_shape<false>(a.cols, [&](auto team, auto nch) {
    constexpr int T = decltype(team)::value, N = decltype(nch)::value;
    const dim3 grid(groups_for(a.rows, T > 4 ? 1 : 4 / T, T > 4 ? 512 : 2048)),
        block(T > 4 ? 64 * T : 256);
    if (x_bf16) {
      if (out == MUON_BF16)
        hipLaunchKernelGGL((layer_norm_kernel<MUON_BF16, MUON_BF16, T, N>), grid, block, 0, s, a);
      else if (out == MUON_FP32)
        hipLaunchKernelGGL((layer_norm_kernel<MUON_BF16, MUON_FP32, T, N>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((layer_norm_kernel<MUON_BF16, kOut8, T, N>), grid, block, 0, s, a);
    } else {
      if (out == MUON_BF16)
        hipLaunchKernelGGL((layer_norm_kernel<MUON_FP32, MUON_BF16, T, N>), grid, block, 0, s, a);
      else if (out == MUON_FP32)
        hipLaunchKernelGGL((layer_norm_kernel<MUON_FP32, MUON_FP32, T, N>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((layer_norm_kernel<MUON_FP32, kOut8, T, N>), grid, block, 0, s, a);
    }
  });
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(int dy_bf16, int x, const NormBackArgs& a, hipStream_t s) {
  if (a.groups > 0) with_shape<true>(a.cols, [&](auto team, auto nch) {
    constexpr int T = decltype(team)::value, N = decltype(nch)::value;
    const dim3 grid(a.groups), block(64 * back_waves(T));
    auto go = [&](auto dt) {
      constexpr int D = decltype(dt)::value;
      if (x == MUON_BF16)
        hipLaunchKernelGGL((layer_norm_back_kernel<D, MUON_BF16, T, N>), grid, block, 0, s, a);
      else if (x == MUON_FP32)
        hipLaunchKernelGGL((layer_norm_back_kernel<D, MUON_FP32, T, N>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((layer_norm_back_kernel<D, kOut8, T, N>), grid, block, 0, s, a);
    };
    if (dy_bf16)
      go(std::integral_constant<int, MUON_BF16>{});
    else
      go(std::integral_constant<int, MUON_FP32>{});
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.groups == 1) return err;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((a.cols + 31) / 32, a.dbias ? 2 : 1), dim3(1024), 0,
                     s, a.part, a.groups, a.cols, a.dweight, a.dbias, a.accumulate);
  return hipGetLastError();
}

}  // namespace muon
