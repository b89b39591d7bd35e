// The norm of many tensors together, and their clipping to it:
//   norm = sqrt(sum over all tensors of g^2),
//   g <- c g,  c = max_norm / (norm + eps) where that is below 1, else 1.
// Squares and sums are fp64: a square of any fp32 number is one there, so
// nothing overflows or vanishes on the way, and the vector unit has the time
// (memory brings 2.6e12 bf16 values a second, and it adds 39e12).
//
// Tensors are cut into tiles; a workgroup takes a run of neighbouring tiles,
// finds its first one's tensor by bisection and goes on from there, so that many
// small tensors and a few large ones share a launch evenly.  Each workgroup
// leaves one sum, and the finishing launch adds those in their order.  Up to as many as
// one launch can have, 2048, each workgroup of a clipping launch adds them itself, which
// saves that launch (129 tensors of 100003 numbers, not clipped: 22.0 us, 23.4 with it);
// more would be a work that grows with the square of the tensors, and the clipping ones
// take the finishing one's sum (4000 of 2^18: 805 us, 2670 without; 300 of them 62, 69).
// The clipping pass goes over its run backwards: what the norm read last is what the
// last-level cache still holds, and its results are stored past that.
//   805e6 numbers, fp32: norm 540 us (6.0 TB/s; a copy runs at 5.2), clipped into
//   bf16 1482 us (5.4 TB/s over two readings and the writing); bf16: norm 273 us
//   (5.9), clipped 939 us (5.1).  With half the workgroups and cached stores 600,
//   1573, 275 and 950 us.
#include "layers/fp8_device.h"
#include "muon_clip.h"

namespace muon {

constexpr int kClipThreads = 512, kClipItems = kClipTile / (8 * kClipThreads);
static_assert(sizeof(ClipLaunch) <= 4096, "kernel arguments");

// Sum over the workgroup, the same in all threads.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* buf) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) v += buf[w];
  return v;
}

// The workgroup's run of tiles, and the tensor of a tile.
struct Run {
  const __attribute__((address_space(4))) ClipTable& t;
  unsigned begin, end;
  int i;
  __device__ __forceinline__ Run(const __attribute__((address_space(4))) ClipLaunch& a,
                                 bool backwards)
      : t(a.t) {
    const unsigned long long all = t.first[a.tensors];
    begin = (unsigned)(all * blockIdx.x / gridDim.x);
    end = (unsigned)(all * (blockIdx.x + 1) / gridDim.x);
    const unsigned at = backwards ? end - 1 : begin;
    int lo = 0, hi = a.tensors;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (t.first[mid] <= at) lo = mid; else hi = mid;
    }
    i = lo;
  }
  // element of the tensor that tile `at` begins with
  __device__ __forceinline__ long long seek(unsigned at) {
    while (at >= t.first[i + 1]) ++i;
    while (at < t.first[i]) --i;
    return (long long)(at - t.first[i]) * kClipTile;
  }
};

__device__ __forceinline__ int left_of(long long n) { return n > 8 ? 8 : (int)n; }

template <typename T>
__device__ __forceinline__ void load_tile(const T* p, long long left, Raw8<T> (&raw)[kClipItems]) {
#pragma unroll
  for (int k = 0; k < kClipItems; ++k) {
    const int e = (k * kClipThreads + (int)threadIdx.x) * 8;
    raw[k].load(p + e, left_of(left - e));
  }
}

__global__ __launch_bounds__(kClipThreads) void norm_parts_kernel(ClipLaunch) {
  const auto& a = kernarg<ClipLaunch>();
  __shared__ double buf[kClipThreads / 64];
  Run run(a, false);
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  auto add = [&](auto* p, long long left) __attribute__((always_inline)) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    Raw8<T> raw[kClipItems];
    load_tile(p, left, raw);
#pragma unroll
    for (int k = 0; k < kClipItems; ++k) {
      float v[8];
      raw[k].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j & 3] = fma((double)v[j], (double)v[j], acc[j & 3]);
    }
  };
  for (unsigned at = run.begin; at < run.end; ++at) {
    const long long e = run.seek(at);
    const unsigned long long size = run.t.size[run.i];
    const long long left = (long long)(size >> 2) - e;
    if (size & 1)
      add(static_cast<const float*>(run.t.in[run.i]) + e, left);
    else
      add(static_cast<const bf16_t*>(run.t.in[run.i]) + e, left);
  }
  const double s = block_sum<kClipThreads / 64>((acc[0] + acc[1]) + (acc[2] + acc[3]), buf);
  if (threadIdx.x == 0) a.part[blockIdx.x] = s;
}

// All launches' sums, each thread every 512th, so the order is always the same.
__device__ __forceinline__ double sum_parts(const double* part, int parts, double* buf) {
  double s = 0.0;
#pragma unroll 8
  for (int j = threadIdx.x; j < parts; j += kClipThreads) s += part[j];
  return block_sum<kClipThreads / 64>(s, buf);
}

// keep: the sum takes the first part's place, which block_sum's barrier leaves free.
__global__ __launch_bounds__(kClipThreads) void norm_finish_kernel(double* part, int parts,
                                                                   float* norm, bool keep) {
  __shared__ double buf[kClipThreads / 64];
  const double s = sum_parts(part, parts, buf);
  if (threadIdx.x == 0) {
    *norm = (float)sqrt(s);
    if (keep) *part = s;
  }
}

__global__ __launch_bounds__(kClipThreads) void clip_kernel(ClipLaunch) {
  const auto& a = kernarg<ClipLaunch>();
  __shared__ double buf[kClipThreads / 64];
  const double norm = sqrt(sum_parts(a.part, a.parts, buf));
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  // (0 / 0, for gradients of zeros without an eps, is not below 1: they stay)
  const double over = norm + (double)a.eps, q = over == 0.0 ? 1.0 : (double)a.max_norm / over;
  // A NaN stays one.  A c below fp32's normal numbers would have lost digits:
  // it is applied as two factors, the second a power of two.
  const bool tiny = q < 0x1p-126;
  const float c = q >= 1.0 ? 1.f : (float)(tiny ? q * 0x1p64 : q), c2 = tiny ? 0x1p-64f : 1.f;
  Run run(a, true);
  auto scale = [&](auto* p, auto* o, long long left) __attribute__((always_inline)) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    Raw8<T> raw[kClipItems];
    load_tile(p, left, raw);
#pragma unroll
    for (int k = 0; k < kClipItems; ++k) {
      const int e = (k * kClipThreads + (int)threadIdx.x) * 8;
      float v[8];
      raw[k].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * c * c2;
      store8_edge<true>(o + e, left_of(left - e), v);  // (not read here again)
    }
  };
  for (unsigned at = run.end; at-- > run.begin;) {
    const long long e = run.seek(at);
    const unsigned long long size = run.t.size[run.i];
    const long long left = (long long)(size >> 2) - e;
    const void* in = run.t.in[run.i];
    void* out = run.t.out[run.i];
    if (in == out && c == 1.f) continue;  // nothing to do in place
    const float* pf = static_cast<const float*>(in) + e;
    const bf16_t* pb = static_cast<const bf16_t*>(in) + e;
    float* of = static_cast<float*>(out) + e;
    bf16_t* ob = static_cast<bf16_t*>(out) + e;
    switch ((int)(size & 3)) {
      case 0: scale(pb, ob, left); break;
      case 1: scale(pf, ob, left); break;
      case 2: scale(pb, of, left); break;
      default: scale(pf, of, left);
    }
  }
}

hipError_t launch_norm_parts(const ClipLaunch& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_parts_kernel, dim3(a.groups), dim3(kClipThreads), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_norm_finish(double* part, int parts, float* norm, bool keep, hipStream_t s) {
  hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(kClipThreads), 0, s, part, parts, norm, keep);
  return hipGetLastError();
}
hipError_t launch_clip(const ClipLaunch& a, hipStream_t s) {
  hipLaunchKernelGGL(clip_kernel, dim3(a.groups), dim3(kClipThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
