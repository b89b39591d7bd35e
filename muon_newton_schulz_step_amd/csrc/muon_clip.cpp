// Host side of the gradients' norm and their clipping: argument checks,
// workspace size, the tensors' distribution over launches.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "layers/muon_checks.h"
#include "muon.h"
#include "muon_clip.h"

using namespace muon;

namespace {

// Tiles of a launch are counted in 32 bits, those of its 128 tensors together.
constexpr long long kMaxSize = 1LL << 38;

long long tiles_of(long long size) { return (size + kClipTile - 1) / kClipTile; }
int groups_of(long long tiles) { return (int)std::min<long long>(tiles, kClipGroups); }

// Calls f(first tensor, one past the last, tiles) for each launch; empty tensors have no
// tiles and take no place.
template <typename F>
void each_launch(int n, const long long* sizes, F&& f) {
  for (int i = 0; i < n;) {
    const int from = i;
    long long tiles = 0;
    for (int places = 0; i < n && places < kClipTensors; ++i)
      if (sizes[i] > 0) {
        ++places;
        tiles += tiles_of(sizes[i]);
      }
    if (tiles > 0) f(from, i, tiles);
  }
}

int parts_of(int n, const long long* sizes) {
  int parts = 0;
  each_launch(n, sizes, [&](int, int, long long tiles) { parts += groups_of(tiles); });
  return parts;
}

bool sizes_ok(int n, const long long* sizes) {
  if (n < 0 || n > (1 << 20) || (n > 0 && !sizes)) return false;
  for (int i = 0; i < n; ++i)
    if (sizes[i] < 0 || sizes[i] > kMaxSize) return false;
  return true;
}

struct Mark {
  uintptr_t begin, end;
  bool written;
};
// A written range meets another range.
bool any_conflict(std::vector<Mark>& marks) {
  std::sort(marks.begin(), marks.end(),
            [](const Mark& a, const Mark& b) { return a.begin < b.begin; });
  uintptr_t end_any = 0, end_written = 0;
  for (const Mark& m : marks) {
    if (m.begin < (m.written ? end_any : end_written)) return true;
    end_any = std::max(end_any, m.end);
    if (m.written) end_written = std::max(end_written, m.end);
  }
  return false;
}

int clip_impl(int n, const long long* sizes, const void* const* grads, const int* dtypes,
              void* const* out, const int* out_dtypes, bool clip, float max_norm, float eps,
              float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!sizes_ok(n, sizes) || !norm || !aligned(norm, 4)) return MUON_ERR_INVALID_ARG;
  if (n > 0 && (!grads || !dtypes || (out && !out_dtypes))) return MUON_ERR_INVALID_ARG;
  if (clip && (!std::isfinite(max_norm) || max_norm < 0.f || !std::isfinite(eps) || eps < 0.f))
    return MUON_ERR_INVALID_ARG;
  const int parts = parts_of(n, sizes);
  const size_t need = (size_t)parts * sizeof(double);
  std::vector<Mark> marks;
  marks.reserve(2 * (size_t)n + 2);
  auto mark = [&](const void* p, size_t bytes, bool written) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    if (bytes) marks.push_back({b, b + bytes, written});
  };
  double bytes = 0.0;
  for (int i = 0; i < n; ++i) {
    if (!is_dtype(dtypes[i]) || (clip && out && !is_dtype(out_dtypes[i])))
      return MUON_ERR_INVALID_ARG;
    if (sizes[i] == 0) continue;
    const size_t es = size_of(dtypes[i]);
    if (!grads[i] || !aligned(grads[i], es)) return MUON_ERR_INVALID_ARG;
    bytes += (double)sizes[i] * es;
    const bool in_place = clip && (!out || (out[i] == grads[i] && out_dtypes[i] == dtypes[i]));
    mark(grads[i], (size_t)sizes[i] * es, in_place);
    if (clip && !in_place) {
      const size_t eo = size_of(out_dtypes[i]);
      if (!out[i] || !aligned(out[i], eo)) return MUON_ERR_INVALID_ARG;
      mark(out[i], (size_t)sizes[i] * eo, true);
    }
  }
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, MUON_WORKSPACE_ALIGN)))
    return MUON_ERR_WORKSPACE;
  mark(norm, sizeof(float), true);
  mark(workspace, need, true);
  if (any_conflict(marks)) return MUON_ERR_INVALID_ARG;
  if (int st = check_stream_device(stream)) return st;

  ClipLaunch a{};
  auto fill = [&](int from, int to, long long tiles) {
    a.tensors = 0;
    unsigned first = 0;
    for (int i = from; i < to; ++i) {
      if (sizes[i] == 0) continue;
      const int k = a.tensors++;
      const int od = clip ? (out ? out_dtypes[i] : dtypes[i]) : MUON_BF16;
      a.t.in[k] = grads[i];
      a.t.out[k] = clip ? (out ? out[i] : const_cast<void*>(grads[i])) : nullptr;
      a.t.size[k] = (unsigned long long)sizes[i] * 4 + (dtypes[i] == MUON_FP32 ? 1 : 0) +
                    (od == MUON_FP32 ? 2 : 0);
      a.t.first[k] = first;
      first += (unsigned)tiles_of(sizes[i]);
    }
    a.t.first[a.tensors] = first;
    a.groups = groups_of(tiles);
  };
  double* part = static_cast<double*>(workspace);
  return status_of(timed_launch(MUON_K_GRAD_NORM, n, 1, 0.0, 0.0, bytes, stream, [&] {
    hipError_t err = hipSuccess;
    int done = 0;
    each_launch(n, sizes, [&](int from, int to, long long tiles) {
      fill(from, to, tiles);
      a.part = part + done;
      done += a.groups;
      if (err == hipSuccess) err = launch_norm_parts(a, stream);
    });
    if (err != hipSuccess) return err;
    // no more sums than one launch can have: clipping's workgroups add them
    const bool few = clip && parts > 0 && parts <= kClipGroups;
    if (!few) err = launch_norm_finish(part, parts, norm, clip && parts > 0, stream);
    if (err != hipSuccess || !clip) return err;
    a.part = part;
    a.parts = few ? parts : 1;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = few ? norm : nullptr;
    each_launch(n, sizes, [&](int from, int to, long long tiles) {
      fill(from, to, tiles);
      if (err == hipSuccess) err = launch_clip(a, stream);
      a.norm = nullptr;
    });
    return err;
  }));
}

// The host's own memory can run out in the tables above.
template <typename F>
int guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

}  // namespace

extern "C" {

size_t muon_grad_norm_workspace_bytes(int n, const long long* sizes) {
  return sizes_ok(n, sizes) ? (size_t)parts_of(n, sizes) * sizeof(double) : 0;
}

int muon_grad_norm(int n, const long long* sizes, const void* const* grads, const int* dtypes,
                   float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return guarded([&] {
    return clip_impl(n, sizes, grads, dtypes, nullptr, nullptr, false, 0.f, 0.f, norm, workspace,
                     workspace_bytes, stream);
  });
}

int muon_clip_grads(int n, const long long* sizes, const void* const* grads, const int* dtypes,
                    void* const* out, const int* out_dtypes, float max_norm, float eps,
                    float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return guarded([&] {
    return clip_impl(n, sizes, grads, dtypes, out, out_dtypes, true, max_norm, eps, norm,
                     workspace, workspace_bytes, stream);
  });
}

}  // extern "C"
