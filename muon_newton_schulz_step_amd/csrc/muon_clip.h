// Internal interface between the host side of the gradients' norm and their
// clipping (muon_clip.cpp) and its kernels (grad_norm.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include "muon.h"

namespace muon {

// Tensors of one launch: their table is a kernel argument, of which there are
// 4 KB.
constexpr int kClipTensors = 128;
// Elements of a tile, the unit of work: a tensor is a whole number of them, the
// last one ragged.
constexpr int kClipTile = 16384;
// Workgroups of a launch at most, each with one partial sum.
constexpr int kClipGroups = 2048;

struct ClipTable {
  const void* in[kClipTensors];
  void* out[kClipTensors];
  // elements * 4, plus 1 where the input is fp32 and 2 where the output is
  unsigned long long size[kClipTensors];
  unsigned first[kClipTensors + 1];  // tiles in front of the tensor
};
struct ClipLaunch {
  ClipTable t;
  int tensors, groups;
  double* part;      // norm: this launch's sums; clip: all launches', or their sum
  int parts;         // clip: how many
  float max_norm, eps;
  float* norm;       // written by the finishing launch, or by clip's first one
};

hipError_t launch_norm_parts(const ClipLaunch& a, hipStream_t s);
// keep: part[0] becomes the sum of all parts
hipError_t launch_norm_finish(double* part, int parts, float* norm, bool keep, hipStream_t s);
hipError_t launch_clip(const ClipLaunch& a, hipStream_t s);

}  // namespace muon
