// fa_norm.h -- launch interface of the norm-and-rotate kernels.
#pragma once

#include <algorithm>

#include "fa_serve.h"

namespace fa {

// Blocks of the backward kernel per SM: as many as its registers allow at once, so that
// all run from beginning to end.  Each leaves one row of D sums of the weights' gradient
// in the workspace.
constexpr int kNormBlocks = 3;

struct NormLaunch {
  RotaryLaunch rot;       // forward: x -> y; backward: x, dx, and inverse
  const void* weight[2];  // [D], or null: ones
  int weight_elem;        // rot.elem or fp32
  float eps;
  // backward
  const void* dy[2];
  RowStrides dys[2];
  void* dweight[2];  // of weight_elem; null: not wanted
  float* partial;    // [kNormBlocks * SMs][D]
  // of queries and of keys, set at launch: blocks, items of a token, heads of a lane group
  int blocks[2], groups[2], per[2];
};

cudaError_t launch_norm_rotary(const NormLaunch& a, bool backward, cudaStream_t s);

}  // namespace fa
