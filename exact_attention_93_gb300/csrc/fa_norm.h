// fa_norm.h -- launch interface of the norm-and-rotate kernels.
#pragma once

#include <algorithm>

#include "fa_serve.h"

namespace fa {

// Blocks of the backward kernel per SM, at most; each leaves one row of D sums of the
// weights' gradient in the workspace.
constexpr int kNormBlocks = 8;

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
  int blocks[2];     // of queries, of keys (set at launch)
};

cudaError_t launch_norm_rotary(const NormLaunch& a, bool backward, cudaStream_t s);

}  // namespace fa
