// Arguments of the mixture-of-experts kernels and the layout of their workspace.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/biloco.h"

namespace biloco {

constexpr int kMoeMaxTokens = BILOCO_MOE_MAX_T;
constexpr int kMoeMaxExperts = BILOCO_MOE_MAX_E;
constexpr int kMoeMaxTopK = BILOCO_MOE_MAX_K;
constexpr int kMoeMaxShared = BILOCO_MOE_MAX_SHARED;
constexpr int kMoeMaxPairs = kMoeMaxTokens * (kMoeMaxTopK + kMoeMaxShared);

struct MoeArgs {
  const uint16_t* x;       // [T][D] bf16, row stride ldx
  const void* router;      // [E][D] bf16 or FP32
  const float* bias;       // [E] or null
  const uint8_t* w13;      // [E + shared][2F][D]
  const float* s13;
  const uint8_t* w2;       // [E + shared][D][F]
  const float* s2;
  uint16_t* y;             // [T][D] bf16
  int* ids;                // [T][k]
  float* weights;          // [T][k]
  // workspace
  int* pair_id;            // [T][k + shared] expert of each (token, choice) pair
  float* pair_w;           // its weight
  uint32_t* hmax;          // bits of the largest |h| of a pair's hidden row
  int* hexp;               // [pairs][F/8] exponent that 8 columns of h are stored relative to
  uint16_t* xh;            // [T][D] FP16 token rows, scaled
  float* xscale;           // [T] what to multiply them by
  uint16_t* h;             // [pairs][F] FP16
  float* share;            // [pairs][D] what a pair adds to y
  long long ldx;
  int T, D, F, E, k, shared;
  bool sigmoid, renorm, router_f32;
  float route_scale;
};

// Places the workspace's arrays behind `base` (256-byte aligned); returns its size.
size_t moe_carve(MoeArgs& a, uint8_t* base);
cudaError_t launch_fp8_moe(MoeArgs& a, cudaStream_t s);

}  // namespace biloco
