// Host-side interface of the router (route.hip), for rows_abi.hip.
#pragma once

#include "w4a8_internal.h"

namespace w4a8 {

constexpr int kMaxTopK = 64;    // a lane per chosen expert
constexpr int kMaxGroups = 64;  // a lane per group

struct RouteArgs {
  const void* logits;
  int dtype;  // W4A8_BF16 / W4A8_F32
  const float* bias;
  int64_t M;
  int E, k;
  bool softmax, renormalize;
  int n_groups, topk_groups, group_top;
  float scale;
  int* ids;
  float* weights;
  int gl = 0;  // log2 lanes per group (set by the launcher)
};

hipError_t launch_route(const RouteArgs& a, hipStream_t st);

}  // namespace w4a8
