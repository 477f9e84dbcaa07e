// Internal declarations of the routing kernels: what the C-ABI front end
// (rows_abi.hip) hands to route.hip.
#pragma once

#include <hip/hip_runtime.h>

#include "experts_plan.hpp"

namespace gemm_f32_impl {

struct RouteProblem {
  int T, E, top;
  const void *Z;
  long long ldz;
  int format, score;
  const float *bias;  // may be null
  int groups, top_groups, group_score, renormalize;
  double scale;
  int *ids;
  float *gates;
  // the backward pass
  const int *given;
  const float *dgates;
  void *dZ;
  long long lddz;
};
hipError_t launch_route(const RouteProblem &p, hipStream_t s);
hipError_t launch_route_backward(const RouteProblem &p, hipStream_t s);

}  // namespace gemm_f32_impl
