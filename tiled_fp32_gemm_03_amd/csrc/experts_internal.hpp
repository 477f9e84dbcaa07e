// Internal declarations of the experts' products: what the C-ABI front end
// (rows_abi.hip) hands to the kernels' translation units, and what those share.
#pragma once

#include <hip/hip_runtime.h>

#include "experts_plan.hpp"

namespace gemm_f32_impl {

struct ExpertsProblem {
  int T, E, top, H, I;
  int tile, format;
  const uint16_t *X;
  long long ldx;
  const int *ids;
  const float *gates;
  const uint16_t *W1;  // pitches in elements
  long long ld1;
  const uint16_t *W2;
  long long ld2;
  float *saved;  // [T top][2 I], by place; may be null in the forward pass
  uint16_t *Y;
  long long ldy;
  // the backward pass
  const uint16_t *dY;
  long long lddy;
  uint16_t *dX;
  long long lddx;
  float *dgates;
  uint16_t *dW1;
  long long lddw1;
  uint16_t *dW2;
  long long lddw2;
  unsigned char *ws;
  ExpertsSpace at;
};

hipError_t launch_experts_forward(const ExpertsProblem &p, hipStream_t s);
hipError_t launch_experts_backward(const ExpertsProblem &p, hipStream_t s);

// The products (one translation unit each).
hipError_t launch_experts_up(const ExpertsProblem &p, hipStream_t s);    // X, W1 -> u, saved
hipError_t launch_experts_down(const ExpertsProblem &p, hipStream_t s);  // u, W2 -> part
hipError_t launch_experts_du(const ExpertsProblem &p, hipStream_t s);    // dY, W2, saved -> dh, u, dg
hipError_t launch_experts_dx(const ExpertsProblem &p, hipStream_t s);    // dh, W1 -> part
hipError_t launch_experts_dw(const ExpertsProblem &p, hipStream_t s);    // dh, X -> dW1; dY, u -> dW2

}  // namespace gemm_f32_impl
