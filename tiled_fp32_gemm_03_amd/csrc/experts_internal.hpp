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
  // Rows by adapter: pairs with no expert are expert E - 1's, which has no row tiles;
  // and rows of the product's tiles.
  int rest, run_tile;
};

// The order of the pairs by expert, in the workspace.
hipError_t launch_list(const ExpertsProblem &p, hipStream_t s);

hipError_t launch_experts_forward(const ExpertsProblem &p, hipStream_t s);
hipError_t launch_experts_backward(const ExpertsProblem &p, hipStream_t s);

// The products (one translation unit each).
hipError_t launch_experts_up(const ExpertsProblem &p, hipStream_t s);    // X, W1 -> u, saved
hipError_t launch_experts_down(const ExpertsProblem &p, hipStream_t s);  // u, W2 -> part
hipError_t launch_experts_du(const ExpertsProblem &p, hipStream_t s);    // dY, W2, saved -> dh, u, dg
hipError_t launch_experts_dx(const ExpertsProblem &p, hipStream_t s);    // dh, W1 -> part
hipError_t launch_experts_dw(const ExpertsProblem &p, hipStream_t s);    // dh, X -> dW1; dY, u -> dW2

// A shared projection with adapters (gemm_adapters.h).
struct AdaptersProblem {
  int T, N, K, R, count, format;
  const uint16_t *X;
  long long ldx;
  const uint16_t *W;
  long long ldw;
  const uint16_t *A;
  long long lda;
  const uint16_t *B;
  long long ldb;
  const int *ids;
  const float *scales;  // may be null
  uint16_t *Y;
  long long ldy;
  unsigned char *ws;
  AdaptersSpace at;
};
hipError_t launch_adapters_thin(const AdaptersProblem &p, hipStream_t s);   // adapters_thin
hipError_t launch_adapters_tiles(const AdaptersProblem &p, hipStream_t s);  // others

}  // namespace gemm_f32_impl
