// Host-only planning of routing, the experts' products and adapters: sizes,
// argument checks, workspaces and the choice of a kernel.  Plain C++17 with no
// HIP types, like host_plan.hpp; nothing here touches a GPU.
#pragma once

#include "mx_plan.hpp"

namespace gemm_f32_impl {

// ---- routing (gemm_route.h) ---------------------------------------------------

constexpr int kRouteMaxTokens = 1 << 22, kRouteMaxExperts = 512, kRouteMaxTop = 16,
              kRouteMaxGroups = 64;
constexpr int kSoftmax = 0, kSigmoid = 1;
constexpr int kGroupMax = 0, kGroupTop2 = 1;
int route_check_sizes(int T, int E, int top);

// ---- the experts' products (gemm_experts.h) -----------------------------------

constexpr int kExpertsMaxTokens = 1 << 22, kExpertsMaxWidth = 1 << 17;
int experts_check_sizes(int T, int E, int top, int H, int I);

// A pair is a token's choice, number token * top + choice.  The pairs whose
// expert is in 0 .. E - 1 are ordered by expert, then by number; a pair's
// number in that order is its place.
constexpr int kListPairs = 1024;  // pairs to a workgroup of the listing kernels
struct ExpertsSpace {
  long long start;   // int [E + 1]: expert e's places are start[e] .. start[e + 1] - 1
  long long tiles;   // int [4 + 4 most_tiles]: the number of row tiles, then from the fifth int on
                     // each one's expert, first place and rows, and 0
  long long list;    // int [T top]: the pair of each place
  long long token;   // int [T top]: its token
  long long where;   // int [T top]: the place of each pair, -1 where it has none
  long long counts;  // int [list workgroups][E]
  long long u;       // 16 bits [T top][ipitch], by place: inner values (backward: times their gate)
  long long part;    // float [T top][hpitch], by pair: what the pair adds to its token
  long long dh;      // 16 bits [T top][2 ipitch], by place: gradient of the first product
  long long dg;      // float [slices][T top], by place: parts of the gates' gradients
  // Of rows by adapter alone: the runs of one adapter (or none) that there are, as
  // `tiles` has the row tiles, and the number of the run in which each row tile of
  // the product begins.
  long long runs;
  long long tile_run;
  long long bytes;
  long long ipitch, hpitch, most_tiles, slices, list_groups;
};
// `tile`: rows and columns of a tile.
ExpertsSpace experts_space(int T, int E, int top, int H, int I, int tile, bool backward);
// Whether a forward pass without `saved` runs on the thin products of the
// mixture-of-experts layer.
bool experts_thin(int T, int E, int top);
// The tile of a call's products, 256 or 128; a call that `trains` counts the backward
// pass's too.
int experts_tile(int T, int E, int top, int H, int I, bool trains);

// ---- adapters (gemm_adapters.h) -----------------------------------------------

constexpr int kAdaptersMaxRows = 1 << 22, kAdaptersMaxWidth = 1 << 17, kAdaptersMaxRank = 512,
              kAdaptersMaxCount = 511;
// Rows that the thin products take at a time, and the rows of a tile of the products
// with A.
constexpr int kAdaptersThin = 64, kAdaptersMostThin = 512, kAdaptersRows = 64;
bool adapters_thin(int T, int N, int K);
int adapters_check_sizes(int T, int N, int K, int R, int count);

// Rows by adapter: as pairs by expert (ExpertsSpace), with the rows without one as
// the last of count + 1.
struct AdaptersSpace {
  ExpertsSpace order;  // u, part, dh and dg: none
  long long part;      // float [splits][T][rpitch], by place: A x in parts of K
  long long v;         // float (bf16: 16 bits) [T][rpitch], by place (thin: by row): scale A x
  long long bytes;
  long long rpitch;
  int tile;            // rows and columns of the product's tiles
  int splits, chunk;   // parts of K in the products with A, of `chunk` values each
  // The same of the projection, where its tiles are few: then their sums.
  int wide_splits, wide_chunk;
  long long wide_part;  // float [wide_splits][T][npitch], by place
  long long npitch;
};
AdaptersSpace adapters_space(int T, int N, int K, int R, int count);

}  // namespace gemm_f32_impl
