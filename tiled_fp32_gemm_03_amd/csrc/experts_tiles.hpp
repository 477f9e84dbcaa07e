// What the experts' products share (row_tiles.hpp has the products): the list of
// row tiles, and the choice of a kernel.
#pragma once

#include "experts_internal.hpp"
#include "row_tiles.hpp"

namespace gemm_f32_impl {
namespace {

template <class T>
__device__ inline T *ws_at(const ExpertsProblem &p, long long off) {
  return reinterpret_cast<T *>(p.ws + off);
}

// Rows of one expert: n of them from place `first` on.
struct Rows {
  int e, first, n;
};
__device__ inline Rows row_tile(const ExpertsProblem &p, int tm) {
  const int *t = ws_at<int>(p, p.at.tiles) + 4 + 4LL * tm;
  return {__builtin_amdgcn_readfirstlane(t[0]), __builtin_amdgcn_readfirstlane(t[1]),
          __builtin_amdgcn_readfirstlane(t[2])};
}

// A workgroup's share of the tiles: t of `count`, those of one round next to one another
// and each XCD's too.
struct Share {
  int first, step, count;
  __device__ explicit Share(int total) {
    const int G = gridDim.x;
    first = xcd_remap(blockIdx.x, G);
    step = G;
    count = __builtin_amdgcn_readfirstlane(first < total ? (total - first + G - 1) / G : 0);
  }
  __device__ int tile(int t) const { return first + t * step; }
};

// A product of one expert's rows: tile (tm, tn) of row tiles and columns.
struct RowJob {
  int steps, rows;
  int e, first, tn;
};
__device__ inline int row_tiles(const ExpertsProblem &p) {
  return __builtin_amdgcn_readfirstlane(*ws_at<int>(p, p.at.tiles));
}
__device__ inline RowJob row_job(const ExpertsProblem &p, int tile, int rows, int columns, int steps) {
  int tm, tn;
  tile_coords(tile, rows, columns, tm, tn);
  // (divisions: the compiler forms them in vector registers)
  const Rows r = row_tile(p, __builtin_amdgcn_readfirstlane(tm));
  return {steps, r.n, r.e, r.first, __builtin_amdgcn_readfirstlane(tn)};
}

// The tokens of a side's rows, on their way: one to each of a lane's loads.
template <class Side>
struct TokenRows {
  int at[Side::kLoads];
  __device__ __forceinline__ void fetch(const int *token, int n, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < Side::kLoads; ++q) {
      const int r = Side::row_of(q, wave, lane);
      at[q] = token[r < n ? r : n - 1];
    }
  }
};

// Whether a matrix's rows can be loaded directly: 16-byte aligned, of whole 16
// bytes, and `rows` of them within 32-bit offsets.  (One row inside that border and one past
// it, ms: 4,096 values, 262,143 and 262,144 tokens on 8 experts of 1,024 7.5 and 10.8, with
// the gradients 21.9 and 34.5; rows with adapters, 4096 x 4096, 7.6 and 13.7.)
inline bool direct(const void *p, long long ld, long long width, long long rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && width % 8 == 0 &&
         2 * rows * ld <= kMostRecords;
}
// Whether they can be read by the words around their values.
inline bool by_words(const void *p, long long width) {
  return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && width >= 8;
}

// The products of a pass whose row tiles are the list's.
inline bool up_direct(const ExpertsProblem &p) {
  return direct(p.X, p.ldx, p.H, p.T) && direct(p.W1, p.ld1, p.H, 2LL * p.I);
}
inline bool down_direct(const ExpertsProblem &p) { return direct(p.W2, p.ld2, p.I, p.H); }
inline bool du_direct(const ExpertsProblem &p) {
  return direct(p.dY, p.lddy, p.H, p.T) && direct(p.W2, p.ld2, p.I, kStepK);
}
inline bool dx_direct(const ExpertsProblem &p) { return direct(p.W1, p.ld1, p.H, kStepK); }

// KERN on at most `tiles` tiles: as many workgroups as the chip holds at once.
template <auto KERN, int THREADS, class P>
hipError_t launch_tiles(const P &p, long long tiles, hipStream_t s) {
  if (tiles <= 0) return hipSuccess;
  const long long most = resident_workgroups<KERN, THREADS>();
  return launch_kernel(KERN, dim3((unsigned)(tiles < most ? tiles : most)), dim3(THREADS),
                       s, p);
}
// KERN<T, format, S, ...> in the call's format.
#define GEMM_F32_LAUNCH_ROWS(KERN, T, S, ...)                                         \
  (p.format == kBf16 ? launch_tiles<KERN<T, kBf16, S>, T::THREADS>(p, __VA_ARGS__, s)               \
                     : launch_tiles<KERN<T, kF16, S>, T::THREADS>(p, __VA_ARGS__, s))

// Two waves to a SIMD: eight of one workgroup, or four of each of two.
typedef RowTile<64, 128, 4, 2> Large;
typedef RowTile<64, 64, 2, 2> Small;
// One, where tiles are too few for two to a compute unit.
typedef RowTile<64, 64, 2, 2, 4> Deep;
static_assert(Large::WGN == 2 && Small::WGN == 2 && Deep::WGN == 2, "slices of ExpertsSpace");
template <class T>
constexpr int kWavesPerSimd = T::STAGES > 2 ? 1 : 2;

// As many tiles of 128 x 128 as there are compute units.
constexpr long long kFewTiles = 256;
// The row tiles that a call's pairs fill where they are spread evenly.
inline long long even_tiles(const ExpertsProblem &p) {
  const long long pairs = (long long)p.T * p.top, asked = p.E < pairs ? p.E : pairs;
  if (asked == 0) return 0;
  return asked * (pairs / (asked * p.tile)) + ceil_div(asked, 2);
}

// `make(tile, integral_constant S)` launches, about `tiles` tiles.  Large tiles are loaded directly
// alone (through registers a wave of 128 x 128 has none left for its loads): a call
// whose row tiles are a list's asks for them only where all its products are.
template <class Make>
hipError_t choose_tiles(int tile, long long tiles, bool direct_loads, bool words, Make make) {
  if (direct_loads) {
    if (tile == Large::BM) return make(Large{}, std::integral_constant<int, kDirect>{});
    if (tiles <= kFewTiles) return make(Deep{}, std::integral_constant<int, kDirect>{});
    return make(Small{}, std::integral_constant<int, kDirect>{});
  }
  if (tile != Small::BM) return hipErrorInvalidValue;
  if (words) return make(Small{}, std::integral_constant<int, kByWords>{});
  return make(Small{}, std::integral_constant<int, kAnyRows>{});
}

}  // namespace
}  // namespace gemm_f32_impl
