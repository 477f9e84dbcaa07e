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

// Calls run(tm, tn) for each of this workgroup's tiles of rows x columns.
template <class Run>
__device__ __forceinline__ void each_row_tile(const ExpertsProblem &p, int columns, Run run) {
  const int rows = __builtin_amdgcn_readfirstlane(*ws_at<int>(p, p.at.tiles));
  const int total = rows * columns;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    int tm, tn;
    tile_coords(xcd_remap(t, total), rows, columns, tm, tn);
    // (divisions: the compiler forms them in vector registers)
    run(__builtin_amdgcn_readfirstlane(tm), __builtin_amdgcn_readfirstlane(tn));
    if (t + (int)gridDim.x < total) ks_lds_barrier();  // the next tile's loads overwrite the LDS
  }
}

// Whether a matrix's rows can be loaded directly: 16-byte aligned, of whole 16
// bytes, and `rows` of them within 32-bit offsets.
inline bool direct(const void *p, long long ld, long long width, long long rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && width % 8 == 0 &&
         2 * rows * ld <= kMostRecords;
}
// Whether they can be read by the words around their values.
inline bool by_words(const void *p, long long width) {
  return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && width >= 8;
}

constexpr int kMostGroups = 1 << 20;
template <class Kernel>
hipError_t launch_tiles(Kernel kern, const ExpertsProblem &p, long long tiles, hipStream_t s) {
  if (tiles <= 0) return hipSuccess;
  const unsigned grid = (unsigned)(tiles < kMostGroups ? tiles : kMostGroups);
  return launch_kernel(kern, dim3(grid), dim3(256), s, p);
}

typedef RowTile<128, 128> Large;
typedef RowTile<64, 64> Small;
template <class T>
constexpr int kPerSimd = T::STAGE > 40 * 1024 ? 1 : 2;  // workgroups to a CU

// `make(tile, integral_constant S)` launches.  Large tiles are loaded directly
// alone (through registers a wave of 128 x 128 has none left for its loads).
template <class Make>
hipError_t choose_tiles(const ExpertsProblem &p, bool direct_loads, bool words, Make make) {
  if (direct_loads) {
    if (p.tile == Large::BM) return make(Large{}, std::integral_constant<int, kDirect>{});
    return make(Small{}, std::integral_constant<int, kDirect>{});
  }
  if (words) return make(Small{}, std::integral_constant<int, kByWords>{});
  return make(Small{}, std::integral_constant<int, kAnyRows>{});
}

}  // namespace
}  // namespace gemm_f32_impl
