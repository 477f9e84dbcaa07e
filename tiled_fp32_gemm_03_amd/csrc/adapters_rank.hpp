// scale A x on its way into the product with B (gemm_adapters.h), shared by the thin
// products and the tiles.
#pragma once

#include "mx_thin.hpp"

namespace gemm_f32_impl {
namespace {

// How it is kept: rounded to bf16 at once; for fp16, whose range is no more than 2^40, in
// fp32 up to the product.  Four values at `at`.
template <int FMT>
struct Kept {
  typedef uint16_t type;
  static __device__ __forceinline__ void store(uint16_t *at, f32x4 v) {
    *reinterpret_cast<u32x2 *>(at) = u32x2{pack2<FMT>(v[0], v[1]), pack2<FMT>(v[2], v[3])};
  }
};
template <>
struct Kept<kF16> {
  typedef float type;
  static __device__ __forceinline__ void store(float *at, f32x4 v) {
    *reinterpret_cast<f32x4 *>(at) = v;
  }
};

// Eight ranks of each of N groups of 32, for lane l those of row l % 16 from 8 (l / 16)
// on: a matrix instruction's operand; `back` is for its product with B.  `from`: the
// lane's values of the first group; `have` groups are there.
template <int FMT, int N>
struct LowRank {
  u32x4 v[N];
  __device__ __forceinline__ LowRank(const uint16_t *from, int have) {
#pragma unroll
    for (int h = 0; h < N; ++h)
      v[h] = h < have ? *reinterpret_cast<const u32x4 *>(from + 32 * h) : u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ float back(float sum) const { return sum; }
};
// The larger of a lane's value and that of the lane which `swap` pairs it with.
template <class Swap>
__device__ __forceinline__ float larger(float v, Swap swap) {
  const uint32_t own = __builtin_bit_cast(uint32_t, v);
  const auto both = swap(own, own);
  // (__builtin_bit_cast of a vector's element takes the first one's bits)
  const uint32_t a = both[0], b = both[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
// A row's groups are multiplied by the power of two that brings their largest value to
// 2^14 .. 2^15, and the product is divided by it: what is lost is each value's half
// step, or 2^-28 of the largest where that is more.  All lanes take part.  (In 16
// bits without an exponent, and so, us: 61 rows, odd sizes, 30 adapters of rank 17 29.6
// and 30.8.)
template <int N>
struct LowRank<kF16, N> {
  u32x4 v[N];
  int up;
  __device__ __forceinline__ LowRank(const float *from, int have) {
    f32x4 x[N][2] = {};
#pragma unroll
    for (int h = 0; h < N; ++h)
      if (h < have) {
        x[h][0] = *reinterpret_cast<const f32x4 *>(from + 32 * h);
        x[h][1] = *reinterpret_cast<const f32x4 *>(from + 32 * h + 4);
      }
    float most = 0.f;
#pragma unroll
    for (int h = 0; h < N; ++h)
#pragma unroll
      for (int c = 0; c < 8; ++c) most = fmaxf(most, fabsf(x[h][c >> 2][c & 3]));
    most = larger(most, [](uint32_t a, uint32_t b) { return __builtin_amdgcn_permlane16_swap(a, b, false, false); });
    most = larger(most, [](uint32_t a, uint32_t b) { return __builtin_amdgcn_permlane32_swap(a, b, false, false); });
    up = 15 - __builtin_amdgcn_frexp_expf(most);  // (of 0 and infinity: 15)
#pragma unroll
    for (int h = 0; h < N; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[h][c] = pack2<kF16>(ldexpf(x[h][c >> 1][2 * (c & 1)], up),
                              ldexpf(x[h][c >> 1][2 * (c & 1) + 1], up));
  }
  __device__ __forceinline__ float back(float sum) const { return ldexpf(sum, -up); }
};

}  // namespace
}  // namespace gemm_f32_impl
