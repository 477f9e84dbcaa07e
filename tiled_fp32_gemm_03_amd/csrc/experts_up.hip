// The experts' first product (gemm_experts.h): u = silu(W1[e][:I] x) (W1[e][I:] x)
// for the tokens that ask for expert e.
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

// A tile's columns are BN / 2 values of u: its blocks of 16 columns are rows of
// the gate and of the other factor in turn, so that a lane ends with both.
// u goes on in 16 bits: it is the second product's operand, and its rounding is
// of the size of the result's own.  SAVE keeps both factors' sums in fp32, for the
// backward pass.
template <class T, int FMT, int S, bool SAVE>
__global__ void __launch_bounds__(256, kPerSimd<T>) experts_up_kernel(ExpertsProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * T::STAGE];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, g = lane >> 4;
  constexpr int kU = T::BN / 2;
  const int *token = ws_at<int>(p, p.at.token);
  each_row_tile(p, (int)ceil_div(p.I, kU), [&](int tm, int tn) __attribute__((always_inline)) {
    const Rows r = row_tile(p, tm);
    const uint16_t *w = p.W1 + 2LL * p.I * r.e * p.ld1;
    const int i0 = kU * tn;
    KcSide<T::BM, S> a;
    a.init(p.X, 2 * ((p.T - 1) * p.ldx + p.H),
           [&](int i) __attribute__((always_inline)) {
             return i < r.n ? p.X + token[r.first + i] * p.ldx : nullptr;
           },
           p.H, kNever, wave, lane);
    KcSide<T::BN, S> b;
    b.init(w, 2 * ((2LL * p.I - 1) * p.ld1 + p.H),
           [&](int j) __attribute__((always_inline)) {
             const int i = i0 + 16 * (j >> 5) + (j & 15);
             return i < p.I ? w + ((j & 16) ? p.I + i : i) * p.ld1 : nullptr;
           },
           p.H, kNever, wave, lane);
    f32x4 acc[T::TBM][T::TBN];
    const int blocks = blocks_of(r.n, wm);
    tile_product<T, FMT, S>(lds, a, b, (int)ceil_div(p.H, kStepK), blocks, wave, lane, acc);
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int row = 16 * (2 * i + wm) + l16;
      if (row >= r.n) continue;
      const long long place = r.first + row;
#pragma unroll
      for (int q = 0; q < T::TBN / 2; ++q) {
        const int at = i0 + 16 * (wn * T::TBN / 2 + q) + 4 * g, left = p.I - at;
        if (at >= p.at.ipitch) continue;
        const f32x4 x = acc[i][2 * q], y = acc[i][2 * q + 1];
        f32x4 u;
#pragma unroll
        for (int c = 0; c < 4; ++c)  // zeros from I to the pitch
          u[c] = c < left ? x[c] / (1.f + expf(-x[c])) * y[c] : 0.f;
        *reinterpret_cast<u32x2 *>(ws_at<uint16_t>(p, p.at.u) + place * p.at.ipitch + at) =
            u32x2{pack2<FMT>(u[0], u[1]), pack2<FMT>(u[2], u[3])};
        if constexpr (SAVE) {
          if (left > 0) {
            store4<kF32>(p.saved, place * 2 * p.I + at, left, x);
            store4<kF32>(p.saved, place * 2 * p.I + p.I + at, left, y);
          }
        }
      }
    }
  });
}

}  // namespace

hipError_t launch_experts_up(const ExpertsProblem &p, hipStream_t s) {
  const bool d = direct(p.X, p.ldx, p.H, p.T) && direct(p.W1, p.ld1, p.H, 2LL * p.I);
  const bool w = by_words(p.X, p.H) && by_words(p.W1, p.H);
  return choose_tiles(p, d, w, [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.I, T::BN / 2);
    if (p.saved)
      return p.format == kBf16 ? launch_tiles(experts_up_kernel<T, kBf16, S, true>, p, tiles, s)
                               : launch_tiles(experts_up_kernel<T, kF16, S, true>, p, tiles, s);
    return p.format == kBf16 ? launch_tiles(experts_up_kernel<T, kBf16, S, false>, p, tiles, s)
                             : launch_tiles(experts_up_kernel<T, kF16, S, false>, p, tiles, s);
  });
}

}  // namespace gemm_f32_impl
