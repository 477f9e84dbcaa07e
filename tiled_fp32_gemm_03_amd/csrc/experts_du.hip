// The backward pass through an expert's second product and its activation
// (gemm_experts.h).
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

// v = W2[e]^T dy for each pair, in fp32, and from it and the saved factors p and q
// (u = p s q, s = 1 / (1 + exp(-p))):
//   the gate's gradient        sum_i v[i] u[i]     (in parts: this wave's columns)
//   gate v q s (1 + p (1 - s)) and gate v p s, the gradients of p and q, and
//   gate u, W2's gradient's operand: in 16 bits, as the operands that they are.
template <class T, int FMT, int S>
__global__ void __launch_bounds__(256, kPerSimd<T>) experts_du_kernel(ExpertsProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * T::STAGE];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, g = lane >> 4;
  const int *token = ws_at<int>(p, p.at.token), *list = ws_at<int>(p, p.at.list);
  each_row_tile(p, (int)ceil_div(p.I, T::BN), [&](int tm, int tn) __attribute__((always_inline)) {
    const Rows r = row_tile(p, tm);
    const int i0 = T::BN * tn;
    const uint16_t *w = p.W2 + (long long)p.H * r.e * p.ld2 + i0;
    KcSide<T::BM, S> a;
    a.init(p.dY, 2 * ((p.T - 1) * p.lddy + p.H),
           [&](int i) __attribute__((always_inline)) {
             return i < r.n ? p.dY + token[r.first + i] * p.lddy : nullptr;
           },
           p.H, kNever, wave, lane);
    KmSide<T::BN, S> b;
    b.init(w, w, p.ld2, p.H, kNever, p.I - i0 < T::BN ? p.I - i0 : T::BN, wave, lane);
    f32x4 acc[T::TBM][T::TBN];
    tile_product<T, FMT, S>(lds, a, b, (int)ceil_div(p.H, kStepK), blocks_of(r.n, wm), wave, lane,
                            acc);
    uint16_t *us = ws_at<uint16_t>(p, p.at.u), *dhs = ws_at<uint16_t>(p, p.at.dh);
    float *dg = ws_at<float>(p, p.at.dg) + (2LL * tn + wn) * p.T * p.top;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int row = 16 * (2 * i + wm) + l16;
      if (16 * (2 * i + wm) >= r.n) continue;  // uniform
      const bool in = row < r.n;
      const long long place = r.first + (in ? row : 0);
      const float gate = p.gates[list[place]];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < T::TBN; ++j) {
        const int at = i0 + 16 * (wn * T::TBN + j) + 4 * g, left = p.I - at;
        if (!in || at >= p.at.ipitch) continue;
        f32x4 x{0, 0, 0, 0}, y{0, 0, 0, 0};
        const float *saved = p.saved + place * 2 * p.I + at;
        if (left >= 4) {
          x = *reinterpret_cast<const f32x4u *>(saved);
          y = *reinterpret_cast<const f32x4u *>(saved + p.I);
        } else {
#pragma unroll
          for (int c = 0; c < 3; ++c)
            if (c < left) x[c] = saved[c], y[c] = saved[p.I + c];
        }
        f32x4 u, dp, dq;  // zeros from I to the pitch
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float sg = 1.f / (1.f + expf(-x[c])), v = acc[i][j][c];
          const float silu = x[c] * sg;
          u[c] = silu * y[c];
          if (c < left) sum += v * u[c];
          dp[c] = c < left ? gate * v * y[c] * sg * (1.f + x[c] * (1.f - sg)) : 0.f;
          dq[c] = c < left ? gate * v * silu : 0.f;
          u[c] *= gate;
        }
        *reinterpret_cast<u32x2 *>(us + place * p.at.ipitch + at) =
            u32x2{pack2<FMT>(u[0], u[1]), pack2<FMT>(u[2], u[3])};
        uint16_t *dh = dhs + place * 2 * p.at.ipitch + at;
        *reinterpret_cast<u32x2 *>(dh) = u32x2{pack2<FMT>(dp[0], dp[1]), pack2<FMT>(dp[2], dp[3])};
        *reinterpret_cast<u32x2 *>(dh + p.at.ipitch) =
            u32x2{pack2<FMT>(dq[0], dq[1]), pack2<FMT>(dq[2], dq[3])};
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (in && g == 0) dg[place] = sum;
    }
  });
}

}  // namespace

hipError_t launch_experts_du(const ExpertsProblem &p, hipStream_t s) {
  const bool d = direct(p.dY, p.lddy, p.H, p.T) && direct(p.W2, p.ld2, p.I, kStepK);
  const bool w = by_words(p.dY, p.H) && by_words(p.W2, p.I);
  return choose_tiles(p, d, w, [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.I, T::BN);
    return p.format == kBf16 ? launch_tiles(experts_du_kernel<T, kBf16, S>, p, tiles, s)
                             : launch_tiles(experts_du_kernel<T, kF16, S>, p, tiles, s);
  });
}

}  // namespace gemm_f32_impl
