// The products whose rows go back to their tokens (gemm_experts.h): the second one
// of the forward pass, gates[pair] W2[e] u, and of the backward pass
// W1[e]^T dh.  Each pair's row is kept apart, in 16 bits, and experts_sum adds a
// token's rows in fp32 in the order of its choices: no atomics, the same bits every
// run.  (In 32 bits those rows cost twice the traffic; rounding each of them is off by
// as little as rounding the result.)
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

template <class T, int FMT, bool GATES>
__device__ __forceinline__ void store_part(const ExpertsProblem &p, const Rows &r, int h0,
                                           const f32x4 (&acc)[T::TBM][T::TBN], int wave, int lane) {
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, g = lane >> 4;
  const int *list = ws_at<int>(p, p.at.list);
#pragma unroll
  for (int i = 0; i < T::TBM; ++i) {
    const int row = 16 * (2 * i + wm) + l16;
    if (row >= r.n) continue;
    const long long pair = list[r.first + row];
    const float gate = GATES ? p.gates[pair] : 1.f;
#pragma unroll
    for (int j = 0; j < T::TBN; ++j) {
      const int h = h0 + 16 * (wn * T::TBN + j) + 4 * g;
      if (h >= p.H) continue;
      const f32x4 v = GATES ? acc[i][j] * gate : acc[i][j];
      *reinterpret_cast<u32x2 *>(ws_at<uint16_t>(p, p.at.part) + pair * p.at.hpitch + h) =
          u32x2{pack2<FMT>(v[0], v[1]), pack2<FMT>(v[2], v[3])};
    }
  }
}

template <class T, int FMT, int S>
__global__ void __launch_bounds__(256, kPerSimd<T>) experts_down_kernel(ExpertsProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * T::STAGE];
  const int lane = threadIdx.x & 63, wave = wave_id();
  each_row_tile(p, (int)ceil_div(p.H, T::BN), [&](int tm, int tn) __attribute__((always_inline)) {
    const Rows r = row_tile(p, tm);
    const uint16_t *u = ws_at<uint16_t>(p, p.at.u) + r.first * p.at.ipitch;
    const uint16_t *w = p.W2 + (long long)p.H * r.e * p.ld2;
    const int h0 = T::BN * tn;
    KcSide<T::BM, S> a;
    a.init(u, 2 * r.n * p.at.ipitch,
           [&](int i) __attribute__((always_inline)) {
             return i < r.n ? u + i * p.at.ipitch : nullptr;
           },
           p.I, kNever, wave, lane);
    KcSide<T::BN, S> b;
    b.init(w, 2 * ((p.H - 1LL) * p.ld2 + p.I),
           [&](int j) __attribute__((always_inline)) {
             return h0 + j < p.H ? w + (h0 + j) * p.ld2 : nullptr;
           },
           p.I, kNever, wave, lane);
    f32x4 acc[T::TBM][T::TBN];
    tile_product<T, FMT, S>(lds, a, b, (int)ceil_div(p.I, kStepK), blocks_of(r.n, wave >> 1), wave,
                            lane, acc);
    store_part<T, FMT, true>(p, r, h0, acc, wave, lane);
  });
}

// dh's rows are two parts of ipitch values, the gate's and the other factor's; so
// are W1's rows, I of each.
template <class T, int FMT, int S>
__global__ void __launch_bounds__(256, kPerSimd<T>) experts_dx_kernel(ExpertsProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * T::STAGE];
  const int lane = threadIdx.x & 63, wave = wave_id();
  each_row_tile(p, (int)ceil_div(p.H, T::BN), [&](int tm, int tn) __attribute__((always_inline)) {
    const Rows r = row_tile(p, tm);
    const long long pitch = 2 * p.at.ipitch;
    const int half = (int)(p.at.ipitch / kStepK), h0 = T::BN * tn;
    const uint16_t *dh = ws_at<uint16_t>(p, p.at.dh) + r.first * pitch;
    const uint16_t *w = p.W1 + 2LL * p.I * r.e * p.ld1 + h0;
    KcSide<T::BM, S> a;
    a.init(dh, 2 * r.n * pitch,
           [&](int i) __attribute__((always_inline)) {
             return i < r.n ? dh + i * pitch : nullptr;
           },
           p.I, half, wave, lane);
    KmSide<T::BN, S> b;
    b.init(w, w + p.I * p.ld1, p.ld1, p.I, half, p.H - h0 < T::BN ? p.H - h0 : T::BN, wave, lane);
    f32x4 acc[T::TBM][T::TBN];
    tile_product<T, FMT, S>(lds, a, b, 2 * half, blocks_of(r.n, wave >> 1), wave, lane, acc);
    store_part<T, FMT, false>(p, r, h0, acc, wave, lane);
  });
}

}  // namespace

hipError_t launch_experts_down(const ExpertsProblem &p, hipStream_t s) {
  return choose_tiles(p, direct(p.W2, p.ld2, p.I, p.H), by_words(p.W2, p.I),
                      [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.H, T::BN);
    return p.format == kBf16 ? launch_tiles(experts_down_kernel<T, kBf16, S>, p, tiles, s)
                             : launch_tiles(experts_down_kernel<T, kF16, S>, p, tiles, s);
  });
}

hipError_t launch_experts_dx(const ExpertsProblem &p, hipStream_t s) {
  return choose_tiles(p, direct(p.W1, p.ld1, p.H, kStepK), by_words(p.W1, p.H),
                      [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.H, T::BN);
    return p.format == kBf16 ? launch_tiles(experts_dx_kernel<T, kBf16, S>, p, tiles, s)
                             : launch_tiles(experts_dx_kernel<T, kF16, S>, p, tiles, s);
  });
}

}  // namespace gemm_f32_impl
