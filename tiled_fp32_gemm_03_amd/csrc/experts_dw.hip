// The gradients of the experts' weights (gemm_experts.h): sums over an expert's
// pairs, whose k runs down the rows of both operands.
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

// Calls run(e, tm, tn) for each of this workgroup's tiles of E matrices.
template <class Run>
__device__ __forceinline__ void each_weight_tile(const ExpertsProblem &p, int tiles_m, int tiles_n,
                                                 Run run) {
  const int per = tiles_m * tiles_n, total = p.E * per;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int id = xcd_remap(t, total), e = id / per;
    int tm, tn;
    tile_coords(id - e * per, tiles_m, tiles_n, tm, tn);
    // (divisions: the compiler forms them in vector registers)
    run(__builtin_amdgcn_readfirstlane(e), __builtin_amdgcn_readfirstlane(tm),
        __builtin_amdgcn_readfirstlane(tn));
    if (t + (int)gridDim.x < total) ks_lds_barrier();
  }
}
__device__ inline Rows expert_rows(const ExpertsProblem &p, int e) {
  const int *start = ws_at<int>(p, p.at.start);
  const int first = __builtin_amdgcn_readfirstlane(start[e]);
  return {e, first, __builtin_amdgcn_readfirstlane(start[e + 1]) - first};
}
// The tokens of an expert's pairs (any readable place where there are none).
__device__ inline const int *tokens_of(const ExpertsProblem &p, const Rows &r) {
  return r.n > 0 ? ws_at<int>(p, p.at.token) + r.first : ws_at<int>(p, p.at.start);
}
__device__ inline int at_most(int a, int b) { return a < b ? a : b; }

// dW1[e] = dh^T x.  The tile's rows are columns of dh: ipitch of the gate's, I of
// which are rows of dW1, then as many of the other factor's.
template <class T, int FMT, int S>
__global__ void __launch_bounds__(256, kPerSimd<T>) experts_dw1_kernel(ExpertsProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * T::STAGE];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, g = lane >> 4;
  const int ip = (int)p.at.ipitch;
  each_weight_tile(p, (int)ceil_div(2 * ip, T::BM), (int)ceil_div(p.H, T::BN),
                   [&](int e, int tm, int tn) __attribute__((always_inline)) {
    const Rows r = expert_rows(p, e);
    const int m0 = T::BM * tm, h0 = T::BN * tn, rows = at_most(T::BM, 2 * ip - m0);
    f32x4 acc[T::TBM][T::TBN];
    KmSide<T::BM, S> a;
    KmListSide<T::BN, S> b;
    const uint16_t *dh = ws_at<uint16_t>(p, p.at.dh) + 2LL * ip * r.first + m0;
    a.init(dh, dh, 2 * ip, r.n, kNever, rows, wave, lane);
    b.init(p.X + h0, 2 * ((p.T - 1) * p.ldx + p.H - h0), p.ldx, tokens_of(p, r), r.n,
           at_most(T::BN, p.H - h0), wave, lane);
    tile_product<T, FMT, S>(lds, a, b, (int)ceil_div(r.n, kStepK), blocks_of(rows, wm), wave, lane,
                            acc);
    uint16_t *out = p.dW1 + 2LL * p.I * e * p.lddw1;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int c = m0 + 16 * (2 * i + wm) + l16, second = c >= ip, at = c - (second ? ip : 0);
      if (c >= 2 * ip || at >= p.I) continue;
      const long long row = (second ? p.I : 0) + at;
#pragma unroll
      for (int j = 0; j < T::TBN; ++j) {
        const int h = h0 + 16 * (wn * T::TBN + j) + 4 * g;
        store4<FMT>(out, row * p.lddw1 + h, p.H - h, acc[i][j]);
      }
    }
  });
}

// dW2[e] = dy^T (gate u).
template <class T, int FMT, int S>
__global__ void __launch_bounds__(256, kPerSimd<T>) experts_dw2_kernel(ExpertsProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * T::STAGE];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, g = lane >> 4;
  const int ip = (int)p.at.ipitch;
  each_weight_tile(p, (int)ceil_div(p.H, T::BM), (int)ceil_div(p.I, T::BN),
                   [&](int e, int tm, int tn) __attribute__((always_inline)) {
    const Rows r = expert_rows(p, e);
    const int h0 = T::BM * tm, i0 = T::BN * tn, rows = at_most(T::BM, p.H - h0);
    f32x4 acc[T::TBM][T::TBN];
    KmListSide<T::BM, S> a;
    KmSide<T::BN, S> b;
    const uint16_t *u = ws_at<uint16_t>(p, p.at.u) + (long long)ip * r.first + i0;
    a.init(p.dY + h0, 2 * ((p.T - 1) * p.lddy + p.H - h0), p.lddy, tokens_of(p, r), r.n, rows, wave,
           lane);
    b.init(u, u, ip, r.n, kNever, at_most(T::BN, ip - i0), wave, lane);
    tile_product<T, FMT, S>(lds, a, b, (int)ceil_div(r.n, kStepK), blocks_of(rows, wm), wave, lane,
                            acc);
    uint16_t *out = p.dW2 + (long long)p.H * e * p.lddw2;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int h = h0 + 16 * (2 * i + wm) + l16;
      if (h >= p.H) continue;
#pragma unroll
      for (int j = 0; j < T::TBN; ++j) {
        const int at = i0 + 16 * (wn * T::TBN + j) + 4 * g;
        store4<FMT>(out, h * p.lddw2 + at, p.I - at, acc[i][j]);
      }
    }
  });
}

}  // namespace

hipError_t launch_experts_dw(const ExpertsProblem &p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.dW1) e = choose_tiles(p, direct(p.X, p.ldx, p.H, p.T), by_words(p.X, p.H),
                                    [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.E * ceil_div(2 * p.at.ipitch, T::BM) * ceil_div(p.H, T::BN);
    return p.format == kBf16 ? launch_tiles(experts_dw1_kernel<T, kBf16, S>, p, tiles, s)
                             : launch_tiles(experts_dw1_kernel<T, kF16, S>, p, tiles, s);
  });
  if (e != hipSuccess || !p.dW2) return e;
  return choose_tiles(p, direct(p.dY, p.lddy, p.H, p.T), by_words(p.dY, p.H),
                      [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.E * ceil_div(p.H, T::BM) * ceil_div(p.I, T::BN);
    return p.format == kBf16 ? launch_tiles(experts_dw2_kernel<T, kBf16, S>, p, tiles, s)
                             : launch_tiles(experts_dw2_kernel<T, kF16, S>, p, tiles, s);
  });
}

}  // namespace gemm_f32_impl
