// The experts' first product (gemm_experts.h): u = silu(W1[e][:I] x) (W1[e][I:] x)
// for the tokens that ask for expert e.
//
// Bound by bringing operands to LDS: 16,384 pairs of 8 experts, 4096 / 4096, took 1,016 us
// (1.08 PFLOP/s), 734 without the loads and 940 without the matrix instructions.
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

// A tile's columns are BN / 2 values of u: its blocks of 16 columns are rows of
// the gate and of the other factor in turn, so that a lane ends with both.
// u goes on in 16 bits: it is the second product's operand, and its rounding is
// of the size of the result's own.  SAVE keeps both factors' sums in fp32, for the
// backward pass.
template <class T, int FMT, int S, bool SAVE>
struct Up {
  typedef RowJob Job;
  typedef KcSide<T::BM, S, T::WAVES> A;
  typedef KcSide<T::BN, S, T::WAVES> B;
  static constexpr int kU = T::BN / 2;
  const ExpertsProblem &p;
  const Share share;
  const int rows, columns, wave, lane;
  A a;
  B b;
  TokenRows<A> token;

  __device__ Job job(int t) const {
    return row_job(p, share.tile(t), rows, columns, (int)ceil_div(p.H, kStepK));
  }
  __device__ __forceinline__ void fetch(const Job &j) {
    token.fetch(ws_at<int>(p, p.at.token) + j.first, j.rows, wave, lane);
  }
  __device__ __forceinline__ void begin(const Job &j) {
    a.init(p.X, 2 * ((p.T - 1) * p.ldx + p.H),
           [&](int i, int q) __attribute__((always_inline)) {
             return i < j.rows ? p.X + token.at[q] * p.ldx : nullptr;
           },
           p.H, kNever, wave, lane);
    const uint16_t *w = p.W1 + 2LL * p.I * j.e * p.ld1;
    b.init(w, 2 * ((2LL * p.I - 1) * p.ld1 + p.H),
           [&](int c, int) __attribute__((always_inline)) {
             const int i = kU * j.tn + 16 * (c >> 5) + (c & 15);
             return i < p.I ? w + ((c & 16) ? p.I + i : i) * p.ld1 : nullptr;
           },
           p.H, kNever, wave, lane);
  }
  __device__ __forceinline__ void store(const Job &j, const f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int row = 16 * (T::WGM * i + wm) + l16;
      if (16 * (T::WGM * i + wm) >= j.rows) continue;  // uniform
      const bool in = row < j.rows;
      const long long place = j.first + row;
#pragma unroll
      for (int q = 0; q < T::TBN / 2; q += 2) {
        const int at = kU * j.tn + 16 * (wn * T::TBN / 2 + q);
        f32x4 u[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c0 = at + 16 * h + 4 * g, left = p.I - c0;
          const f32x4 x = acc[i][2 * (q + h)], y = acc[i][2 * (q + h) + 1];
#pragma unroll
          for (int c = 0; c < 4; ++c)  // zeros from I to the pitch
            u[h][c] = c < left ? x[c] / (1.f + expf(-x[c])) * y[c] : 0.f;
          if constexpr (SAVE) {
            if (in && left > 0) {
              store4<kF32>(p.saved, place * 2 * p.I + c0, left, x);
              store4<kF32>(p.saved, place * 2 * p.I + p.I + c0, left, y);
            }
          }
        }
        const Eights e = eights<FMT>(u[0], u[1], lane);
        if (in && at < p.at.ipitch)  // whole 64s
          *reinterpret_cast<u32x4 *>(ws_at<uint16_t>(p, p.at.u) + place * p.at.ipitch + at + e.at) =
              e.v;
      }
    }
  }
};

template <class T, int FMT, int S, bool SAVE>
__device__ __forceinline__ void up_tiles(const ExpertsProblem &p) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int rows = row_tiles(p), columns = (int)ceil_div(p.I, T::BN / 2);
  Up<T, FMT, S, SAVE> op{p, Share(rows * columns), rows, columns, wave, lane, {}, {}, {}};
  tile_loop<T, FMT, S>(lds, op, op.share.count, wave, lane);
}
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) experts_up_kernel(ExpertsProblem p) {
  up_tiles<T, FMT, S, false>(p);
}
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) experts_up_save_kernel(ExpertsProblem p) {
  up_tiles<T, FMT, S, true>(p);
}

}  // namespace

hipError_t launch_experts_up(const ExpertsProblem &p, hipStream_t s) {
  const bool w = by_words(p.X, p.H) && by_words(p.W1, p.H);
  return choose_tiles(p.tile, even_tiles(p) * ceil_div(p.I, p.tile / 2), up_direct(p), w, [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.I, T::BN / 2);
    return p.saved ? GEMM_F32_LAUNCH_ROWS(experts_up_save_kernel, T, S, tiles)
                   : GEMM_F32_LAUNCH_ROWS(experts_up_kernel, T, S, tiles);
  });
}

}  // namespace gemm_f32_impl
