// The backward pass through an expert's second product and its activation
// (gemm_experts.h).  16,384 pairs of 64 experts, 2048 / 1024: 200 us, of which the
// matrix instructions' share at a library product's rate is 53; the rest is tiles that
// end with four stored matrices, and their 256 rows read again from `saved` in fp32.
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

// v = W2[e]^T dy for each pair, in fp32, and from it and the saved factors p and q
// (u = p s q, s = 1 / (1 + exp(-p))):
//   the gate's gradient        sum_i v[i] u[i]     (in parts: this wave's columns)
//   gate v q s (1 + p (1 - s)) and gate v p s, the gradients of p and q, and
//   gate u, W2's gradient's operand: in 16 bits, as the operands that they are.
template <class T, int FMT, int S>
struct Du {
  typedef RowJob Job;
  typedef KcSide<T::BM, S, T::WAVES> A;
  typedef KmSide<T::BN, S, T::WAVES> B;
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
    a.init(p.dY, 2 * ((p.T - 1) * p.lddy + p.H),
           [&](int i, int q) __attribute__((always_inline)) {
             return i < j.rows ? p.dY + token.at[q] * p.lddy : nullptr;
           },
           p.H, kNever, wave, lane);
    const int i0 = T::BN * j.tn;
    const uint16_t *w = p.W2 + (long long)p.H * j.e * p.ld2 + i0;
    b.init(w, w, p.ld2, p.H, kNever, p.I - i0 < T::BN ? p.I - i0 : T::BN, wave, lane);
  }
  __device__ __forceinline__ void store(const Job &j, const f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15, g = lane >> 4;
    const int *list = ws_at<int>(p, p.at.list) + j.first;
    float *dg = ws_at<float>(p, p.at.dg) + ((long long)T::WGN * j.tn + wn) * p.T * p.top;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int row = 16 * (T::WGM * i + wm) + l16;
      if (16 * (T::WGM * i + wm) >= j.rows) continue;  // uniform
      const bool in = row < j.rows;
      const long long place = j.first + (in ? row : 0);
      const float gate = p.gates[list[in ? row : 0]];
      uint16_t *us = ws_at<uint16_t>(p, p.at.u) + place * p.at.ipitch;
      uint16_t *dh = ws_at<uint16_t>(p, p.at.dh) + place * 2 * p.at.ipitch;
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < T::TBN; m += 2) {
        const int at = T::BN * j.tn + 16 * (wn * T::TBN + m);
        f32x4 u[2], dp[2], dq[2];  // zeros from I to the pitch
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c0 = at + 16 * h + 4 * g, left = p.I - c0;
          f32x4 x{0, 0, 0, 0}, y{0, 0, 0, 0};
          const float *saved = p.saved + place * 2 * p.I + c0;
          if (left >= 4) {
            x = *reinterpret_cast<const f32x4u *>(saved);
            y = *reinterpret_cast<const f32x4u *>(saved + p.I);
          } else {
#pragma unroll
            for (int c = 0; c < 3; ++c)
              if (c < left) x[c] = saved[c], y[c] = saved[p.I + c];
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float sg = 1.f / (1.f + expf(-x[c])), v = acc[i][m + h][c];
            const float silu = x[c] * sg, full = silu * y[c];
            if (c < left) sum += v * full;
            dp[h][c] = c < left ? gate * v * y[c] * sg * (1.f + x[c] * (1.f - sg)) : 0.f;
            dq[h][c] = c < left ? gate * v * silu : 0.f;
            u[h][c] = c < left ? gate * full : 0.f;
          }
        }
        const Eights eu = eights<FMT>(u[0], u[1], lane), ep = eights<FMT>(dp[0], dp[1], lane),
                     eq = eights<FMT>(dq[0], dq[1], lane);
        if (in && at < p.at.ipitch) {  // whole 64s
          *reinterpret_cast<u32x4 *>(us + at + eu.at) = eu.v;
          *reinterpret_cast<u32x4 *>(dh + at + ep.at) = ep.v;
          *reinterpret_cast<u32x4 *>(dh + p.at.ipitch + at + eq.at) = eq.v;
        }
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (in && g == 0) dg[place] = sum;
    }
  }
};

template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) experts_du_kernel(ExpertsProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int rows = row_tiles(p), columns = (int)ceil_div(p.I, T::BN);
  Du<T, FMT, S> op{p, Share(rows * columns), rows, columns, wave, lane, {}, {}, {}};
  tile_loop<T, FMT, S>(lds, op, op.share.count, wave, lane);
}

}  // namespace

hipError_t launch_experts_du(const ExpertsProblem &p, hipStream_t s) {
  const bool w = by_words(p.dY, p.H) && by_words(p.W2, p.I);
  return choose_tiles(p.tile, even_tiles(p) * ceil_div(p.I, p.tile), du_direct(p), w, [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.I, T::BN);
    return GEMM_F32_LAUNCH_ROWS(experts_du_kernel, T, S, tiles);
  });
}

}  // namespace gemm_f32_impl
