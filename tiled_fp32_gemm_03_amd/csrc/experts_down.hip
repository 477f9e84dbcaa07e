// The products whose rows go back to their tokens (gemm_experts.h): the second one
// of the forward pass, gates[pair] W2[e] u, and of the backward pass
// W1[e]^T dh.  Each pair's row is kept apart, in fp32, and experts_sum adds a token's
// rows in the order of its choices: no atomics, the same bits every run.  (In 16 bits
// 8,192 tokens on 8 experts, 4096 / 4096 took 3% less, and results were off by 1.7
// times their own rounding instead of 1.4.)  That size: 540 to 580 us, 0.95 to 1.02 PFLOP/s,
// and the sums 59; W1^T dh of 16,384 pairs of 64 experts, 2048 / 1024: 252 us.
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

template <class T, bool GATES>
__device__ __forceinline__ void store_part(const ExpertsProblem &p, const RowJob &j,
                                           const f32x4 (&acc)[T::TBM][T::TBN], int wave, int lane) {
  const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15, g = lane >> 4;
  const int *list = ws_at<int>(p, p.at.list) + j.first;
#pragma unroll
  for (int i = 0; i < T::TBM; ++i) {
    const int row = 16 * (T::WGM * i + wm) + l16;
    if (16 * (T::WGM * i + wm) >= j.rows) continue;  // uniform
    const bool in = row < j.rows;
    if (!in) continue;
    const long long pair = list[row];
    const float gate = GATES ? p.gates[pair] : 1.f;
    float *part = ws_at<float>(p, p.at.part) + pair * p.at.hpitch;
#pragma unroll
    for (int m = 0; m < T::TBN; ++m) {
      const int h = T::BN * j.tn + 16 * (wn * T::TBN + m) + 4 * g;
      if (h < p.H) *reinterpret_cast<f32x4 *>(part + h) = GATES ? acc[i][m] * gate : acc[i][m];
    }
  }
}

template <class T, int FMT, int S>
struct Down {
  typedef RowJob Job;
  typedef KcSide<T::BM, S, T::WAVES> A;
  typedef KcSide<T::BN, S, T::WAVES> B;
  const ExpertsProblem &p;
  const Share share;
  const int rows, columns, wave, lane;
  A a;
  B b;

  __device__ Job job(int t) const {
    return row_job(p, share.tile(t), rows, columns, (int)ceil_div(p.I, kStepK));
  }
  __device__ __forceinline__ void fetch(const Job &) {}
  __device__ __forceinline__ void begin(const Job &j) {
    const uint16_t *u = ws_at<uint16_t>(p, p.at.u) + j.first * p.at.ipitch;
    a.init(u, 2 * j.rows * p.at.ipitch,
           [&](int i, int) __attribute__((always_inline)) {
             return i < j.rows ? u + i * p.at.ipitch : nullptr;
           },
           p.I, kNever, wave, lane);
    const uint16_t *w = p.W2 + (long long)p.H * j.e * p.ld2;
    b.init(w, 2 * ((p.H - 1LL) * p.ld2 + p.I),
           [&](int c, int) __attribute__((always_inline)) {
             const int h = T::BN * j.tn + c;
             return h < p.H ? w + h * p.ld2 : nullptr;
           },
           p.I, kNever, wave, lane);
  }
  __device__ __forceinline__ void store(const Job &j, const f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    store_part<T, true>(p, j, acc, wave, lane);
  }
};

// dh's rows are two parts of ipitch values, the gate's and the other factor's; so
// are W1's rows, I of each.
template <class T, int FMT, int S>
struct Dx {
  typedef RowJob Job;
  typedef KcSide<T::BM, S, T::WAVES> A;
  typedef KmSide<T::BN, S, T::WAVES> B;
  const ExpertsProblem &p;
  const Share share;
  const int rows, columns, wave, lane;
  A a;
  B b;

  __device__ Job job(int t) const {
    return row_job(p, share.tile(t), rows, columns, (int)(2 * p.at.ipitch / kStepK));
  }
  __device__ __forceinline__ void fetch(const Job &) {}
  __device__ __forceinline__ void begin(const Job &j) {
    const long long pitch = 2 * p.at.ipitch;
    const int half = (int)(p.at.ipitch / kStepK), h0 = T::BN * j.tn;
    const uint16_t *dh = ws_at<uint16_t>(p, p.at.dh) + j.first * pitch;
    a.init(dh, 2 * j.rows * pitch,
           [&](int i, int) __attribute__((always_inline)) {
             return i < j.rows ? dh + i * pitch : nullptr;
           },
           p.I, half, wave, lane);
    const uint16_t *w = p.W1 + 2LL * p.I * j.e * p.ld1 + h0;
    b.init(w, w + p.I * p.ld1, p.ld1, p.I, half, p.H - h0 < T::BN ? p.H - h0 : T::BN, wave, lane);
  }
  __device__ __forceinline__ void store(const Job &j, const f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    store_part<T, false>(p, j, acc, wave, lane);
  }
};

template <class T, int FMT, int S, template <class, int, int> class Op>
__device__ __forceinline__ void part_tiles(const ExpertsProblem &p) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int rows = row_tiles(p), columns = (int)ceil_div(p.H, T::BN);
  Op<T, FMT, S> op{p, Share(rows * columns), rows, columns, wave, lane, {}, {}};
  tile_loop<T, FMT, S>(lds, op, op.share.count, wave, lane);
}
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) experts_down_kernel(ExpertsProblem p) {
  part_tiles<T, FMT, S, Down>(p);
}
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) experts_dx_kernel(ExpertsProblem p) {
  part_tiles<T, FMT, S, Dx>(p);
}

}  // namespace

hipError_t launch_experts_down(const ExpertsProblem &p, hipStream_t s) {
  return choose_tiles(p.tile, even_tiles(p) * ceil_div(p.H, p.tile), down_direct(p), by_words(p.W2, p.I),
                      [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.H, T::BN);
    return GEMM_F32_LAUNCH_ROWS(experts_down_kernel, T, S, tiles);
  });
}

hipError_t launch_experts_dx(const ExpertsProblem &p, hipStream_t s) {
  return choose_tiles(p.tile, even_tiles(p) * ceil_div(p.H, p.tile), dx_direct(p), by_words(p.W1, p.H),
                      [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.at.most_tiles * ceil_div(p.H, T::BN);
    return GEMM_F32_LAUNCH_ROWS(experts_dx_kernel, T, S, tiles);
  });
}

}  // namespace gemm_f32_impl
