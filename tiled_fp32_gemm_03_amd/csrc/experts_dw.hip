// The gradients of the experts' weights (gemm_experts.h): sums over an expert's
// pairs, whose k runs down the rows of both operands.  The rows of X (dY) are listed by
// expert and read in place: no sorted copy.  16,384 pairs of 64 experts, 2048 / 1024: 292 us
// for dW1 and 168 for dW2, four steps to a tile, so that its start and stores weigh as much.
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

// A tile of one expert's gradient.
struct WeightJob {
  int steps, rows;
  int e, first, n, m0, n0;
};
template <class T>
__device__ inline WeightJob weight_job(const ExpertsProblem &p, int tile, int tiles_m, int tiles_n,
                                       int rows) {
  const int per = tiles_m * tiles_n;
  // (divisions: the compiler forms them in vector registers)
  const int e = __builtin_amdgcn_readfirstlane(tile / per);
  int tm, tn;
  tile_coords(tile - e * per, tiles_m, tiles_n, tm, tn);
  const int *start = ws_at<int>(p, p.at.start);
  WeightJob j;
  j.e = e;
  j.first = __builtin_amdgcn_readfirstlane(start[e]);
  j.n = __builtin_amdgcn_readfirstlane(start[e + 1]) - j.first;
  j.steps = (j.n + kStepK - 1) / kStepK;
  j.m0 = T::BM * __builtin_amdgcn_readfirstlane(tm);
  j.n0 = T::BN * __builtin_amdgcn_readfirstlane(tn);
  j.rows = rows - j.m0 < T::BM ? rows - j.m0 : T::BM;
  return j;
}
// The tokens of an expert's pairs (any readable place where there are none).
__device__ inline const int *tokens_of(const ExpertsProblem &p, const WeightJob &j) {
  return j.n > 0 ? ws_at<int>(p, p.at.token) + j.first : ws_at<int>(p, p.at.start);
}
__device__ inline int at_most(int a, int b) { return a < b ? a : b; }

// dW1[e] = dh^T x.  The tile's rows are columns of dh: ipitch of the gate's, I of
// which are rows of dW1, then as many of the other factor's.
template <class T, int FMT, int S>
struct Dw1 {
  typedef WeightJob Job;
  typedef KmSide<T::BM, S, T::WAVES> A;
  typedef KmListSide<T::BN, S, T::WAVES> B;
  const ExpertsProblem &p;
  const Share share;
  const int tiles_m, tiles_n, wave, lane;
  A a;
  B b;

  __device__ Job job(int t) const {
    return weight_job<T>(p, share.tile(t), tiles_m, tiles_n, (int)(2 * p.at.ipitch));
  }
  __device__ __forceinline__ void fetch(const Job &j) {
    b.init(p.X + j.n0, 2 * ((p.T - 1) * p.ldx + p.H - j.n0), p.ldx, tokens_of(p, j), j.n,
           at_most(T::BN, p.H - j.n0), wave, lane);
  }
  __device__ __forceinline__ void begin(const Job &j) {
    const long long pitch = 2 * p.at.ipitch;
    const uint16_t *dh = ws_at<uint16_t>(p, p.at.dh) + pitch * j.first + j.m0;
    a.init(dh, dh, pitch, j.n, kNever, j.rows, wave, lane);
  }
  __device__ __forceinline__ void store(const Job &j, const f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15, ip = (int)p.at.ipitch;
    uint16_t *out = p.dW1 + 2LL * p.I * j.e * p.lddw1;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int c = j.m0 + 16 * (T::WGM * i + wm) + l16, second = c >= ip, at = c - (second ? ip : 0);
      const bool in = c < 2 * ip && at < p.I;
      uint16_t *row = out + ((second ? p.I : 0) + at) * p.lddw1;
#pragma unroll
      for (int m = 0; m < T::TBN; m += 2) {
        const int h = j.n0 + 16 * (wn * T::TBN + m);
        const Eights e = eights<FMT>(acc[i][m], acc[i][m + 1], lane);
        if (in) store_eights(row + h, e, p.H - h);
      }
    }
  }
};

// dW2[e] = dy^T (gate u).
template <class T, int FMT, int S>
struct Dw2 {
  typedef WeightJob Job;
  typedef KmListSide<T::BM, S, T::WAVES> A;
  typedef KmSide<T::BN, S, T::WAVES> B;
  const ExpertsProblem &p;
  const Share share;
  const int tiles_m, tiles_n, wave, lane;
  A a;
  B b;

  __device__ Job job(int t) const {
    return weight_job<T>(p, share.tile(t), tiles_m, tiles_n, p.H);
  }
  __device__ __forceinline__ void fetch(const Job &j) {
    a.init(p.dY + j.m0, 2 * ((p.T - 1) * p.lddy + p.H - j.m0), p.lddy, tokens_of(p, j), j.n, j.rows,
           wave, lane);
  }
  __device__ __forceinline__ void begin(const Job &j) {
    const uint16_t *u = ws_at<uint16_t>(p, p.at.u) + p.at.ipitch * j.first + j.n0;
    b.init(u, u, p.at.ipitch, j.n, kNever, at_most(T::BN, (int)p.at.ipitch - j.n0), wave, lane);
  }
  __device__ __forceinline__ void store(const Job &j, const f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15;
    uint16_t *out = p.dW2 + (long long)p.H * j.e * p.lddw2;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int h = j.m0 + 16 * (T::WGM * i + wm) + l16;
      uint16_t *row = out + h * p.lddw2;
#pragma unroll
      for (int m = 0; m < T::TBN; m += 2) {
        const int at = j.n0 + 16 * (wn * T::TBN + m);
        const Eights e = eights<FMT>(acc[i][m], acc[i][m + 1], lane);
        if (h < p.H) store_eights(row + at, e, p.I - at);
      }
    }
  }
};

template <class T, int FMT, int S, template <class, int, int> class Op>
__device__ __forceinline__ void weight_tiles(const ExpertsProblem &p, int rows, int columns) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int tiles_m = (int)ceil_div(rows, T::BM), tiles_n = (int)ceil_div(columns, T::BN);
  Op<T, FMT, S> op{p, Share(p.E * tiles_m * tiles_n), tiles_m, tiles_n, wave, lane, {}, {}};
  tile_loop<T, FMT, S>(lds, op, op.share.count, wave, lane);
}
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) experts_dw1_kernel(ExpertsProblem p) {
  weight_tiles<T, FMT, S, Dw1>(p, (int)(2 * p.at.ipitch), p.H);
}
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) experts_dw2_kernel(ExpertsProblem p) {
  weight_tiles<T, FMT, S, Dw2>(p, p.H, p.I);
}

}  // namespace

hipError_t launch_experts_dw(const ExpertsProblem &p, hipStream_t s) {
  hipError_t e = hipSuccess;
  // (These tiles are not the list's: each of the two has its own.)
  const bool d1 = direct(p.X, p.ldx, p.H, p.T), d2 = direct(p.dY, p.lddy, p.H, p.T);
  const int t1 = d1 ? p.tile : Small::BM, t2 = d2 ? p.tile : Small::BM;
  if (p.dW1) e = choose_tiles(t1, p.E * ceil_div(2 * p.at.ipitch, t1) * ceil_div(p.H, t1), d1, by_words(p.X, p.H),
                              [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.E * ceil_div(2 * p.at.ipitch, T::BM) * ceil_div(p.H, T::BN);
    return GEMM_F32_LAUNCH_ROWS(experts_dw1_kernel, T, S, tiles);
  });
  if (e != hipSuccess || !p.dW2) return e;
  return choose_tiles(t2, p.E * ceil_div(p.H, t2) * ceil_div(p.I, t2), d2, by_words(p.dY, p.H),
                      [&](auto tile, auto how) {
    typedef decltype(tile) T;
    constexpr int S = decltype(how)::value;
    const long long tiles = p.E * ceil_div(p.H, T::BM) * ceil_div(p.I, T::BN);
    return GEMM_F32_LAUNCH_ROWS(experts_dw2_kernel, T, S, tiles);
  });
}

}  // namespace gemm_f32_impl
