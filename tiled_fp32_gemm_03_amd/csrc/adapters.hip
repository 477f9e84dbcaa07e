// A shared projection with low-rank adapters for many rows (gemm_adapters.h): the
// rows in the order of their adapters, A[r] x as products of few columns with K in
// parts, then the projection's tiles, which add B[r] of scale A[r] x for each run of
// rows with one adapter before they are stored.
//
// Bound as any product of such tiles: 8,192 rows, 4096 x 4096, 16 adapters of rank 32 take 254
// to 271 us by box, a call among others (1.03 to 1.10 PFLOP/s).  Traced, calls apart from
// one another take 300: 265 in the projection (238 at least), 18 for A x, 11 for the order,
// 6 to join.
#include "adapters_rank.hpp"
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

template <class T>
__device__ inline T *ws_at(const AdaptersProblem &p, long long off) {
  return reinterpret_cast<T *>(p.ws + off);
}

// ---- A[r] x ------------------------------------------------------------------------

typedef RowTile<32, 32, 2, 2> Narrow;
static_assert(Narrow::BM == kAdaptersRows && Narrow::BN == kAdaptersRows, "adapters_space");

struct LowJob {
  int steps, rows;
  int e, first, tn, split;
};
template <class T, int FMT, int S>
struct Low {
  typedef LowJob Job;
  typedef KcSide<T::BM, S, T::WAVES> A;
  typedef KcSide<T::BN, S, T::WAVES> B;
  const AdaptersProblem &p;
  const Share share;
  const int rows, columns, wave, lane;
  A a;
  B b;
  TokenRows<A> token;

  __device__ Job job(int t) const {
    const int per = rows * columns, id = share.tile(t), split = id / per, in = id - split * per;
    const int tm = uniform(in % rows);
    const int *at = ws_at<int>(p, p.at.order.tiles) + 4 + 4LL * tm;
    Job j;
    j.split = uniform(split);
    j.tn = uniform(in / rows);
    j.e = uniform(at[0]), j.first = uniform(at[1]), j.rows = uniform(at[2]);
    j.steps = (values(j) + kStepK - 1) / kStepK;
    return j;
  }
  // of K in the job's part
  __device__ int values(const Job &j) const {
    const int left = p.K - j.split * p.at.chunk;
    return left < p.at.chunk ? left : p.at.chunk;
  }
  __device__ __forceinline__ void fetch(const Job &j) {
    token.fetch(ws_at<int>(p, p.at.order.list) + j.first, j.rows, wave, lane);
  }
  __device__ __forceinline__ void begin(const Job &j) {
    const int k0 = j.split * p.at.chunk, n = values(j);
    const uint16_t *x = p.X + k0, *m = p.A + (long long)p.R * j.e * p.lda + k0;
    a.init(x, 2 * ((p.T - 1) * p.ldx + n),
           [&](int i, int q) __attribute__((always_inline)) {
             return i < j.rows ? x + token.at[q] * p.ldx : nullptr;
           },
           n, kNever, wave, lane);
    b.init(m, 2 * ((p.R - 1) * p.lda + n),
           [&](int c, int) __attribute__((always_inline)) {
             const int r = T::BN * j.tn + c;
             return r < p.R ? m + r * p.lda : nullptr;
           },
           n, kNever, wave, lane);
  }
  __device__ __forceinline__ void store(const Job &j, const f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15, g = lane >> 4;
    float *part = ws_at<float>(p, p.at.part) + (long long)j.split * p.T * p.at.rpitch;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int row = 16 * (T::WGM * i + wm) + l16;
      if (row >= j.rows) continue;
#pragma unroll
      for (int m = 0; m < T::TBN; ++m)  // rpitch: whole tiles
        *reinterpret_cast<f32x4 *>(part + (j.first + row) * p.at.rpitch + T::BN * j.tn +
                                   16 * (wn * T::TBN + m) + 4 * g) = acc[i][m];
    }
  }
};
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) adapters_low_kernel(AdaptersProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int rows = uniform(*ws_at<int>(p, p.at.order.tiles));
  const int columns = (int)ceil_div(p.R, T::BN);
  Low<T, FMT, S> op{p, Share(rows * columns * p.at.splits), rows, columns, wave, lane, {}, {}, {}};
  tile_loop<T, FMT, S>(lds, op, op.share.count, wave, lane);
}

// v: the parts added in order, times the scale.  Four values to a thread.
template <int FMT>
__global__ void __launch_bounds__(256) adapters_join_kernel(AdaptersProblem p) {
  const int per = (int)(p.at.rpitch / 4);
  const long long i = 256LL * blockIdx.x + threadIdx.x;
  const int place = (int)(i / per);
  if (place >= ws_at<int>(p, p.at.order.start)[p.count]) return;  // rows with an adapter come first
  const float *part = ws_at<float>(p, p.at.part) + 4 * i;
  f32x4 sum{0, 0, 0, 0};
  for (int s = 0; s < p.at.splits; ++s)
    sum += *reinterpret_cast<const f32x4 *>(part + s * p.T * p.at.rpitch);
  const int r = p.ids[ws_at<int>(p, p.at.order.list)[place]];
  if (p.scales) sum *= p.scales[r];
  const int left = p.R - 4 * (int)(i - (long long)place * per);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c >= left) sum[c] = 0.f;
  Kept<FMT>::store(ws_at<typename Kept<FMT>::type>(p, p.at.v) + 4 * i, sum);
}

// ---- the projection -------------------------------------------------------------------

struct WideJob {
  int steps, rows;
  int first, tn, run, runs, split;
};
template <class T, int FMT, int S>
struct Wide {
  typedef WideJob Job;
  typedef KcSide<T::BM, S, T::WAVES> A;
  typedef KcSide<T::BN, S, T::WAVES> B;
  const AdaptersProblem &p;
  const Share share;
  const int rows, columns, wave, lane;
  A a;
  B b;
  TokenRows<A> token;

  __device__ Job job(int t) const {
    int tm, tn;
    const int id = share.tile(t), split = uniform(id / (rows * columns));
    tile_coords(id - split * rows * columns, rows, columns, tm, tn);
    tm = uniform(tm);
    const int *runs = ws_at<int>(p, p.at.order.runs), *of = ws_at<int>(p, p.at.order.tile_run);
    Job j;
    j.split = split;
    j.steps = (values(split) + kStepK - 1) / kStepK;
    j.tn = uniform(tn);
    j.first = T::BM * tm;
    j.rows = p.T - j.first < T::BM ? p.T - j.first : T::BM;
    j.run = uniform(of[tm]);
    // The last run of the tile; rows without an adapter are the last run of all.
    int last = uniform(runs[0]) - 1;
    if (j.first + j.rows < p.T) {
      last = uniform(of[tm + 1]);
      if (uniform(runs[4 + 4 * last + 1]) == j.first + j.rows) --last;
    }
    if (uniform(runs[4 + 4 * last]) == p.count) --last;
    j.runs = split == 0 ? last - j.run + 1 : 0;  // the first part of K adds them
    return j;
  }
  // of K in a part
  __device__ int values(int split) const {
    const int left = p.K - split * p.at.wide_chunk;
    return left < p.at.wide_chunk ? left : p.at.wide_chunk;
  }
  __device__ __forceinline__ void fetch(const Job &j) {
    token.fetch(ws_at<int>(p, p.at.order.list) + j.first, j.rows, wave, lane);
  }
  __device__ __forceinline__ void begin(const Job &j) {
    const int k0 = j.split * p.at.wide_chunk, n = values(j.split);
    const uint16_t *x = p.X + k0, *w = p.W + k0;
    a.init(x, 2 * ((p.T - 1) * p.ldx + n),
           [&](int i, int q) __attribute__((always_inline)) {
             return i < j.rows ? x + token.at[q] * p.ldx : nullptr;
           },
           n, kNever, wave, lane);
    b.init(w, 2 * ((p.N - 1) * p.ldw + n),
           [&](int c, int) __attribute__((always_inline)) {
             const int row = T::BN * j.tn + c;
             return row < p.N ? w + row * p.ldw : nullptr;
           },
           n, kNever, wave, lane);
  }
  // Adds B[r] v.  The matrix instruction multiplies all 16 rows of a block; the sums
  // of rows that are not the run's are dropped, not multiplied by zeros: an
  // infinity in one request's B is none of the others'.
  __device__ __forceinline__ void add_run(const Job &j, int run, f32x4 (&acc)[T::TBM][T::TBN],
                                          int wave, int lane) const {
    const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15, g = lane >> 4;
    const int *at = ws_at<int>(p, p.at.order.runs) + 4 + 4LL * run;
    const int from = uniform(at[1]) - j.first, to = from + uniform(at[2]);
    const uint16_t *m = p.B + (long long)p.N * uniform(at[0]) * p.ldb;
    const auto *v = ws_at<typename Kept<FMT>::type>(p, p.at.v) + j.first * p.at.rpitch;
#pragma unroll 1
    for (int r0 = 0; r0 < p.R; r0 += 32) {
      const int r = r0 + 8 * g;
      u32x4 bf[T::TBN];
#pragma unroll
      for (int c = 0; c < T::TBN; ++c) {
        const int n = T::BN * j.tn + 16 * (wn * T::TBN + c) + l16;
        bf[c] = load_guarded(
            reinterpret_cast<const unsigned char *>(m + (n < p.N ? n : p.N - 1) * p.ldb),
            r < p.R ? r : p.R, p.R);
      }
#pragma unroll
      for (int i = 0; i < T::TBM; ++i) {
        const int row0 = 16 * (T::WGM * i + wm);
        if (row0 + 16 <= from || row0 >= to || row0 >= j.rows) continue;  // uniform
        const bool in = row0 + l16 >= from && row0 + l16 < to && row0 + l16 < j.rows;
        const LowRank<FMT, 1> x(v + (in ? row0 + l16 : row0) * p.at.rpitch + r, 1);
#pragma unroll
        for (int c = 0; c < T::TBN; ++c) {
          const f32x4 sum = mfma_rows<FMT>(__builtin_bit_cast(i16x8, bf[c]),
                                           __builtin_bit_cast(i16x8, x.v[0]), f32x4{0, 0, 0, 0});
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][c][q] += in ? x.back(sum[q]) : 0.f;
        }
      }
    }
  }
  __device__ __forceinline__ void store(const Job &j, f32x4 (&acc)[T::TBM][T::TBN], int wave,
                                        int lane) const {
    const int wm = wave / T::WGN, wn = wave % T::WGN, l16 = lane & 15;
#pragma unroll 1
    for (int run = j.run; run < j.run + j.runs; ++run) add_run(j, run, acc, wave, lane);
    if (p.at.wide_splits > 1) {
      float *sums = ws_at<float>(p, p.at.wide_part) + (long long)j.split * p.T * p.at.npitch;
#pragma unroll
      for (int i = 0; i < T::TBM; ++i) {
        const int row = 16 * (T::WGM * i + wm) + l16;
        if (row >= j.rows) continue;
#pragma unroll
        for (int m = 0; m < T::TBN; ++m) {
          const int n = T::BN * j.tn + 16 * (wn * T::TBN + m) + 4 * (lane >> 4);
          if (n < p.N)
            *reinterpret_cast<f32x4 *>(sums + (j.first + row) * p.at.npitch + n) = acc[i][m];
        }
      }
      return;
    }
    const int *list = ws_at<int>(p, p.at.order.list) + j.first;
#pragma unroll
    for (int i = 0; i < T::TBM; ++i) {
      const int row = 16 * (T::WGM * i + wm) + l16;
      if (16 * (T::WGM * i + wm) >= j.rows) continue;  // uniform
      const bool in = row < j.rows;
      uint16_t *y = p.Y + list[in ? row : 0] * p.ldy;
#pragma unroll
      for (int m = 0; m < T::TBN; m += 2) {
        const int n = T::BN * j.tn + 16 * (wn * T::TBN + m);
        const Eights e = eights<FMT>(acc[i][m], acc[i][m + 1], lane);
        if (in) store_eights(y + n, e, p.N - n);
      }
    }
  }
};
template <class T, int FMT, int S>
__global__ void __launch_bounds__(T::THREADS, kWavesPerSimd<T>) adapters_wide_kernel(AdaptersProblem p) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int rows = (int)ceil_div(p.T, T::BM), columns = (int)ceil_div(p.N, T::BN);
  Wide<T, FMT, S> op{p, Share(rows * columns * p.at.wide_splits), rows, columns, wave, lane, {}, {}, {}};
  tile_loop<T, FMT, S>(lds, op, op.share.count, wave, lane);
}

// y: the parts of K added in order.  Eight values to a thread.
template <int FMT>
__global__ void __launch_bounds__(256) adapters_sum_kernel(AdaptersProblem p) {
  const int per = (int)(p.at.npitch / 8);
  const long long i = 256LL * blockIdx.x + threadIdx.x;
  const int place = (int)(i / per), n = 8 * (int)(i - (long long)place * per);
  if (place >= p.T) return;
  const float *part = ws_at<float>(p, p.at.wide_part) + place * p.at.npitch + n;
  float y[8] = {};
  for (int s = 0; s < p.at.wide_splits; ++s) {
    const f32x4 *q = reinterpret_cast<const f32x4 *>(part + s * p.T * p.at.npitch);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] += a[c], y[4 + c] += b[c];
  }
  store8<FMT>(p.Y, ws_at<int>(p, p.at.order.list)[place] * p.ldy + n, p.N - n, y);
}

}  // namespace

hipError_t launch_adapters_tiles(const AdaptersProblem &p, hipStream_t s) {
  const bool d = direct(p.X, p.ldx, p.K, p.T) && direct(p.W, p.ldw, p.K, p.N);
  const bool w = by_words(p.X, p.K) && by_words(p.W, p.K);
  const int tile = d ? p.at.tile : Small::BM;
  ExpertsProblem order{};
  order.T = p.T, order.E = p.count + 1, order.top = 1, order.ids = p.ids;
  order.tile = kAdaptersRows, order.rest = 1, order.run_tile = tile;
  order.ws = p.ws, order.at = p.at.order;
  hipError_t e = launch_list(order, s);
  if (e == hipSuccess && p.count > 0) {
    const bool ad = direct(p.X, p.ldx, p.K, p.T) && direct(p.A, p.lda, p.K, p.R);
    const bool aw = by_words(p.X, p.K) && by_words(p.A, p.K);
    const long long tiles =
        p.at.order.most_tiles * ceil_div(p.R, Narrow::BN) * p.at.splits;
    auto low = [&](auto how) {
      constexpr int S = decltype(how)::value;
      return GEMM_F32_LAUNCH_ROWS(adapters_low_kernel, Narrow, S, tiles);
    };
    e = ad ? low(std::integral_constant<int, kDirect>{})
           : aw ? low(std::integral_constant<int, kByWords>{})
                : low(std::integral_constant<int, kAnyRows>{});
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)ceil_div(p.T * (p.at.rpitch / 4), 256));
    e = p.format == kBf16 ? launch_kernel(adapters_join_kernel<kBf16>, grid, dim3(256), s, p)
                          : launch_kernel(adapters_join_kernel<kF16>, grid, dim3(256), s, p);
  }
  if (e != hipSuccess) return e;
  const long long all = ceil_div(p.T, tile) * ceil_div(p.N, tile) * p.at.wide_splits;
  e = choose_tiles(tile, all, d, w, [&](auto tiles, auto how) {
    typedef decltype(tiles) T;
    constexpr int S = decltype(how)::value;
    return GEMM_F32_LAUNCH_ROWS(adapters_wide_kernel, T, S, all);
  });
  if (e != hipSuccess || p.at.wide_splits == 1) return e;
  const dim3 grid((unsigned)ceil_div(p.T * (p.at.npitch / 8), 256));
  return p.format == kBf16 ? launch_kernel(adapters_sum_kernel<kBf16>, grid, dim3(256), s, p)
                           : launch_kernel(adapters_sum_kernel<kF16>, grid, dim3(256), s, p);
}

}  // namespace gemm_f32_impl
