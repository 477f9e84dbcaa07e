// Thin products with MX weights: 16-bit activations (gemm_mx_a16) and the
// few-row form of gemm_mx.  See mx_thin.hpp for the operands.  A workgroup
// takes 16 NB columns of C and up to 16 MB rows; its waves take the pieces of
// K in turn and their sums are added in wave order through LDS.
#include "mx_internal.hpp"
#include "mx_thin.hpp"

namespace gemm_f32_impl {
namespace {

// A's rows: 16-bit values, or MX rows (a_scales not null).
struct ThinProblem {
  int M, N, K;
  const unsigned char *A;
  long long lda;  // bytes
  const unsigned char *SA;
  long long ldsa;
  MxMatrix B;
  void *C;
  long long ldc;
  int c_format;
};

// LDS for activations: what leaves room for two workgroups, and the most that
// one round of pieces may take.
constexpr int kThinLds = 64 * 1024, kThinMostLds = 140 * 1024;

// ks: the waves that share 16 columns.
template <int A, int MB, int WAVES, bool ODD>
__global__ void __launch_bounds__(64 * WAVES) mx_thin_kernel(ThinProblem p, Tile tile, int ks) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  typedef Thin<kMx, A, MB, 1, ODD> Product;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int l16 = lane & 15, g = lane >> 4;
  const long long n0 = 16LL * (blockIdx.x * (WAVES / ks) + wave / ks);
  const long long n = n0 + l16 < p.N ? n0 + l16 : p.N - 1;
  const Row w[1] = {{p.B.codes + n * p.B.ld, p.B.scales + n * p.B.lds}};
  const typename Product::Walk at{wave & (ks - 1), ks, n0 < p.N, false};
  typename Product::Weights x;
  Product::load_first(x, w, at, p.K, lane);
  for (long long m0 = 16LL * MB * blockIdx.y; m0 < p.M; m0 += 16LL * MB * gridDim.y) {
    Product t;
    t.clear();
    const int rows = (int)(p.M - m0 < 16 * MB ? p.M - m0 : 16 * MB);
    t.template run<64 * WAVES>(
        lds, tile, [&](int r) { return Row{p.A + (m0 + r) * p.lda, p.SA + (m0 + r) * p.ldsa}; },
        rows, w, w, x, at, p.K, lane);
    if (ks > 1) {  // the waves' sums, added in wave order
      f32x4 *part = reinterpret_cast<f32x4 *>(lds);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MB; ++i) part[(i * WAVES + wave) * 64 + lane] = t.acc[i][0];
      __syncthreads();
      if (at.first == 0)
        for (int q = 1; q < ks; ++q)
#pragma unroll
          for (int i = 0; i < MB; ++i) t.acc[i][0] += part[(i * WAVES + wave + q) * 64 + lane];
    }
    if (at.first != 0 || !at.any) continue;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int r = 16 * i + l16;
      if (r >= rows) continue;
      const long long col = n0 + 4 * g, left = p.N - col;
      store4_fmt(p.c_format, p.C, (m0 + r) * p.ldc + col, (int)(left < 4 ? left : 4), t.acc[i][0]);
    }
  }
}

template <int A, int MB, int WAVES, bool ODD>
hipError_t launch_thin_waves(const ThinProblem &p, int ks, int keep, hipStream_t s) {
  const long long groups = ceil_div(p.N, 16), gy = ceil_div(p.M, 16 * MB);
  Tile tile{keep, tile_values<A>(keep, p.K, ks * kPieceK<kMx>, kThinLds / MB)};
  const int bytes = MB * act_bytes<A>(tile), parts = ks > 1 ? MB * WAVES * 1024 : 0;
  const dim3 grid((unsigned)ceil_div(groups * ks, WAVES),
                  (unsigned)(gy < kMaxGridY ? gy : kMaxGridY));
  ThinProblem q = p;
  void *args[] = {&q, &tile, &ks};
  return hipLaunchKernel(reinterpret_cast<const void *>(mx_thin_kernel<A, MB, WAVES, ODD>), grid,
                         dim3(64 * WAVES), args, (size_t)(bytes > parts ? bytes : parts), s);
}

template <int A, int MB, bool ODD>
hipError_t launch_thin_rows(const ThinProblem &p, hipStream_t s) {
  const long long groups = ceil_div(p.N, 16);
  const int keep = p.M <= 4 ? 4 : 16;
  int ks = waves_per_group(groups, p.K, kPieceK<kMx>, 8, 8 * 256);
  while (ks > 1 && MB * act_bytes<A>(Tile{keep, ks * kPieceK<kMx>}) > kThinMostLds) ks /= 2;
  return ks == 8 || groups * ks >= 8 * 256 ? launch_thin_waves<A, MB, 8, ODD>(p, ks, keep, s)
                                           : launch_thin_waves<A, MB, 4, ODD>(p, ks, keep, s);
}

template <int A, bool ODD>
hipError_t launch_thin(const ThinProblem &p, hipStream_t s) {
  return p.M <= 16 ? launch_thin_rows<A, 1, ODD>(p, s) : launch_thin_rows<A, 2, ODD>(p, s);
}

// Rows that start in the middle of a word, of a matrix that starts on one.
bool odd_rows(const void *base, long long pitch_bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 3) == 0 && (pitch_bytes & 3) != 0;
}

}  // namespace

hipError_t launch_mx_a16(const MxA16Problem &p, hipStream_t s) {
  const ThinProblem t{p.M, p.N, p.K, reinterpret_cast<const unsigned char *>(p.A), 2 * p.lda,
                      nullptr, 0, p.B, p.C, p.ldc, p.c_format};
  if (odd_rows(p.A, 2 * p.lda) && p.M > 1)
    return p.a_format == kBf16 ? launch_thin<kBf16, true>(t, s) : launch_thin<kF16, true>(t, s);
  return p.a_format == kBf16 ? launch_thin<kBf16, false>(t, s) : launch_thin<kF16, false>(t, s);
}

hipError_t launch_mx_thin(const MxProblem &p, hipStream_t s) {
  const ThinProblem t{p.M, p.N, p.K, p.A.codes, p.A.ld, p.A.scales, p.A.lds, p.B, p.C, p.ldc,
                      p.c_format};
  return launch_thin<kMx, false>(t, s);
}

}  // namespace gemm_f32_impl
