// Thin products with MX weights: 16-bit activations (gemm_mx_a16) and the
// few-row form of gemm_mx.  See mx_thin.hpp for the operands.  A workgroup
// takes 16 NB columns of C and up to 16 MB rows; its waves take the pieces of
// K in turn and their sums are added in wave order through LDS.
#include "mx_internal.hpp"
#include "mx_thin.hpp"

namespace gemm_f32_impl {
namespace {

// C's blocks [i][b] of all waves, summed and stored, four blocks at a time.
template <int WAVES, int MB, int NB>
__device__ __forceinline__ void thin_store(const f32x4 (&acc)[MB][NB], f32x4 (*part)[4][64],
                                           long long m0, long long n0, int M, int N, void *C,
                                           long long ldc, int c_format) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  constexpr int kBlocks = MB * NB, kRound = kBlocks < 4 ? kBlocks : 4;
#pragma unroll
  for (int r = 0; r < kBlocks; r += kRound) {
#pragma unroll
    for (int q = 0; q < kRound; ++q) part[wave][q][lane] = acc[(r + q) / NB][(r + q) % NB];
    __syncthreads();
    if (wave < kRound) {
      f32x4 sum = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum += part[w][wave][lane];
      const long long m = m0 + 16 * ((r + wave) / NB) + (lane & 15);
      const long long n = n0 + 16 * ((r + wave) % NB) + 4 * (lane >> 4), left = N - n;
      if (m < M) store4_fmt(c_format, C, m * ldc + n, (int)(left < 4 ? left : 4), sum);
    }
    __syncthreads();
  }
}

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

template <int A, int MB, int NB, int WAVES, bool ODD>
__global__ void __launch_bounds__(64 * WAVES) mx_thin_kernel(ThinProblem p) {
  __shared__ f32x4 part[WAVES][4][64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int l16 = lane & 15;
  const long long n0 = 16LL * NB * blockIdx.x;
  Rows w[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    auto row = [&](int r) { return n0 + 16 * b + r < p.N ? n0 + 16 * b + r : p.N - 1; };
#pragma unroll
    for (int t = 0; t < 4; ++t) w[b].p[t] = p.B.codes + row(load_row(lane, t)) * p.B.ld;
    w[b].q = p.B.scales + row(l16) * p.B.lds;
  }
  for (long long m0 = 16LL * MB * blockIdx.y; m0 < p.M; m0 += 16LL * MB * gridDim.y) {
    typename ActRow<A>::type a[MB];
    bool valid[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      auto row = [&](int r) { return m0 + 16 * i + r < p.M ? m0 + 16 * i + r : p.M - 1; };
      if constexpr (A == kMx) {
        valid[i] = m0 + 16 * i + load_row(lane, 0) < p.M;
#pragma unroll
        for (int t = 0; t < 4; ++t) a[i].p[t] = p.A + row(load_row(lane, t)) * p.lda;
        a[i].q = p.SA + row(l16) * p.ldsa;
      } else {
        valid[i] = m0 + 16 * i + l16 < p.M;
        a[i] = {p.A + row(l16) * p.lda, nullptr};
      }
    }
    Thin<kMx, A, MB, NB, ODD> t;
    t.clear();
    t.run(a, valid, w, wave, WAVES, p.K, lane);
    thin_store<WAVES, MB, NB>(t.acc, part, m0, n0, p.M, p.N, p.C, p.ldc, p.c_format);
  }
}

template <int A, int MB, int NB, bool ODD>
hipError_t launch_thin_blocks(const ThinProblem &p, hipStream_t s) {
  const long long gy = ceil_div(p.M, 16 * MB);
  const dim3 grid((unsigned)ceil_div(p.N, 16 * NB), (unsigned)(gy < kMaxGridY ? gy : kMaxGridY));
  if (p.K <= 4 * kPieceK<kMx>)
    return launch_kernel(mx_thin_kernel<A, MB, NB, 4, ODD>, grid, dim3(256), s, p);
  return launch_kernel(mx_thin_kernel<A, MB, NB, 8, ODD>, grid, dim3(512), s, p);
}

template <int A, bool ODD>
hipError_t launch_thin(const ThinProblem &p, hipStream_t s) {
  // Columns per workgroup: as many as leave a workgroup per compute unit.
  const long long cols = ceil_div(p.N, 16);
  const int nb = cols >= 4 * 256 ? 4 : cols >= 2 * 256 ? 2 : 1;
  if (p.M <= 16)
    return nb == 4   ? launch_thin_blocks<A, 1, 4, ODD>(p, s)
           : nb == 2 ? launch_thin_blocks<A, 1, 2, ODD>(p, s)
                     : launch_thin_blocks<A, 1, 1, ODD>(p, s);
  return nb == 4   ? launch_thin_blocks<A, 2, 4, ODD>(p, s)
         : nb == 2 ? launch_thin_blocks<A, 2, 2, ODD>(p, s)
                   : launch_thin_blocks<A, 2, 1, ODD>(p, s);
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
