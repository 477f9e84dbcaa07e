// 16-bit activations times MX weights (gemm_mx_a16): see mx_thin.hpp for the
// operands.  The workgroup's waves take 128-deep steps of K in turn and their
// sums are added in a fixed order through LDS.
#include "mx_internal.hpp"
#include "mx_thin.hpp"

namespace gemm_f32_impl {
namespace {

template <int AF, int MB, int W>
__global__ void __launch_bounds__(64 * W) mx_a16_kernel(MxA16Problem p) {
  __shared__ f32x4 part[W][MB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const long long n0 = 16LL * blockIdx.x;
  const long long rb = n0 + l16 < p.N ? n0 + l16 : p.N - 1;
  const WRow row{p.B.codes + rb * p.B.ld, p.B.scales + rb * p.B.lds};
  const int steps = (int)ceil_div(p.K, 128);
  for (long long m0 = 16LL * MB * blockIdx.y; m0 < p.M; m0 += 16LL * MB * gridDim.y) {
    const uint16_t *arow[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const long long m = m0 + 16 * i + l16;
      arow[i] = p.A + (m < p.M ? m : p.M - 1) * p.lda;
    }
    f32x4 acc[MB] = {};
    for (int step = wave; step < steps; step += W) {
      u32x4 w[4];
      load_weights<kWMx>(row, step, g, p.K, w);
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const long long k = 128LL * step + thin_k<kWMx>(g, j);
          acc[i] = thin_mfma<kWMx, AF>(w[j], load_act(arow[i], k, p.K - k), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < MB; i += W) {
      f32x4 sum = part[0][i][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) sum += part[w][i][lane];
      const long long m = m0 + 16 * i + l16, n = n0 + 4 * g, left = p.N - n;
      if (m < p.M) store4_fmt(p.c_format, p.C, m * p.ldc + n, (int)(left < 4 ? left : 4), sum);
    }
    __syncthreads();
  }
}

template <int AF>
hipError_t launch_a16(const MxA16Problem &p, hipStream_t s) {
  constexpr int W = 8;
  const int mb = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
  const long long gy = ceil_div(p.M, 16 * mb);
  const dim3 grid((unsigned)ceil_div(p.N, 16), (unsigned)(gy < kMaxGridY ? gy : kMaxGridY));
  auto kern = mb == 1   ? mx_a16_kernel<AF, 1, W>
              : mb == 2 ? mx_a16_kernel<AF, 2, W>
                        : mx_a16_kernel<AF, 4, W>;
  return launch_kernel(kern, grid, dim3(64 * W), s, p);
}

}  // namespace

hipError_t launch_mx_a16(const MxA16Problem &p, hipStream_t s) {
  return p.a_format == kBf16 ? launch_a16<kBf16>(p, s) : launch_a16<kF16>(p, s);
}

}  // namespace gemm_f32_impl
