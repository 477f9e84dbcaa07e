// The product of two MX matrices (gemm_mx.h), on
// v_mfma_scale_f32_16x16x128_f8f6f4: a lane's operand is one block of 32
// codes, 16 bytes, with its scale byte, so both operands are read in the
// layout they are stored in and a block is never taken apart.
#include "mx_internal.hpp"
#include "mx_values.hpp"
#include "addr_math.hpp"

namespace gemm_f32_impl {
namespace {

// Block `kb` of row `r`, with its scale byte; past the row's blocks zeros
// with scale 1, so that a product's partial last step adds exact zeros.
struct MxBlock {
  u32x4 codes;
  int scale;
};
__device__ inline MxBlock mx_load_block(const MxMatrix &m, long long r, int kb, int nb) {
  MxBlock x{u32x4{0, 0, 0, 0}, 127};
  if (kb < nb) {
    x.codes = *reinterpret_cast<const u32x4 *>(m.codes + r * m.ld + 16LL * kb);
    x.scale = m.scales[r * m.lds + kb];
  }
  return x;
}

// Entry 0: 64 x 64 tiles, 4 waves of 32 x 32, operands straight from memory
// with 64-bit addresses; rows past the matrices are read from the last row
// and not stored.
__global__ void __launch_bounds__(256) mx_direct_kernel(MxProblem p, int tiles_m, int tiles_n) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  int tm, tn;
  tile_coords(xcd_remap(blockIdx.x, gridDim.x), tiles_m, tiles_n, tm, tn);
  const long long m0 = 64LL * tm + 32 * (wave >> 1), n0 = 64LL * tn + 32 * (wave & 1);
  const int nb = (int)mx_blocks(p.K);
  long long ra[2], rb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ra[i] = m0 + 16 * i + l16 < p.M ? m0 + 16 * i + l16 : p.M - 1;
    rb[i] = n0 + 16 * i + l16 < p.N ? n0 + 16 * i + l16 : p.N - 1;
  }
  f32x4 acc[2][2] = {};
  for (int kb0 = 0; kb0 < nb; kb0 += 4) {
    MxBlock a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = mx_load_block(p.A, ra[i], kb0 + g, nb);
      b[i] = mx_load_block(p.B, rb[i], kb0 + g, nb);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = mfma_mx(b[j].codes, b[j].scale, a[i].codes, a[i].scale, acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const long long m = m0 + 16 * i + l16;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const long long n = n0 + 16 * j + 4 * g;
      const long long left = p.N - n;
      store4_fmt(p.c_format, p.C, m * p.ldc + n, (int)(left < 4 ? left : 4), acc[i][j]);
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) mx_zero_kernel(void *C, int M, int N, long long ldc) {
  for (long long m = blockIdx.y; m < M; m += gridDim.y)
    for (long long n = blockIdx.x * 256LL + threadIdx.x; n < N; n += gridDim.x * 256LL)
      store1<FMT>(C, m * ldc + n, 0.f);
}

}  // namespace

hipError_t launch_mx_zero(void *C, int M, int N, long long ldc, int c_format, hipStream_t s) {
  const long long gx = ceil_div(N, 256);
  const dim3 grid((unsigned)(gx < 1024 ? gx : 1024), (unsigned)(M < kMaxGridY ? M : kMaxGridY));
  auto kern = c_format == kF32 ? mx_zero_kernel<kF32> : mx_zero_kernel<kBf16>;  // 16-bit zeros are alike
  return launch_kernel(kern, grid, dim3(256), s, C, M, N, ldc);
}

hipError_t launch_mx_gemm(int entry, const MxProblem &p, hipStream_t s) {
  const long long tiles_m = ceil_div(p.M, 64), tiles_n = ceil_div(p.N, 64);
  if (tiles_m * tiles_n > 0x7fffffffLL) return hipErrorInvalidValue;
  return launch_kernel(mx_direct_kernel, dim3((unsigned)(tiles_m * tiles_n)), dim3(256), s, p,
                       (int)tiles_m, (int)tiles_n);
}

}  // namespace gemm_f32_impl
