// Internal declarations of the MX operators: what the C-ABI front end
// (mx_abi.hip) hands to the kernels' translation units.
#pragma once

#include <hip/hip_runtime.h>

#include "mx_plan.hpp"

namespace gemm_f32_impl {

// An MX matrix: codes and scales, row pitches in bytes.
struct MxMatrix {
  const unsigned char *codes;
  long long ld;
  const unsigned char *scales;
  long long lds;
};

// One conversion between a row-major matrix (pitch in elements) and an MX
// matrix of `rows` rows of K values.
struct MxConvert {
  int rows, K;
  const void *x;  // quantise: source
  void *y;        // dequantise: destination
  long long ldx;
  unsigned char *codes;
  long long ld;
  unsigned char *scales;
  long long lds;
};
hipError_t launch_mx_quantize(int format, int along, const MxConvert &c, hipStream_t s);
hipError_t launch_mx_dequantize(int format, int along, const MxConvert &c, hipStream_t s);

// C = A B^T with both operands MX; C in `c_format`, pitch in elements.
struct MxProblem {
  int M, N, K;
  MxMatrix A, B;
  void *C;
  long long ldc;
  int c_format;
};
hipError_t launch_mx_thin(const MxProblem &p, hipStream_t s);  // any M, 32 rows at a time
hipError_t launch_mx_gemm(int entry, const MxProblem &p, hipStream_t s);

// C = A B^T with A in 16 bits (pitch in elements) and B MX.
struct MxA16Problem {
  int M, N, K;
  const uint16_t *A;
  long long lda;
  int a_format;
  MxMatrix B;
  void *C;
  long long ldc;
  int c_format;
};
hipError_t launch_mx_a16(const MxA16Problem &p, hipStream_t s);

// The mixture-of-experts layer (gemm_moe.h).
struct MoeProblem {
  int T, E, top, H, I;
  const uint16_t *X;
  long long ldx;
  const uint16_t *R;
  long long ldr;
  int format;
  const unsigned char *W1;  // rows of 2-byte values or of codes
  long long ld1;            // bytes
  const unsigned char *S1;
  long long lds1;
  const unsigned char *W2;
  long long ld2;
  const unsigned char *S2;
  long long lds2;
  int mx, renormalize;
  void *Y;
  long long ldy;
  int y_format;
  int *ids;  // may be null
  float *gates;
  unsigned char *ws;
  MoeSpace at;
};
hipError_t launch_moe(const MoeProblem &p, hipStream_t s);

// The launches of a product whose grid's x goes along columns, 16 of them to
// a workgroup of up to 512 threads or more to more: several where one grid
// cannot have as many workgroups (a grid has fewer than 2^32 threads in x; past that
// the runtime takes their number modulo 2^32, without an error).
constexpr long long kMostColumns = 1LL << 26;
template <class P, class Launch>
hipError_t in_columns(const P &p, Launch launch) {
  const long long size = format_bytes(p.c_format);
  for (long long n = 0; n < p.N; n += kMostColumns) {
    P q = p;
    q.N = (int)(p.N - n < kMostColumns ? p.N - n : kMostColumns);
    q.B.codes += n * p.B.ld;
    q.B.scales += n * p.B.lds;
    q.C = static_cast<char *>(p.C) + n * size;
    const hipError_t e = launch(q);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// C = 0 in any format.
hipError_t launch_mx_zero(void *C, int M, int N, long long ldc, int c_format, hipStream_t s);

}  // namespace gemm_f32_impl
