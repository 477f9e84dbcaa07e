// Quantisation to MX rows and back (gemm_mx.h), memory-bound conversions.
//
// Along rows, 16 lanes share 128 values of one row (4 blocks): a lane holds
// 8, a block's largest magnitude comes from two exchanges inside its 4
// lanes, each lane stores one 4-byte word of codes and the 16 lanes' first
// one word of 4 scale bytes.  Down columns, a workgroup takes 128 columns by
// 256 k: a lane reads two adjacent columns' 32 values each (coalesced along
// the rows of X), the codes are turned through LDS, and each MX row's 128
// bytes leave as 16-byte stores of 8 neighbouring lanes.
#include "addr_math.hpp"
#include "mx_internal.hpp"
#include "mx_values.hpp"

namespace gemm_f32_impl {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 128;  // values that 16 lanes share

// Lane exchanges inside a row of 16 lanes.
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;    // quad_perm [1,0,3,2] and [2,3,0,1]
constexpr int kRowRor4 = 0x124, kRowRor8 = 0x128;    // row_ror:4 and row_ror:8
__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// A workgroup's 16 groups of lanes cover 2^lg groups of 128 values along K
// and 16 >> lg rows.
struct RowPlace {
  bool in;      // whether the row has this group (of `groups`)
  int k0;       // this lane's first value
  int r, step;  // first row, and the step to the next
};
__device__ inline RowPlace row_place(int lg, int groups) {
  const int tid = threadIdx.x, gi = tid >> 4, per = 16 >> lg;
  const int g = (int)(blockIdx.x << lg) + (gi & ((1 << lg) - 1));
  return {g < groups, (g < groups ? g : 0) * kGroup + 8 * (tid & 15),
          (int)blockIdx.y * per + (gi >> lg), (int)gridDim.y * per};
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(MxConvert c, int lg, int groups) {
  const RowPlace at = row_place(lg, groups);
  if (!at.in) return;  // the same for the 16 lanes of a group
  const int nb = (int)mx_blocks(c.K);
  const int n = c.K - at.k0;               // values of this lane (may be <= 0)
  const int sub = threadIdx.x & 15;
  for (long long r = at.r; r < c.rows; r += at.step) {
    float v[8];
    load8<FMT>(c.x, r * c.ldx + at.k0, n, v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, mag_bits(v[j]));
    m = umax(m, dpp<kQuadXor1>(m));
    m = umax(m, dpp<kQuadXor2>(m));
    const uint32_t sb = scale_byte(m);
    if (at.k0 / 32 < nb)
      *reinterpret_cast<uint32_t *>(c.codes + r * c.ld + at.k0 / 2) = encode8(v, sb);
    uint32_t w = sb << (8 * (sub >> 2));
    w |= dpp<kRowRor4>(w);
    w |= dpp<kRowRor8>(w);
    if (sub == 0) *reinterpret_cast<uint32_t *>(c.scales + r * c.lds + at.k0 / 32) = w;
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) dequant_rows_kernel(MxConvert c, int lg, int groups) {
  const RowPlace at = row_place(lg, groups);
  const int n = c.K - at.k0;
  if (!at.in || n <= 0) return;
  for (long long r = at.r; r < c.rows; r += at.step) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(c.codes + r * c.ld + at.k0 / 2);
    const uint32_t sb = c.scales[r * c.lds + at.k0 / 32];
    float v[8];
    decode8(w, sb, v);
    store8<FMT>(c.y, r * c.ldx + at.k0, n, v);
  }
}

// Down columns: 128 MX rows (columns of X) by 256 k (8 blocks).
constexpr int kColRows = 128, kColBlocks = 8;
constexpr int kColPitch = 16 * kColBlocks + 16;  // LDS bytes per MX row (padded against banks)

template <int FMT>
__device__ inline f32x2 load2(const void *p, long long i, int n) {
  if (n >= 2) {
    if constexpr (FMT == kF32) {
      return *reinterpret_cast<const f32x2u *>(static_cast<const float *>(p) + i);
    } else {
      const uint32_t w = *reinterpret_cast<const u32h *>(static_cast<const uint16_t *>(p) + i);
      return f32x2{to_f32<FMT>((uint16_t)w), to_f32<FMT>((uint16_t)(w >> 16))};
    }
  }
  return f32x2{n > 0 ? load1<FMT>(p, i) : 0.f, 0.f};
}
template <int FMT>
__device__ inline void store2(void *p, long long i, int n, float a, float b) {
  if (n >= 2) {
    if constexpr (FMT == kF32)
      *reinterpret_cast<f32x2u *>(static_cast<float *>(p) + i) = f32x2{a, b};
    else
      *reinterpret_cast<u32h *>(static_cast<uint16_t *>(p) + i) = pack2<FMT>(a, b);
  } else if (n > 0) {
    store1<FMT>(p, i, a);
  }
}

// A workgroup's first column and first tile of k.  Neighbours share the lines
// that X's rows have at the edge between them, so they go to one XCD (its L2).
__device__ inline long long cols_of(int &kt) {
  const int lid = xcd_remap((int)(blockIdx.x + gridDim.x * blockIdx.y), (int)(gridDim.x * gridDim.y));
  kt = lid / (int)gridDim.x;
  return (long long)(lid % (int)gridDim.x) * kColRows;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) quant_cols_kernel(MxConvert c, int ktiles) {
  __shared__ __attribute__((aligned(16))) unsigned char tile[kColRows * kColPitch];
  __shared__ __attribute__((aligned(16))) unsigned char sc[kColRows * kColBlocks];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nb = (int)mx_blocks(c.K);
  const int scale_row = (int)mx_scale_bytes(c.K);
  int kt0;
  const long long r0 = cols_of(kt0);
  const int ncol = (int)(c.rows - r0 < kColRows ? c.rows - r0 : kColRows);
  for (int kt = kt0; kt < ktiles; kt += gridDim.y) {
    const int kb0 = kt * kColBlocks;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int blk = 2 * wave + b;
      const long long k0 = 32LL * (kb0 + blk), left = c.K - k0;
      float v[2][4][8];
      uint32_t m0 = 0, m1 = 0;
      // All 32 loads together where none needs a check (each behind its own, they
      // were waited for one by one: 8191 x 16383 fp32 235 us).
      if (left >= 32 && ncol == kColRows) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const f32x2 x = load2<FMT>(c.x, (k0 + k) * c.ldx + r0 + 2 * lane, 2);
          v[0][k >> 3][k & 7] = x[0];
          v[1][k >> 3][k & 7] = x[1];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          f32x2 x{0.f, 0.f};
          if (k < left)
            x = load2<FMT>(c.x, (k0 + k) * c.ldx + r0 + 2 * lane, ncol - 2 * lane);
          v[0][k >> 3][k & 7] = x[0];
          v[1][k >> 3][k & 7] = x[1];
        }
      }
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        m0 = umax(m0, mag_bits(v[0][k >> 3][k & 7]));
        m1 = umax(m1, mag_bits(v[1][k >> 3][k & 7]));
      }
      const uint32_t s0 = scale_byte(m0), s1 = scale_byte(m1);
      u32x4 w0, w1;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        w0[q] = encode8(v[0][q], s0);
        w1[q] = encode8(v[1][q], s1);
      }
      *reinterpret_cast<u32x4 *>(tile + (2 * lane) * kColPitch + 16 * blk) = w0;
      *reinterpret_cast<u32x4 *>(tile + (2 * lane + 1) * kColPitch + 16 * blk) = w1;
      sc[(2 * lane) * kColBlocks + blk] = (unsigned char)s0;
      sc[(2 * lane + 1) * kColBlocks + blk] = (unsigned char)s1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kColRows * kColBlocks / kThreads; ++i) {
      const int id = i * kThreads + tid, row = id / kColBlocks, blk = id % kColBlocks;
      if (row < ncol && kb0 + blk < nb)
        *reinterpret_cast<u32x4 *>(c.codes + (r0 + row) * c.ld + 16LL * (kb0 + blk)) =
            *reinterpret_cast<const u32x4 *>(tile + row * kColPitch + 16 * blk);
    }
    const int row = tid >> 1, half = 4 * (tid & 1);
    if (row < ncol && kb0 + half < scale_row)
      *reinterpret_cast<uint32_t *>(c.scales + (r0 + row) * c.lds + kb0 + half) =
          *reinterpret_cast<const uint32_t *>(sc + row * kColBlocks + half);
    __syncthreads();
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) dequant_cols_kernel(MxConvert c, int ktiles) {
  __shared__ __attribute__((aligned(16))) unsigned char tile[kColRows * kColPitch];
  __shared__ __attribute__((aligned(16))) unsigned char sc[kColRows * kColBlocks];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nb = (int)mx_blocks(c.K);
  int kt0;
  const long long r0 = cols_of(kt0);
  const int ncol = (int)(c.rows - r0 < kColRows ? c.rows - r0 : kColRows);
  for (int kt = kt0; kt < ktiles; kt += gridDim.y) {
    const int kb0 = kt * kColBlocks;
#pragma unroll
    for (int i = 0; i < kColRows * kColBlocks / kThreads; ++i) {
      const int id = i * kThreads + tid, row = id / kColBlocks, blk = id % kColBlocks;
      if (row < ncol && kb0 + blk < nb) {
        *reinterpret_cast<u32x4 *>(tile + row * kColPitch + 16 * blk) =
            *reinterpret_cast<const u32x4 *>(c.codes + (r0 + row) * c.ld + 16LL * (kb0 + blk));
        sc[row * kColBlocks + blk] = c.scales[(r0 + row) * c.lds + kb0 + blk];
      }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int blk = 2 * wave + b;
      const long long k0 = 32LL * (kb0 + blk), left = c.K - k0;
      if (left <= 0) continue;
      const u32x4 w0 = *reinterpret_cast<const u32x4 *>(tile + (2 * lane) * kColPitch + 16 * blk);
      const u32x4 w1 =
          *reinterpret_cast<const u32x4 *>(tile + (2 * lane + 1) * kColPitch + 16 * blk);
      const uint32_t s0 = sc[(2 * lane) * kColBlocks + blk];
      const uint32_t s1 = sc[(2 * lane + 1) * kColBlocks + blk];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float a[8], d[8];
        decode8(w0[q], s0, a);
        decode8(w1[q], s1, d);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (8 * q + j < left)
            store2<FMT>(c.y, (k0 + 8 * q + j) * c.ldx + r0 + 2 * lane,
                        ncol - 2 * lane, a[j], d[j]);
      }
    }
    __syncthreads();
  }
}

// Grid of the kernels along rows: groups of 128 values by rows.
dim3 rows_grid(long long groups, int rows, int &lg) {
  lg = 0;
  while (lg < 4 && (1LL << lg) < groups) ++lg;
  const long long gy = ceil_div(rows, 16 >> lg);
  return dim3((unsigned)ceil_div(groups, 1LL << lg), (unsigned)(gy < kMaxGridY ? gy : kMaxGridY));
}
dim3 cols_grid(long long ktiles, int rows) {
  const long long gx = ceil_div(rows, kColRows), most = (1LL << 30) / gx;  // < 2^31 together
  const long long gy = ktiles < kMaxGridY ? ktiles : kMaxGridY;
  return dim3((unsigned)gx, (unsigned)(gy < most ? gy : most));
}
// The launches of a conversion down columns: two where one would have 2^32
// threads in x.
template <class Kernel>
hipError_t in_cols(Kernel kern, const MxConvert &c, int format, long long ktiles, hipStream_t s) {
  constexpr int kMostCols = 1 << 30;
  for (long long r = 0; r < c.rows; r += kMostCols) {
    MxConvert q = c;
    q.rows = (int)(c.rows - r < kMostCols ? c.rows - r : kMostCols);
    if (c.x) q.x = static_cast<const char *>(c.x) + r * format_bytes(format);
    if (c.y) q.y = static_cast<char *>(c.y) + r * format_bytes(format);
    q.codes += r * c.ld;
    q.scales += r * c.lds;
    const hipError_t e = launch_kernel(kern, cols_grid(ktiles, q.rows), dim3(kThreads), s, q, (int)ktiles);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx_quantize(int format, int along, const MxConvert &c, hipStream_t s) {
  if (along == kAlongRows) {
    const long long groups = mx_scale_bytes(c.K) / 4;  // whole scale rows are written
    auto kern = format == kBf16  ? quant_rows_kernel<kBf16>
                : format == kF16 ? quant_rows_kernel<kF16>
                                 : quant_rows_kernel<kF32>;
    int lg;
    const dim3 grid = rows_grid(groups, c.rows, lg);
    return launch_kernel(kern, grid, dim3(kThreads), s, c, lg, (int)groups);
  }
  auto kern = format == kBf16  ? quant_cols_kernel<kBf16>
              : format == kF16 ? quant_cols_kernel<kF16>
                               : quant_cols_kernel<kF32>;
  const long long ktiles = mx_scale_bytes(c.K) / kColBlocks;  // whole scale rows are written
  return in_cols(kern, c, format, ktiles, s);
}

hipError_t launch_mx_dequantize(int format, int along, const MxConvert &c, hipStream_t s) {
  if (along == kAlongRows) {
    auto kern = format == kBf16  ? dequant_rows_kernel<kBf16>
                : format == kF16 ? dequant_rows_kernel<kF16>
                                 : dequant_rows_kernel<kF32>;
    int lg;
    const long long groups = ceil_div(c.K, kGroup);
    const dim3 grid = rows_grid(groups, c.rows, lg);
    return launch_kernel(kern, grid, dim3(kThreads), s, c, lg, (int)groups);
  }
  auto kern = format == kBf16  ? dequant_cols_kernel<kBf16>
              : format == kF16 ? dequant_cols_kernel<kF16>
                               : dequant_cols_kernel<kF32>;
  const long long ktiles = ceil_div(mx_blocks(c.K), kColBlocks);
  return in_cols(kern, c, format, ktiles, s);
}

}  // namespace gemm_f32_impl
