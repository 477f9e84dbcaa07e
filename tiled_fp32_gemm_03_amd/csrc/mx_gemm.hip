// The product of two MX matrices (gemm_mx.h), on
// v_mfma_scale_f32_16x16x128_f8f6f4: a lane's operand is one block of 32
// codes, 16 bytes, with its scale byte, so both operands are read in the
// layout they are stored in and a block is never taken apart.
#include "mx_internal.hpp"
#include "mx_values.hpp"
#include "addr_math.hpp"
#include "addr_math16.hpp"
#include "buffer_lds.hpp"
#include "w16_tiles.hpp"


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

// ---- direct-load tiles ----------------------------------------------------
//
// A tile of 2 WT x 2 WT over 4 waves (2 x 2), each WT x WT as 16 x 16
// blocks; steps of 256 k (8 blocks, 128 bytes of each row) in two LDS
// stages.  Both operands are stored alike, so both are loaded alike: rows of
// 8 chunks of 16 bytes straight into LDS (chunk c of row r at m16_a_pos), and
// an operand of a 128-deep group is one 16-byte read.  Scales come by
// 16-byte chunks too, a row's 16 scales of two steps, double-buffered on
// their own; a lane reads the byte of its block.
//
// The loads are buffer loads: in a partial last step (TAIL) a lane whose
// block lies past the row's blocks takes an offset past the buffer's record
// count and gets zeros.  Scale bytes past the last block may hold anything,
// 255 among it: with TAIL they are replaced by 127 before use.  The offsets
// of a tile are 32-bit from its first row (the launcher checks the pitch).
// C is at least one tile each way; edge tiles are moved back inside it.
//
// 8192 cubed takes 279 to 289 us (3.8 to 3.9 PFLOP/s, 2.2 us a step; 4096 cubed
// with fp32 C 40 us, of which about 5 are its launch, first loads and stores).  The
// matrix unit is busy 0.38 of the time at 2.2 GHz.  Timing copies: without the
// direct loads 253 us, without the operand reads 296, without both 217.  Measured
// and not kept: the 32x32x64 instruction (308 us), the next step's first operands
// read before the barrier (316), non-temporal stores (319), eight waves of 128 x 64
// (287; a fifth fewer cycles at a lower clock, and 4096 cubed slower).  Odd sizes
// with 16-bit C cost more than their steps: 4097 x 4095 x 2049 takes 40 us before
// its last row, 20 of them its 9 steps (its stores are 32 bytes to a row and
// instruction at 2-byte alignment, and these forms spill 3 to 5 registers).

template <int WT_>
struct MxTile {
  static constexpr int WT = WT_, BM = 2 * WT_, TB = WT_ / 16;
  static constexpr int KB = 8;                      // blocks per step
  static constexpr int KG = KB / 4;                 // 128-deep groups per step
  static constexpr int CODES = BM * 16 * KB;        // bytes of one operand's step
  static constexpr int STAGE = 2 * CODES;
  static constexpr int SCALES = BM * 16;            // bytes of one operand's two steps
  static constexpr int DMA = CODES / 1024 / 4;      // code loads per wave, operand and step
  static constexpr int SROWS = BM / 64;             // scale loads per operand
  static constexpr int LDS = 2 * STAGE + 2 * 2 * SCALES;
  static_assert(LDS <= kLdsBytes, "LDS budget");
  static_assert(SROWS == 4 || SROWS == 2, "one wave takes at most one scale load per operand");
};

// One operand of a tile: buffers from the tile's first row.
struct MxSide {
  rsrc_t codes, scales;
};
__device__ inline MxSide mx_side(const MxMatrix &m, int row0, int rows, int nb, int scale_bytes) {
  MxSide s;
  s.codes = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<unsigned char *>(m.codes + (long long)row0 * m.ld), 0,
      (int)((rows - 1) * m.ld + 16LL * nb), 0x00020000);
  s.scales = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<unsigned char *>(m.scales + (long long)row0 * m.lds), 0,
      (int)((rows - 1) * m.lds + scale_bytes), 0x00020000);
  return s;
}

template <int WT, bool TAIL, int CF>
__global__ void __launch_bounds__(256) mx_tile_kernel(MxProblem p, int tiles_m, int tiles_n) {
  using W = MxTile<WT>;
  constexpr int TB = W::TB;
  __shared__ __attribute__((aligned(16))) char lds[W::LDS];
  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t *)lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, g = lane >> 4;
  const int ntiles = tiles_m * tiles_n;
  const int nb = (int)mx_blocks(p.K), nk = (nb + W::KB - 1) / W::KB;
  const int scale_bytes = (int)mx_scale_bytes(p.K);
  const int G = gridDim.x;
  const int lid = xcd_remap(blockIdx.x, G);
  if (lid >= ntiles) return;  // uniform per workgroup
  const int my_tiles = (ntiles - lid + G - 1) / G;

  // Load q of a wave fills rows 8 (DMA wave + q) .. + 7: a lane's row moves by
  // 16 for every second q and its chunk (m16_a_pos undone) flips by 4 between
  // even and odd q, so two offsets and a scalar serve all.
  const int c0 = (lane & 7) ^ (lane >> 4);
  int va[2], vb[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * (W::DMA * wave + h) + (lane >> 3);
    va[h] = (int)(r * p.A.ld) + 16 * (c0 ^ (4 * h));
    vb[h] = (int)(r * p.B.ld) + 16 * (c0 ^ (4 * h));
  }
  const int vsa = (int)((64 * wave + lane) * p.A.lds), vsb = (int)((64 * wave + lane) * p.B.lds);
  // Byte places of a lane's first operand row and scales in a stage.
  const int ra128 = 128 * (wm * WT + l16), rb128 = W::CODES + 128 * (wn * WT + l16);
  const int sa16 = 16 * (wm * WT + l16) + g, sb16 = W::SCALES + 16 * (wn * WT + l16) + g;
  const int a16 = (int)(16 * p.A.ld), b16 = (int)(16 * p.B.ld);

  auto origin = [&](int t, int &m0, int &n0) __attribute__((always_inline)) {
    edge_tile_origin(lid + t * G, tiles_m, tiles_n, W::BM, W::BM, p.M, p.N, m0, n0);
  };
  // Code loads q0 .. q1 - 1 of step kk (A's DMA first, then B's).
  auto issue = [&](unsigned st, const MxSide &a, const MxSide &b, int kk, int q0, int q1)
      __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 2 * W::DMA; ++q) {
      if (q < q0 || q >= q1) continue;
      const int i = q % W::DMA, h = i & 1;
      int v = q < W::DMA ? va[h] : vb[h];
      if constexpr (TAIL) v = W::KB * kk + (c0 ^ (4 * h)) < nb ? v : kOutside;
      const unsigned to = st + (q < W::DMA ? 0 : W::CODES) + (W::DMA * wave + i) * 1024;
      const int soff = 16 * W::KB * kk + (i >> 1) * (q < W::DMA ? a16 : b16);
      buffer_load_to_lds16(v, q < W::DMA ? a.codes : b.codes, soff, to);
    }
  };
  auto issue_scales = [&](int buf, const MxSide &a, const MxSide &b, int kk)
      __attribute__((always_inline)) {
    if (W::SROWS == 4 || wave < W::SROWS) {
      const unsigned to = lds_u + 2 * W::STAGE + buf * 2 * W::SCALES + wave * 1024;
      buffer_load_to_lds16(vsa, a.scales, 8 * kk, to);
      buffer_load_to_lds16(vsb, b.scales, 8 * kk, to + W::SCALES);
    }
  };

  int m0, n0;
  origin(0, m0, n0);
  MxSide sa = mx_side(p.A, m0, W::BM, nb, scale_bytes);
  MxSide sb = mx_side(p.B, n0, W::BM, nb, scale_bytes);
  int stage = 0, sbuf = 0;
  issue(lds_u, sa, sb, 0, 0, 2 * W::DMA);
  issue_scales(0, sa, sb, 0);

  f32x4 acc[TB][TB];
  for (int t = 0; t < my_tiles; ++t) {
    int nm0, nn0;
    origin(t + 1 < my_tiles ? t + 1 : t, nm0, nn0);  // the last step reloads its own tile's first
    const MxSide na = mx_side(p.A, nm0, W::BM, nb, scale_bytes);
    const MxSide nbs = mx_side(p.B, nn0, W::BM, nb, scale_bytes);
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int kk = 0; kk < nk; ++kk) {
      const bool last = kk + 1 == nk;
      const MxSide &ia = last ? na : sa, &ib = last ? nbs : sb;
      const int ik = last ? 0 : kk + 1;
      __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(0));  // this step's loads (own)
      ks_lds_barrier();                                // everyone's; the other stage free
      const char *st = lds + stage * W::STAGE;
      const unsigned nst = lds_u + (stage ^ 1) * W::STAGE;
      const char *sc = lds + 2 * W::STAGE + sbuf * 2 * W::SCALES + 8 * (kk & 1);
      const bool new_scales = (ik & 1) == 0;
      if (new_scales) issue_scales(sbuf ^ 1, ia, ib, ik);

      u32x4 fa[2][TB], fb[2][TB];
      int xa[2][TB], xb[2][TB];
      auto read = [&](int kg) __attribute__((always_inline)) {
        const int z = kg & 1;
        // m16_a_pos(r, c) of rows 16 i + l16: the permutation is the same for
        // every i, so blocks lie a constant apart.
        const char *pa = st + ra128 + 16 * ((4 * kg + g) ^ (l16 >> 1));
        const char *pb = st + rb128 + 16 * ((4 * kg + g) ^ (l16 >> 1));
#pragma unroll
        for (int i = 0; i < TB; ++i) {
          fb[z][i] = *reinterpret_cast<const u32x4 *>(pb + 2048 * i);
          xb[z][i] = *reinterpret_cast<const unsigned char *>(sc + sb16 + 256 * i + 4 * kg);
          fa[z][i] = *reinterpret_cast<const u32x4 *>(pa + 2048 * i);
          xa[z][i] = *reinterpret_cast<const unsigned char *>(sc + sa16 + 256 * i + 4 * kg);
        }
        if constexpr (TAIL) {
          const bool in = W::KB * kk + 4 * kg + g < nb;
#pragma unroll
          for (int i = 0; i < TB; ++i) {
            xa[z][i] = in ? xa[z][i] : 127;
            xb[z][i] = in ? xb[z][i] : 127;
          }
        }
      };
      read(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kg = 0; kg < W::KG; ++kg) {
        const int z = kg & 1;
#pragma unroll
        for (int i = 0; i < TB; ++i) {
#pragma unroll
          for (int j = 0; j < TB; ++j)
            acc[i][j] = mfma_mx(fb[z][j], xb[z][j], fa[z][i], xa[z][i], acc[i][j]);
          constexpr int kPerRow = 2;  // 8192 cubed: 289 us, one by one 302, four 309
          const int row = kg * TB + i;
          if (row * kPerRow < 2 * W::DMA) {
            __builtin_amdgcn_sched_barrier(0);
            issue(nst, ia, ib, ik, row * kPerRow, (row + 1) * kPerRow);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (kg + 1 < W::KG && i == TB / 2 - 1) {
            __builtin_amdgcn_sched_barrier(0);
            read(kg + 1);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      stage ^= 1;
      if (new_scales) sbuf ^= 1;
#pragma unroll
      for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) asm volatile("" : "+a"(acc[i][j]));
    }

    const int n = n0 + wn * WT + 4 * g;
#pragma unroll
    for (int i = 0; i < TB; ++i) {
      const long long at = (long long)(m0 + wm * WT + 16 * i + l16) * p.ldc + n;
#pragma unroll
      for (int j = 0; j < TB; ++j) store4<CF>(p.C, at + 16 * j, 4, acc[i][j]);
    }
    m0 = nm0;
    n0 = nn0;
    sa = na;
    sb = nbs;
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(0));  // the redundant last reload
}

template <int WT>
bool mx_tile_fits(const MxProblem &p) {
  auto fits = [](const MxMatrix &m) {
    const long long pitch = m.ld > m.lds ? m.ld : m.lds;
    return 2 * WT * pitch < (1LL << 31);
  };
  return p.M >= 2 * WT && p.N >= 2 * WT && fits(p.A) && fits(p.B);
}

template <int WT, bool TAIL, int CF>
hipError_t launch_mx_tile(const MxProblem &p, hipStream_t s) {
  constexpr auto kern = mx_tile_kernel<WT, TAIL, CF>;
  const long long tm = ceil_div(p.M, 2 * WT), tn = ceil_div(p.N, 2 * WT), ntiles = tm * tn;
  if (ntiles > 0x7fffffffLL) return hipErrorInvalidValue;
  long long grid = resident_workgroups<kern, 256>();
  if (grid > ntiles) grid = ntiles;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(256), s, p, (int)tm, (int)tn);
}
template <int WT>
hipError_t launch_mx_tiles(const MxProblem &p, hipStream_t s) {
  const bool tail = mx_blocks(p.K) % MxTile<WT>::KB != 0;
  switch (p.c_format) {
    case kF32: return tail ? launch_mx_tile<WT, true, kF32>(p, s) : launch_mx_tile<WT, false, kF32>(p, s);
    case kBf16: return tail ? launch_mx_tile<WT, true, kBf16>(p, s) : launch_mx_tile<WT, false, kBf16>(p, s);
    default: return tail ? launch_mx_tile<WT, true, kF16>(p, s) : launch_mx_tile<WT, false, kF16>(p, s);
  }
}

// Entry 0, in launches of at most 2^23 tiles (a grid has fewer than 2^32
// threads): columns 2^26 at a time, then as many rows as those leave.
hipError_t launch_mx_direct(const MxProblem &p, hipStream_t s) {
  return in_columns(p, [&](const MxProblem &part) {
    const long long tiles_n = ceil_div(part.N, 64), most = 64 * ((1LL << 23) / tiles_n);
    const long long size = format_bytes(p.c_format);
    for (long long m = 0; m < p.M; m += most) {
      MxProblem q = part;
      q.M = (int)(p.M - m < most ? p.M - m : most);
      q.A.codes += m * p.A.ld;
      q.A.scales += m * p.A.lds;
      q.C = static_cast<char *>(part.C) + m * p.ldc * size;
      const long long tiles_m = ceil_div(q.M, 64);
      const hipError_t e = launch_kernel(mx_direct_kernel, dim3((unsigned)(tiles_m * tiles_n)),
                                         dim3(256), s, q, (int)tiles_m, (int)tiles_n);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
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
  if (entry == 3) return launch_mx_thin(p, s);
  if (entry == 1 && mx_tile_fits<128>(p)) {
    // A few rows past whole tiles would cost every column of tiles one more:
    // where that is another round of tiles, the few-row form takes them.
    const int rest = p.M % 256;
    const long long tn = ceil_div(p.N, 256), rounds = ceil_div(ceil_div(p.M, 256) * tn, 256);
    if (rest != 0 && rest <= 32 && ceil_div(p.M / 256 * tn, 256) < rounds) {
      MxProblem q = p;
      q.M -= rest;
      const hipError_t e = launch_mx_tiles<128>(q, s);
      if (e != hipSuccess) return e;
      const size_t size = p.c_format == kF32 ? 4 : 2;
      q.A.codes += q.M * p.A.ld;
      q.A.scales += q.M * p.A.lds;
      q.C = static_cast<char *>(p.C) + q.M * p.ldc * size;
      q.M = rest;
      return launch_mx_thin(q, s);
    }
    return launch_mx_tiles<128>(p, s);
  }
  if (entry == 2 && mx_tile_fits<64>(p)) return launch_mx_tiles<64>(p, s);
  return launch_mx_direct(p, s);
}

}  // namespace gemm_f32_impl
