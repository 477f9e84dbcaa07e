// Products with MX weights: 16-bit activations (gemm_mx_a16), in a form for
// little work and one for much, and the few-row form of gemm_mx.  See
// mx_thin.hpp for the operands.
#include "mx_internal.hpp"
#include "mx_thin.hpp"

namespace gemm_f32_impl {
namespace {

struct ThinProblem {
  int M, N, K;
  const unsigned char *A;
  long long lda;  // bytes
  MxMatrix B;
  void *C;
  long long ldc;
  int c_format;
};

// The launches of a kernel that takes `rows` rows in each grid row: several
// where one cannot have as many grid rows, or columns.
template <class Launch>
hipError_t in_grid_rows(const ThinProblem &all, int rows, Launch launch) {
  return in_columns(all, [&](ThinProblem p) {
    const long long most = (long long)rows * kMaxGridY;
    const int M = p.M;
    const size_t size = p.c_format == kF32 ? 4 : 2;
    for (long long m = 0; m < M; m += most) {
      p.M = (int)(M - m < most ? M - m : most);
      const hipError_t e = launch(p, (unsigned)ceil_div(p.M, rows));
      if (e != hipSuccess) return e;
      p.A += p.M * p.lda;
      p.C = static_cast<char *>(p.C) + (size_t)p.M * p.ldc * size;
    }
    return hipSuccess;
  });
}

// Little work: 16 columns to a workgroup, whose waves share K, 8 / MB to
// each of its blocks of 16 rows, with activations straight from memory.  One
// round of loads and one exchange of sums (eight waves: four took 5.5 us for 24
// x 1024 x 2048, eight 4.6), so the latency of both bounds it:
// 17 x 4095 x 2049 takes 6.0 us with its launch (19 us with each lane
// reading its own rows, the end of K behind guarded loads), 1 x 4096 x 4096
// 4.6 us.
constexpr int kSmallWaves = 8;
template <int A, int MB, int ROWS>
__global__ void __launch_bounds__(64 * kSmallWaves) mx_small_kernel(ThinProblem p) {
  constexpr int kShares = kSmallWaves / MB;
  __shared__ f32x4 part[kSmallWaves][64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = 16 * blockIdx.x, pieces = (int)ceil_div(p.K, 512);
  const long long n = n0 + (lane >> 2) < p.N ? n0 + (lane >> 2) : p.N - 1;
  const Row w{p.B.codes + n * p.B.ld, p.B.scales + n * p.B.lds};
  const long long m0 = 16LL * (MB * blockIdx.y + wave % MB), m = m0 + l16, mr = m0 + (lane >> 2);
  const unsigned char *a = p.A + (mr < p.M ? mr : p.M - 1) * p.lda;
  Direct<A, ROWS> t;
  t.acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int q = wave / MB; q < pieces; q += kShares) t.piece(w, a, q, lane, p.K);
  part[wave][lane] = t.acc;
  __syncthreads();
  if (wave >= MB || m >= p.M) return;
  f32x4 sum = part[wave][lane];
#pragma unroll
  for (int q = 1; q < kShares; ++q) sum += part[q * MB + wave][lane];
  const int col = n0 + 4 * g, left = p.N - col;
  store4_fmt(p.c_format, p.C, m * p.ldc + col, left < 4 ? left : 4, sum);
}

template <int A, int MB, int ROWS>
hipError_t launch_small(const ThinProblem &p, hipStream_t s) {
  return in_grid_rows(p, 16 * MB, [&](const ThinProblem &q, unsigned gy) {
    const dim3 grid((unsigned)ceil_div(q.N, 16), gy);
    return launch_kernel(mx_small_kernel<A, MB, ROWS>, grid, dim3(64 * kSmallWaves), s, q);
  });
}

// Many columns: 16 MB rows by 64 columns to a workgroup.  K is taken 512
// values at a time; of the first eight waves, wave (c, s) multiplies columns
// 32 c .. + 31 with the s-th 128 of them, so that an operand read from LDS
// serves two products and a weight is widened for all rows.  It loads its own
// weights, kAhead chunks ahead.  The other eight waves bring the activations to
// LDS, whose two halves take the chunks in turn, and have asked for the two
// after the one they write.  Waves of their own, because a wave's loads complete
// in order and activations would be waited for behind weights.
//
// 64 x 16384 x 8192 takes 28 us (76 MB, 2.7 TB/s).  What bounds it: a chunk's
// 64 KB of activations cross the L1 (1,024 cycles), are written to LDS and
// read twice (1,500 cycles) next to 1,024 cycles of matrix work.  With lanes
// that each read their own row of weights it took 41 us, with the rows of 32 in
// registers (the thin products' form) 61.
constexpr int kWideWaves = 16, kWideThreads = 64 * kWideWaves, kWideK = 512;
template <int A, int MB, int ROWS>
struct Wide {
  static constexpr int kRows = 16 * MB, kGroup = 16 * kRows + 16;
  static constexpr int kStage = kWideK / 8 * kGroup, kLoads = kRows / 8;
  static constexpr int kAhead = MB == 2 ? 4 : 2;  // even
  // 16 rows of codes and the scales of both blocks of columns, as loaded: four
  // lanes take 64 bytes of a row of codes (lanes that each read their own row
  // cost the L1 four times the accesses), lane l the four scales of column
  // l % 32 of this chunk (l < 32) or the next one.
  struct Weights {
    u32x4 c[2];
  };
  struct Columns {
    const unsigned char *codes[2];  // row l / 4
    const unsigned char *scales;
  };
  typedef Eight<ROWS> Acts[kLoads];

  // The staging lane's 16-byte units: number `lane` of rows r0 + 8 i.  (No
  // load behind a branch, here and below: it would be waited for as if it had
  // not been taken.)
  static __device__ __forceinline__ void load(Acts &v, const unsigned char *const (&row)[kLoads],
                                              long long k0, int lane, int K) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i].load(row[i], k0 + 8 * lane, K);
  }
  // `to`: the place of row r0 in LDS.
  static __device__ __forceinline__ void keep(unsigned char *to, const Acts &v, long long k0,
                                              int lane, int K) {
    const int group = (lane & ~15) | (lane & 3) << 2 | (lane >> 2 & 3);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      u32x4 x = v[i].get();
      if (k0 + kWideK > K) x = v[i].end(x, k0 + 8 * lane, K);  // uniform
      *reinterpret_cast<u32x4 *>(to + group * kGroup + 16 * 8 * i) = x;
    }
  }

  f32x4 acc[MB][2];
  static __device__ __forceinline__ void load(Weights &x, const Columns &w, int kb, int nb) {
    const int in = kb < nb ? kb : nb - 1;
#pragma unroll
    for (int b = 0; b < 2; ++b) x.c[b] = *reinterpret_cast<const u32x4 *>(w.codes[b] + 16LL * in);
  }
  static __device__ __forceinline__ uint32_t load_scales(const Columns &w, int kb, int nb) {
    return *reinterpret_cast<const uint32_t *>(w.scales + ((kb < nb ? kb : nb - 1) & ~3));
  }
  // `at`: the lane's operands of the wave's 128 values.
  template <Widen HOW>
  __device__ __forceinline__ void words(const unsigned char *at, int j, const uint32_t (&c)[2],
                                        const uint32_t (&sb)[2], int down = 0) {
    const u32x4 w0 = widen<HOW>(c[0], sb[0], down), w1 = widen<HOW>(c[1], sb[1], down);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      u32x4 a = *reinterpret_cast<const u32x4 *>(at + 4 * j * kGroup + 256 * i), lo{};
      if constexpr (HOW == kToF16) {
        acc[i][0] = mfma_f16(w0, a, acc[i][0]);
        acc[i][1] = mfma_f16(w1, a, acc[i][1]);
      } else {
        if constexpr (A == kF16) split_f16(a, a, lo);
        acc[i][0] = mfma_bf16(w0, a, acc[i][0]);
        acc[i][1] = mfma_bf16(w1, a, acc[i][1]);
        if constexpr (A == kF16) {
          acc[i][0] = mfma_bf16(w0, lo, acc[i][0]);
          acc[i][1] = mfma_bf16(w1, lo, acc[i][1]);
        }
      }
    }
  }
  // `kb`: the lane's block, number l / 16 of the wave's; `half`: of the lanes
  // that hold the chunk's scales.
  __device__ __forceinline__ void use(const Weights &x, uint32_t scales, int half,
                                      const unsigned char *at, int lane, int kb, int nb) {
    const int from = loader(lane);
    bool ok = true;
    uint32_t sb[2], c[4][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t s = from_lane(scales, 32 * half + 16 * b + (lane & 15));
      sb[b] = kb < nb ? s >> (8 * (lane >> 4)) & 255u : 127u;
      uint32_t any = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = from_lane(x.c[b][j], from);
        c[j][b] = kb < nb ? v : 0u;
        any |= c[j][b];
      }
      ok &= widens_fast<A>(sb[b], any);
    }
    if (__all(ok)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) words<A == kF16 ? kToF16 : kToBf16>(at, j, c[j], sb);
    } else {  // rare, and kept short
      const Quartered quarter(top_scale(sb[0]) | top_scale(sb[1]));
#pragma unroll
      for (int i = 0; i < MB; ++i) quarter.before(acc[i][0]), quarter.before(acc[i][1]);
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const uint32_t d[2] = {j < 2 ? (j ? c[1][0] : c[0][0]) : j == 2 ? c[2][0] : c[3][0],
                               j < 2 ? (j ? c[1][1] : c[0][1]) : j == 2 ? c[2][1] : c[3][1]};
        words<kThroughF32>(at, j, d, sb, quarter.down);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) quarter.after(acc[i][0]), quarter.after(acc[i][1]);
    }
  }
};

template <int A, int MB, int ROWS>
__global__ void __launch_bounds__(kWideThreads) mx_wide_kernel(ThinProblem p) {
  typedef Wide<A, MB, ROWS> Product;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];  // two stages
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int l16 = lane & 15, g = lane >> 4, nb = (int)mx_blocks(p.K);
  // All waves take whole rounds of turns (a way out between would let the
  // compiler wait for the newest loads at the top), the last ones perhaps idle.
  const int chunks = (int)ceil_div(p.K, kWideK);
  const int turns = (int)ceil_div(chunks, Product::kAhead) * Product::kAhead;
  const long long m0 = (long long)Product::kRows * blockIdx.y;
  f32x4 *part = reinterpret_cast<f32x4 *>(lds);
  if (wave >= 8) {
    const unsigned char *row[Product::kLoads];
#pragma unroll
    for (int i = 0; i < Product::kLoads; ++i) {
      const long long m = m0 + (wave - 8) + 8 * i;
      row[i] = p.A + (m < p.M ? m : p.M - 1) * p.lda;
    }
    unsigned char *to = lds + 16 * (wave - 8);
    typename Product::Acts v[2];
    Product::load(v[0], row, 0, lane, p.K);
    __builtin_amdgcn_sched_barrier(0);  // loads in order of use, or the loop's first wait is for all
    Product::load(v[1], row, kWideK, lane, p.K);
    // Turn c: chunk c goes to LDS, where chunk c - 1 is in use.
#pragma unroll 1
    for (int c = 0; c < turns; c += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int now = c + u;
        if (now < chunks)
          Product::keep(to + u * Product::kStage, v[u], (long long)now * kWideK, lane, p.K);
        Product::load(v[u], row, (now + 2LL) * kWideK, lane, p.K);
        __syncthreads();
      }
    }
    __syncthreads();  // the last chunk's products
    __syncthreads();  // the sums
    return;
  }
  const int pair = wave >> 2, share = wave & 3;
  const long long n0 = 64LL * blockIdx.x + 32 * pair;
  typename Product::Columns w;
  auto column = [&](long long n) { return n < p.N ? n : p.N - 1; };
#pragma unroll
  for (int b = 0; b < 2; ++b) w.codes[b] = p.B.codes + column(n0 + 16 * b + (lane >> 2)) * p.B.ld;
  w.scales = p.B.scales + column(n0 + (lane & 31)) * p.B.lds;
  Product t;
#pragma unroll
  for (int i = 0; i < MB; ++i) t.acc[i][0] = t.acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  typename Product::Weights x[Product::kAhead];
  uint32_t sc[Product::kAhead / 2];
  // The first chunk's blocks: the lane's in use, in loading codes and scales.
  const int kb = 4 * share + g, kc = 4 * share + (lane & 3), ks = 4 * share + 16 * (lane >> 5);
#pragma unroll
  for (int u = 0; u < Product::kAhead; ++u) {
    if (u % 2 == 0) sc[u / 2] = Product::load_scales(w, ks + 16 * u, nb);
    Product::load(x[u], w, kc + 16 * u, nb);
    __builtin_amdgcn_sched_barrier(0);  // loads in order of use, or the loop's first wait is for all
  }
#pragma unroll 1
  for (int c = 0; c < turns; c += Product::kAhead) {
#pragma unroll
    for (int u = 0; u < Product::kAhead; ++u) {
      const int now = c + u;
      __syncthreads();  // chunk `now` is in LDS
      if (now < chunks)
        t.use(x[u], sc[u / 2], u & 1,
              lds + (u & 1) * Product::kStage + (16 * share + g) * Product::kGroup + 16 * l16, lane,
              kb + 16 * now, nb);
      if (u % 2 == 1) sc[u / 2] = Product::load_scales(w, ks + 16 * (now - 1 + Product::kAhead), nb);
      Product::load(x[u], w, kc + 16 * (now + Product::kAhead), nb);
    }
  }
  __syncthreads();
  // The shares' sums, added in their order.
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b) part[((2 * i + b) * 8 + wave) * 64 + lane] = t.acc[i][b];
  __syncthreads();
#pragma unroll
  for (int o = 0; o < MB / 2; ++o) {
    const int i = (4 * o + share) >> 1, b = share & 1;
    const f32x4 *from = part + ((2 * i + b) * 8 + 4 * pair) * 64 + lane;
    const f32x4 sum = from[0] + from[64] + from[128] + from[192];
    const long long m = m0 + 16 * i + l16, col = n0 + 16 * b + 4 * g, left = p.N - col;
    if (m < p.M) store4_fmt(p.c_format, p.C, m * p.ldc + col, (int)(left < 4 ? left : 4), sum);
  }
}

template <int A, int MB, int ROWS>
hipError_t launch_wide(const ThinProblem &p, hipStream_t s) {
  return in_grid_rows(p, 16 * MB, [&](ThinProblem q, unsigned gy) {
    void *args[] = {&q};
    return hipLaunchKernel(reinterpret_cast<const void *>(mx_wide_kernel<A, MB, ROWS>),
                           dim3((unsigned)ceil_div(q.N, 64), gy), dim3(kWideThreads), args,
                           2 * Wide<A, MB, ROWS>::kStage, s);
  });
}

// The wide kernel from about 96 workgroups on (192 for up to 16 rows, most of
// whose products it would do for nothing), where K is long enough to pay for
// its start.  Small and wide, us: 64 x 4096 x 8192 25.0 and 26.7, 64 x 6144 x
// 8192 35.9 and 27.7, 64 x 8192 x 512 5.0 and 6.1, x 1024 7.7 and 7.4, 16 x 8192
// x 8192 16.3 and 17.6, 16 x 16384 x 8192 28.3 and 20.4.
template <int A, int ROWS>
hipError_t launch_a16(const ThinProblem &p, hipStream_t s) {
  const long long groups = ceil_div(p.N, 64) * ceil_div(p.M, 64);
  const bool wide = groups >= (p.M <= 16 ? 192 : 96) && p.K >= 8 &&
                    ceil_div(p.N, 16) * ceil_div(p.M, 32) * p.K >= 1 << 20;
  if (wide) return p.M <= 32 ? launch_wide<A, 2, ROWS>(p, s) : launch_wide<A, 4, ROWS>(p, s);
  return p.M <= 16 ? launch_small<A, 1, ROWS>(p, s) : launch_small<A, 2, ROWS>(p, s);
}

// ---- few rows of MX by MX ------------------------------------------------------
// Both operands as they are stored.  Four lanes that read four rows cost the
// L1 four accesses, four that read 64 bytes of one row one; so lane l loads
// 16 bytes number l % 4 (of group l / 16) of rows 4 (l / 4 % 4) + t, t = 0 ..
// 3, and a 4 x 4 transpose inside each four lanes brings row l % 16's four
// blocks into the lane: 32 x 4096 x 16384 took 16.5 us with the lanes' own
// rows.  A lane then holds blocks 4 g + s of a piece's 16 (g = l / 16) and
// their scales as the bytes of a word, which the matrix instruction picks.

// Lane i's r[t] goes to lane t's r[i], in each four lanes.
__device__ __forceinline__ void quad_transpose(u32x4 (&r)[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
#pragma unroll
    for (int t = 0; t < 4; t += 2) {
      const uint32_t a = r[t][d], b = r[t + 1][d], fa = quad<0xB1>(a), fb = quad<0xB1>(b);
      r[t][d] = odd ? fb : a;
      r[t + 1][d] = odd ? b : fa;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t a = r[t][d], b = r[t + 2][d], fa = quad<0x4E>(a), fb = quad<0x4E>(b);
      r[t][d] = high ? fb : a;
      r[t + 2][d] = high ? b : fa;
    }
  }
}

// 16 rows of an MX matrix from row r0 on (past the last: the last), a piece of
// 16 blocks at a time.
struct FewRows {
  const unsigned char *p[4], *q;
  __device__ __forceinline__ void at(const MxMatrix &m, long long r0, long long rows, int lane) {
    auto row = [&](int r) { return r0 + r < rows ? r0 + r : rows - 1; };
#pragma unroll
    for (int t = 0; t < 4; ++t) p[t] = m.codes + row((lane & 12) + t) * m.ld;
    q = m.scales + row(lane & 15) * m.lds;
  }
};
struct FewPiece {
  u32x4 c[4];
  uint32_t s;
  __device__ __forceinline__ void load(const FewRows &r, int piece, int lane, int nb) {
    const int kb = 16 * piece + 4 * (lane >> 4) + (lane & 3), in = kb < nb ? kb : nb - 1;
    s = *reinterpret_cast<const uint32_t *>(r.q + 16LL * piece + 4 * (lane >> 4));
#pragma unroll
    for (int t = 0; t < 4; ++t) c[t] = *reinterpret_cast<const u32x4 *>(r.p[t] + 16LL * in);
  }
  // The lane's own row; blocks past the row's become zeros with scale 1.
  __device__ __forceinline__ void turn(int piece, int lane, int nb) {
    quad_transpose(c, lane);
    if (16 * (piece + 1) > nb) {  // uniform
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * piece + 4 * (lane >> 4) + i >= nb) {
          c[i] = u32x4{0, 0, 0, 0};
          s = (s & ~(255u << (8 * i))) | 127u << (8 * i);
        }
    }
  }
};

// Four waves, so that two workgroups share a compute unit: 32 x 8192 x 4096 8.8
// us, with eight 11.0; 32 x 4096 x 16384 12.3 and 13.5.
constexpr int kFewWaves = 4;
template <int MB>
__global__ void __launch_bounds__(64 * kFewWaves) mx_few_kernel(MxProblem p) {
  constexpr int WAVES = kFewWaves;
  __shared__ f32x4 part[WAVES][MB][64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int l16 = lane & 15, g = lane >> 4, nb = (int)mx_blocks(p.K);
  const long long n0 = 16LL * blockIdx.x;
  FewRows w, a[MB];
  w.at(p.B, n0, p.N, lane);
  const int pieces = (nb + 15) / 16;
  for (long long m0 = 16LL * MB * blockIdx.y; m0 < p.M; m0 += 16LL * MB * gridDim.y) {
    f32x4 acc[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      a[i].at(p.A, m0 + 16 * i, p.M, lane);
      acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    FewPiece x, y[MB];
    if (wave < pieces) {
      x.load(w, wave, lane, nb);
#pragma unroll
      for (int i = 0; i < MB; ++i) y[i].load(a[i], wave, lane, nb);
    }
#pragma unroll 1
    for (int q = wave; q < pieces; q += WAVES) {
      FewPiece xn, yn[MB];
      const int next = q + WAVES < pieces ? q + WAVES : q;
      xn.load(w, next, lane, nb);
#pragma unroll
      for (int i = 0; i < MB; ++i) yn[i].load(a[i], next, lane, nb);
      x.turn(q, lane, nb);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        y[i].turn(q, lane, nb);
        acc[i] = mfma_mx<0>(x.c[0], (int)x.s, y[i].c[0], (int)y[i].s, acc[i]);
        acc[i] = mfma_mx<1>(x.c[1], (int)x.s, y[i].c[1], (int)y[i].s, acc[i]);
        acc[i] = mfma_mx<2>(x.c[2], (int)x.s, y[i].c[2], (int)y[i].s, acc[i]);
        acc[i] = mfma_mx<3>(x.c[3], (int)x.s, y[i].c[3], (int)y[i].s, acc[i]);
      }
      x = xn;
#pragma unroll
      for (int i = 0; i < MB; ++i) y[i] = yn[i];
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < MB; i += WAVES) {
      f32x4 sum = part[0][i][lane];
#pragma unroll
      for (int q = 1; q < WAVES; ++q) sum += part[q][i][lane];
      const long long m = m0 + 16 * i + l16, col = n0 + 4 * g, left = p.N - col;
      if (m < p.M) store4_fmt(p.c_format, p.C, m * p.ldc + col, (int)(left < 4 ? left : 4), sum);
    }
    __syncthreads();
  }
}

template <int MB>
hipError_t launch_few(const MxProblem &p, hipStream_t s) {
  return in_columns(p, [&](const MxProblem &q) {
    const long long gy = ceil_div(q.M, 16 * MB);
    const dim3 grid((unsigned)ceil_div(q.N, 16), (unsigned)(gy < kMaxGridY ? gy : kMaxGridY));
    return launch_kernel(mx_few_kernel<MB>, grid, dim3(64 * kFewWaves), s, q);
  });
}

// Rows that start in the middle of a word, of a matrix that starts on one.
bool odd_rows(const void *base, long long pitch_bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 3) == 0 && (pitch_bytes & 3) != 0;
}

}  // namespace

hipError_t launch_mx_a16(const MxA16Problem &p, hipStream_t s) {
  const ThinProblem t{p.M, p.N, p.K, reinterpret_cast<const unsigned char *>(p.A), 2 * p.lda,
                      p.B, p.C, p.ldc, p.c_format};
  if (odd_rows(p.A, 2 * p.lda) && p.M > 1)
    return p.a_format == kBf16 ? launch_a16<kBf16, kOdd>(t, s) : launch_a16<kF16, kOdd>(t, s);
  return p.a_format == kBf16 ? launch_a16<kBf16, kWords>(t, s) : launch_a16<kF16, kWords>(t, s);
}

hipError_t launch_mx_thin(const MxProblem &p, hipStream_t s) {
  return p.M <= 16 ? launch_few<1>(p, s) : launch_few<2>(p, s);
}

}  // namespace gemm_f32_impl
