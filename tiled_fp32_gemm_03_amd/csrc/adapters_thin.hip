// A shared projection with low-rank adapters for up to 64 rows (gemm_adapters.h):
// single tokens of many requests.  Two launches: scale A[r] x by a workgroup to each
// adapter that is asked and 16 of its ranks, and the projection, which reads W once,
// straight into the matrix instructions' operands (mx_thin.hpp), and the asked
// adapters' B.
#include "experts_tiles.hpp"

namespace gemm_f32_impl {
namespace {

template <class T>
__device__ inline T *ws_at(const AdaptersProblem &p, long long off) {
  return reinterpret_cast<T *>(p.ws + off);
}
__device__ inline const unsigned char *bytes_of(const uint16_t *p) {
  return reinterpret_cast<const unsigned char *>(p);
}
template <int FMT>
__device__ inline f32x4 mfma_16(u32x4 b, u32x4 a, f32x4 acc) {
  if constexpr (FMT == kBf16) return mfma_bf16(b, a, acc);
  else return mfma_f16(b, a, acc);
}
// The adapter of row i, or -1.
__device__ inline int adapter_of(const AdaptersProblem &p, int i) {
  const int e = i < p.T ? p.ids[i] : -1;
  return e >= 0 && e < p.count ? e : -1;
}

// ---- v = scale A[r] x -----------------------------------------------------------------
// Workgroup (i, b): ranks 16 b .. + 15 of row i's adapter, if i is its first row, for
// all its rows, 16 at a time.  The waves take the pieces of K in turn; their sums
// are added in wave order.
constexpr int kLowWaves = 8;
template <int FMT, int ROWS>
__global__ void __launch_bounds__(64 * kLowWaves) adapters_low_thin_kernel(AdaptersProblem p) {
  __shared__ f32x4 part[kLowWaves][64];
  __shared__ int rows[64];
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g = lane >> 4;
  const int i = blockIdx.x, r0 = 16 * blockIdx.y;
  const int id = adapter_of(p, lane), e = __builtin_amdgcn_readlane(id, i);
  if (e < 0) return;  // uniform
  const unsigned long long same = __ballot(id == e);
  if (__builtin_ctzll(same) != i) return;
  const int n = __popcll(same);
  if (wave == 0 && id == e) rows[__popcll(same & ((1ULL << lane) - 1))] = lane;
  __syncthreads();
  const int rank = r0 + (lane >> 2) < p.R ? r0 + (lane >> 2) : p.R - 1;
  const unsigned char *a = bytes_of(p.A + ((long long)p.R * e + rank) * p.lda);
  const int pieces = (int)ceil_div(p.K, 128);
  const float scale = p.scales ? p.scales[e] : 1.f;
  for (int m0 = 0; m0 < n; m0 += 16) {
    const int mine = m0 + (lane >> 2);
    const unsigned char *x = bytes_of(p.X + rows[mine < n ? mine : n - 1] * p.ldx);
    f32x4 acc{0, 0, 0, 0};
    HalfPiece<ROWS> wa[2], wx[2];
    auto load = [&](int u, int piece) __attribute__((always_inline)) {
      const int at = piece < pieces ? piece : pieces - 1;
      wa[u].load(a, at, lane, p.K);
      wx[u].load(x, at, lane, p.K);
    };
    load(0, wave);
    load(1, wave + kLowWaves);
#pragma unroll 1
    for (int q = wave; q < pieces; q += 2 * kLowWaves) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int piece = q + u * kLowWaves;
        if (piece < pieces) {  // uniform
          if (piece >= p.K / 128) {
            wa[u].end(a, piece, lane, p.K);
            wx[u].end(x, piece, lane, p.K);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc = mfma_16<FMT>(from_lane(wa[u].get(j, lane), loader(lane)),
                               from_lane(wx[u].get(j, lane), loader(lane)), acc);
        }
        load(u, piece + 2 * kLowWaves);
      }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      for (int w = 1; w < kLowWaves; ++w) acc += part[w][lane];
      acc *= scale;
#pragma unroll
      for (int c = 0; c < 4; ++c)  // zeros from R on
        if (r0 + 4 * g + c >= p.R) acc[c] = 0.f;
      if (m0 + l16 < n)
        *reinterpret_cast<u32x2 *>(ws_at<uint16_t>(p, p.at.v) + rows[m0 + l16] * p.at.rpitch + r0 +
                                   4 * g) =
            u32x2{pack2<FMT>(acc[0], acc[1]), pack2<FMT>(acc[2], acc[3])};
    }
    __syncthreads();
  }
}

// ---- the projection ----------------------------------------------------------------------
// Both kernels: RB blocks of 16 rows, in the order of their adapters, by blocks of 16
// columns; `ks` waves share a block of columns, taking the steps of K in turn.

// The rows in the order of their adapters, those without one first, and the adapters.
__device__ inline void order_rows(const AdaptersProblem &p, int (&order)[64], int (&ids)[64]) {
  if (wave_id() != 0) return;
  const int lane = threadIdx.x & 63, id = adapter_of(p, lane);
  int at = 0;
  for (int i = 0; i < p.T; ++i) {
    const int o = __builtin_amdgcn_readlane(id, i);
    at += o < id || (o == id && i < lane);
  }
  if (lane < p.T) order[at] = lane, ids[at] = id;
  else order[lane] = 0, ids[lane] = -1;
}

// Adds B[r] v, four of a block's adapters at a time, whose B is asked for together; the
// waves that share columns take them in turn.  Each sum is kept by its own rows alone:
// an infinity in one request's B is none of the others'.
template <int FMT, int RB>
__device__ __forceinline__ void add_adapters(const AdaptersProblem &p, const int (&order)[64],
                                             const int (&ids)[64], int columns, int ks, int first,
                                             f32x4 (&acc)[RB]) {
  constexpr int kBatch = 4;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int n = columns + l16 < p.N ? columns + l16 : p.N - 1;
  const unsigned char *m = bytes_of(p.B + (long long)n * p.ldb);
  const long long each = 2LL * p.N * p.ldb;  // bytes of an adapter's B
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int id = ids[16 * b + l16];
    const uint16_t *v = ws_at<uint16_t>(p, p.at.v) + order[16 * b + l16] * p.at.rpitch;
    const unsigned any = (unsigned)__ballot(id >= 0) & 0xffffu;
    if (any == 0) continue;  // uniform
#pragma unroll 1
    for (int r0 = 0; r0 < p.R; r0 += 64) {
      const bool two = r0 + 32 < p.R;  // uniform
      u32x4 xv[2] = {};
      if (id >= 0) {
        xv[0] = *reinterpret_cast<const u32x4 *>(v + r0 + 8 * g);
        if (two) xv[1] = *reinterpret_cast<const u32x4 *>(v + r0 + 32 + 8 * g);
      }
      unsigned left = any;
      int item = 0;
      while (left) {  // uniform
        int e[kBatch];
        u32x4 bv[kBatch][2];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          e[q] = -1;
          while (left && e[q] < 0) {
            const int o = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
            left &= ~(unsigned)__ballot(id == o);
            if (item++ % ks == first) e[q] = o;
          }
          const unsigned char *row = m + (e[q] < 0 ? 0 : e[q]) * each;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = r0 + 32 * h + 8 * g;
            if (e[q] >= 0 && (h == 0 || two))  // uniform
              bv[q][h] = load_guarded(row, r < p.R ? r : p.R, p.R);
          }
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          if (e[q] < 0) break;  // uniform
          f32x4 sum = mfma_16<FMT>(bv[q][0], xv[0], f32x4{0, 0, 0, 0});
          if (two) sum = mfma_16<FMT>(bv[q][1], xv[1], sum);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[b][c] += id == e[q] ? sum[c] : 0.f;
        }
      }
    }
  }
}

// The sums of the waves that share columns, added in wave order, and stored.
template <int FMT, int RB>
__device__ __forceinline__ void store_rows(const AdaptersProblem &p, unsigned char *lds,
                                           const int (&order)[64], int columns, int ks, int first,
                                           f32x4 (&acc)[RB]) {
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g = lane >> 4;
  if (ks > 1) {
    f32x4 *part = reinterpret_cast<f32x4 *>(lds);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < RB; ++b) part[(wave * RB + b) * 64 + lane] = acc[b];
    __syncthreads();
    if (first != 0) return;
    for (int o = 1; o < ks; ++o)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[b] += part[((wave + o) * RB + b) * 64 + lane];
  }
  const int c0 = columns + 4 * g;
#pragma unroll
  for (int b = 0; b < RB; ++b)
    if (16 * b + l16 < p.T)
      store4<FMT>(p.Y, order[16 * b + l16] * p.ldy + c0, p.N - c0, acc[b]);
}

constexpr int kThinWaves = 4, kThinThreads = 64 * kThinWaves;

// ---- rows of whole 16 bytes ----------------------------------------------------------------
// A round is a 64-deep step for each of the KS waves of a block of columns: x's rows and W's
// of the workgroup's 64 / KS columns come straight into one of STAGES stages, those of
// the STAGES - 1 rounds ahead on their way.  Every wave asks for as many loads each
// round, so that their number tells which have come.
template <int RB, int KS>
struct Rounds {
  static constexpr int X = RB * 2048, W = 2048;      // bytes of a wave's step
  static constexpr int STAGE = KS * X + kThinWaves * W;
  static constexpr int STAGES = 150 * 1024 / STAGE < 8 ? 150 * 1024 / STAGE : 8;
  static constexpr int X_LOADS = (2 * RB * KS + kThinWaves - 1) / kThinWaves;  // a wave's, 1 KB each
  static constexpr int LOADS = X_LOADS + 2;
  static constexpr int LDS = STAGES * STAGE;
  static_assert(STAGES >= 3 && LOADS * (STAGES - 2) < 64, "loads that can be counted");
  static_assert(kThinWaves * RB * 1024 <= LDS, "the waves' sums");
};

template <int FMT, int RB, int KS>
__global__ void __launch_bounds__(kThinThreads) adapters_rounds_kernel(AdaptersProblem p) {
  typedef Rounds<RB, KS> R;
  __shared__ __attribute__((aligned(16))) unsigned char lds[R::LDS];
  __shared__ int order[64], ids[64];
  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t *)lds;
  const int lane = threadIdx.x & 63, wave = wave_id();
  order_rows(p, order, ids);
  const int first = wave % KS;
  const int columns = 16 * ((int)blockIdx.x * (kThinWaves / KS) + wave / KS);
  const rsrc_t xs = buffer_of(p.X, records_of(2 * ((p.T - 1) * p.ldx + p.K)));
  const uint16_t *w0 = p.W + (long long)columns * p.ldw;
  const int have = p.N - columns < 16 ? p.N - columns : 16;  // columns, or none
  const rsrc_t ws = buffer_of(have > 0 ? w0 : p.W,
                              have > 0 ? records_of(2 * ((have - 1) * p.ldw + p.K)) : 0);
  // A load brings 8 rows of 8 chunks: row l / 8, chunk c0 of even loads (m16_a_pos).
  const int c0 = (lane & 7) ^ (lane >> 4);
  int wv[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) wv[h] = (int)(2 * (8 * h + (lane >> 3)) * p.ldw) + 16 * (c0 ^ (4 * h));
  __syncthreads();
  // x's loads are dealt to the waves, some twice where they do not come out even.
  int xv[R::X_LOADS], part[R::X_LOADS], place[R::X_LOADS];
#pragma unroll
  for (int q = 0; q < R::X_LOADS; ++q) {
    const int i = (wave + kThinWaves * q) % (2 * RB * KS), in = i % (2 * RB);
    const int r = 8 * in + (lane >> 3);
    part[q] = i / (2 * RB);
    place[q] = part[q] * R::X + in * 1024;
    xv[q] = r < p.T ? (int)(2 * order[r] * p.ldx) + 16 * (c0 ^ (4 * (in & 1))) : kOutside;
  }
  const int steps = (p.K + kStepK - 1) / kStepK, rounds = (steps + KS - 1) / KS;
  auto issue = [&](int round, int stage) __attribute__((always_inline)) {
    const unsigned to = lds_u + stage * R::STAGE;
#pragma unroll
    for (int q = 0; q < R::X_LOADS; ++q) {
      const int k0 = kStepK * (round * KS + part[q]);
      const int i = (wave + kThinWaves * q) % (2 * RB * KS);
      const bool in = k0 + 8 * (c0 ^ (4 * (i & 1))) < p.K;
      buffer_load_to_lds16(in ? xv[q] : kOutside, xs, uniform(2 * k0),
                           (unsigned)uniform((int)(to + place[q])));
    }
    const int k0 = kStepK * (round * KS + first);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k0 + 8 * (c0 ^ (4 * h)) < p.K;
      buffer_load_to_lds16(in ? wv[h] : kOutside, ws, uniform(2 * k0),
                           (unsigned)uniform((int)(to + KS * R::X + wave * R::W + h * 1024)));
    }
  };
#pragma unroll
  for (int i = 0; i < R::STAGES - 1; ++i) issue(i, i);
  f32x4 acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = f32x4{0, 0, 0, 0};
  int stage = 0, ahead = R::STAGES - 1;
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(R::LOADS * (R::STAGES - 2)));  // round i's, own
    ks_lds_barrier();  // everyone's; the stage of round i - 1 is free
    issue(i + R::STAGES - 1, ahead);  // past the end: zeros
    const char *st = reinterpret_cast<const char *>(lds) + stage * R::STAGE;
#pragma unroll
    for (int kg = 0; kg < 2; ++kg) {
      const i16x8 wf = read_operand<false, 16>(st + KS * R::X + wave * R::W, 0, kg, lane);
#pragma unroll
      for (int b = 0; b < RB; ++b)
        acc[b] = mfma_rows<FMT>(wf, read_operand<false, 16>(st + first * R::X, b, kg, lane), acc[b]);
    }
    stage = stage + 1 == R::STAGES ? 0 : stage + 1;
    ahead = ahead + 1 == R::STAGES ? 0 : ahead + 1;
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(0));
  add_adapters<FMT, RB>(p, order, ids, columns, KS, first, acc);
  store_rows<FMT, RB>(p, lds, order, columns, KS, first, acc);
}

// ---- any rows ----------------------------------------------------------------------------------
// x waits in LDS, the weights of two pieces of 128 values are on their way while a third
// is used.
constexpr int kThinLds = 74 * 1024;  // of x: two workgroups to a compute unit

template <int FMT, int RB, int ROWS>
__global__ void __launch_bounds__(kThinThreads, 2) adapters_thin_kernel(AdaptersProblem p, Tile tile,
                                                                        int ks) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ int order[64], ids[64];  // rows, and their adapters
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g = lane >> 4;
  order_rows(p, order, ids);
  __syncthreads();
  const int first = wave & (ks - 1);
  const int columns = 16 * ((int)blockIdx.x * (kThinWaves / ks) + wave / ks);
  const int col = columns + (lane >> 2) < p.N ? columns + (lane >> 2) : p.N - 1;
  const unsigned char *w = bytes_of(p.W + col * p.ldw);
  auto row = [&](int r) __attribute__((always_inline)) {
    return bytes_of(p.X + order[r] * p.ldx);
  };
  const int pieces = (int)ceil_div(p.K, 128), rounds = (int)ceil_div(pieces, ks);
  const int per = tile.kc / (128 * ks);  // rounds in a tile of x
  const int G = tile.group();
  HalfPiece<ROWS> x[2];
  auto load = [&](int u, int round) __attribute__((always_inline)) {
    const int piece = first + round * ks;
    x[u].load(w, piece < pieces ? piece : pieces - 1, lane, p.K);
  };
  stage_acts<FMT, FMT, ROWS>(lds, tile, row, p.T, 0, p.K, threadIdx.x, kThinThreads);
  load(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  load(1, 1);
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();
  f32x4 acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = f32x4{0, 0, 0, 0};
#pragma unroll 1
  for (int q = 0; q < rounds; q += 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int round = q + u, piece = first + round * ks;
      if (round < rounds) {  // uniform
        if (round > 0 && round % per == 0) {
          __syncthreads();
          stage_acts<FMT, FMT, ROWS>(lds, tile, row, p.T, round * ks * 128, p.K, threadIdx.x,
                                     kThinThreads);
          __syncthreads();
        }
        if (piece < pieces) {
          if (piece >= p.K / 128) x[u].end(w, piece, lane, p.K);
          const unsigned char *from = lds + ((round % per * ks + first) * 16 + g) * G;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4 wv = from_lane(x[u].get(j, lane), loader(lane));
#pragma unroll
            for (int b = 0; b < RB; ++b) {
              const int r = RB == 1 ? lane & (tile.rows - 1) : 16 * b + l16;
              acc[b] = mfma_16<FMT>(wv, *reinterpret_cast<const u32x4 *>(from + j * 4 * G + 16 * r),
                                    acc[b]);
            }
          }
        }
        load(u, round + 2);
      }
    }
  }
  add_adapters<FMT, RB>(p, order, ids, columns, ks, first, acc);
  store_rows<FMT, RB>(p, lds, order, columns, ks, first, acc);
}

template <int FMT, int RB, int ROWS>
hipError_t launch_thin(const AdaptersProblem &p, hipStream_t s) {
  const long long groups = ceil_div(p.N, 16), pieces = ceil_div(p.K, 128);
  // Waves to a block of columns: until there are four to a SIMD.
  int ks = 1;
  while (ks < kThinWaves && 2 * ks <= pieces && groups * ks < 4 * 4 * 256) ks *= 2;
  const Tile tile = tile_of<FMT>(RB == 1 ? tile_rows(p.T) : 16 * RB, p.K, 128 * ks, kThinLds);
  int lds = act_bytes<FMT>(tile);
  const int sums = ks > 1 ? kThinWaves * RB * 1024 : 0;
  lds = lds > sums ? lds : sums;
  AdaptersProblem q = p;
  Tile t = tile;
  void *args[] = {&q, &t, &ks};
  return hipLaunchKernel(reinterpret_cast<const void *>(adapters_thin_kernel<FMT, RB, ROWS>),
                         dim3((unsigned)ceil_div(groups, kThinWaves / ks)), dim3(kThinThreads), args,
                         (size_t)lds, s);
}
template <int FMT, int RB, int KS>
hipError_t launch_rounds(const AdaptersProblem &p, hipStream_t s) {
  return launch_kernel(adapters_rounds_kernel<FMT, RB, KS>,
                       dim3((unsigned)ceil_div(p.N, 16 * kThinWaves / KS)), dim3(kThinThreads), s, p);
}
// Waves to a block of columns: until there is a workgroup to each compute unit.
template <int FMT, int RB>
hipError_t launch_direct(const AdaptersProblem &p, hipStream_t s) {
  const long long groups = ceil_div(p.N, 16);
  if (groups >= 4 * 256) return launch_rounds<FMT, RB, 1>(p, s);
  if (groups >= 2 * 256) return launch_rounds<FMT, RB, 2>(p, s);
  return launch_rounds<FMT, RB, 4>(p, s);
}

template <int FMT, int ROWS>
hipError_t launch_both(const AdaptersProblem &p, hipStream_t s) {
  if (p.count > 0) {
    // (whole 32s of ranks: the second product reads them)
    const hipError_t e =
        launch_kernel(adapters_low_thin_kernel<FMT, ROWS>,
                      dim3((unsigned)p.T, (unsigned)(2 * ceil_div(p.R, 32))), dim3(64 * kLowWaves), s, p);
    if (e != hipSuccess) return e;
  }
  if (direct(p.X, p.ldx, p.K, p.T) && direct(p.W, p.ldw, p.K, 16)) {
    if (p.T <= 16) return launch_direct<FMT, 1>(p, s);
    return p.T <= 32 ? launch_direct<FMT, 2>(p, s) : launch_direct<FMT, 4>(p, s);
  }
  if (p.T <= 16) return launch_thin<FMT, 1, ROWS>(p, s);
  if (p.T <= 32) return launch_thin<FMT, 2, ROWS>(p, s);
  return launch_thin<FMT, 4, ROWS>(p, s);
}
// Rows that start in the middle of a 4-byte word are read by whole words, where the
// matrices start on one.
template <int FMT>
hipError_t launch_format(const AdaptersProblem &p, hipStream_t s) {
  if (p.K < 8) return launch_both<FMT, kShort>(p, s);
  const bool words = (reinterpret_cast<uintptr_t>(p.X) & 3) == 0 &&
                     (reinterpret_cast<uintptr_t>(p.W) & 3) == 0 &&
                     (p.count == 0 || (reinterpret_cast<uintptr_t>(p.A) & 3) == 0);
  const bool some = p.ldx % 2 || p.ldw % 2 || (p.count > 0 && p.lda % 2);
  return words && some ? launch_both<FMT, kOdd>(p, s) : launch_both<FMT, kWords>(p, s);
}

}  // namespace

hipError_t launch_adapters_thin(const AdaptersProblem &p, hipStream_t s) {
  return p.format == kBf16 ? launch_format<kBf16>(p, s) : launch_format<kF16>(p, s);
}

}  // namespace gemm_f32_impl
