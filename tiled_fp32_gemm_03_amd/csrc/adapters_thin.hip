// A shared projection with low-rank adapters for few rows (gemm_adapters.h), 64 at a
// time: single tokens of many requests.  Two launches: scale A[r] x by a workgroup to each
// adapter that is asked and 16 of its ranks, and the projection, which reads W once,
// through a ring of LDS stages or, where a matrix starts in the middle of a word or 16 rows
// of W (64 of X) pass 2^31 bytes, straight into the matrix instructions' operands
// (mx_thin.hpp), and the asked adapters' B.
//
// 64 rows, 16384 x 8192, 32 adapters of rank 64: 90 us, 4.0 TB/s of W, A and B; x goes
// through each compute unit's LDS beside W, as many bytes again.
#include "adapters_rank.hpp"
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
// A launch takes 64 rows at a time: those of block b of them.
__device__ inline AdaptersProblem rows_of(AdaptersProblem p, int b) {
  const long long from = kAdaptersThin * (long long)b;
  p.X += from * p.ldx;
  p.Y += from * p.ldy;
  p.ids += from;
  p.at.v += 4 * from * p.at.rpitch;
  p.T = p.T - from < kAdaptersThin ? (int)(p.T - from) : kAdaptersThin;
  return p;
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
__global__ void __launch_bounds__(64 * kLowWaves) adapters_low_thin_kernel(AdaptersProblem all) {
  const AdaptersProblem p = rows_of(all, blockIdx.x / kAdaptersThin);
  __shared__ f32x4 part[kLowWaves][64];
  __shared__ int rows[64];
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g = lane >> 4;
  const int i = blockIdx.x % kAdaptersThin, r0 = 16 * blockIdx.y;
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
        Kept<FMT>::store(ws_at<typename Kept<FMT>::type>(p, p.at.v) +
                             rows[m0 + l16] * p.at.rpitch + r0 + 4 * g,
                         acc);
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
    const auto *v = ws_at<typename Kept<FMT>::type>(p, p.at.v) + order[16 * b + l16] * p.at.rpitch;
    const unsigned any = (unsigned)__ballot(id >= 0) & 0xffffu;
    if (any == 0) continue;  // uniform
#pragma unroll 1
    for (int r0 = 0; r0 < p.R; r0 += 64) {
      const bool two = r0 + 32 < p.R;  // uniform
      const LowRank<FMT, 2> x(v + r0 + 8 * g, id < 0 ? 0 : two ? 2 : 1);
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
          f32x4 sum = mfma_16<FMT>(bv[q][0], x.v[0], f32x4{0, 0, 0, 0});
          if (two) sum = mfma_16<FMT>(bv[q][1], x.v[1], sum);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[b][c] += id == e[q] ? x.back(sum[c]) : 0.f;
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

// ---- matrices that start on a 4-byte word ---------------------------------------------------
// A round is a 64-deep step for each of the KS waves of a block of columns: x's rows and W's
// of the workgroup's 64 / KS columns come straight into one of STAGES stages, those of
// the STAGES - 1 rounds ahead on their way.  Every wave asks for as many loads each
// round, so that their number tells which have come.
//
// Rows of whole 16 bytes lie in LDS by 8 chunks of 16 bytes, as in row_tiles.hpp.  WORDS:
// rows that may start in the middle of a word, or end inside 16 bytes, by 9 chunks from the
// word that a row's first value is in (144 bytes: 16 rows meet on no bank); the values
// are moved into place, and those past K cleared, when they are read.
template <int RB, int KS, bool WORDS>
struct Rounds {
  static constexpr int CHUNKS = WORDS ? 9 : 8, ROW = 16 * CHUNKS;
  static constexpr int X_ALL = (RB * 16 * CHUNKS + 63) / 64;  // loads of a wave's step of x, 1 KB each
  static constexpr int W_LOADS = (16 * CHUNKS + 63) / 64;
  static constexpr int X = X_ALL * 1024, W = W_LOADS * 1024;
  static constexpr int STAGE = KS * X + kThinWaves * W;
  static constexpr int STAGES = 150 * 1024 / STAGE < 8 ? 150 * 1024 / STAGE : 8;
  static constexpr int X_LOADS = (X_ALL * KS + kThinWaves - 1) / kThinWaves;  // a wave's
  static constexpr int LOADS = X_LOADS + W_LOADS;
  static constexpr int LDS = STAGES * STAGE;
  static_assert(STAGES >= 3 && LOADS * (STAGES - 2) < 64, "loads that can be counted");
  static_assert(kThinWaves * RB * 1024 <= LDS, "the waves' sums");

  // Where position n of a step's chunks comes from: row, and chunk of it.
  static __device__ __forceinline__ int row_of(int n) { return n / CHUNKS; }
  static __device__ __forceinline__ int chunk_of(int n) {
    return WORDS ? n % CHUNKS : (n & 7) ^ ((row_of(n) >> 1) & 7);
  }
};

// A lane's operand: block `block` of 16 rows, group kg of 32; WORDS: of rows that are
// `shift` bits into their words, the first `left` values of the step.
template <bool WORDS>
__device__ __forceinline__ i16x8 read_round(const unsigned char *st, int block, int kg, int lane,
                                            int shift, int left) {
  if constexpr (!WORDS) {
    return read_operand<false, 16>(reinterpret_cast<const char *>(st), block, kg, lane);
  } else {
    const int g = lane >> 4;
    const unsigned char *at = st + (16 * block + (lane & 15)) * 144 + 16 * (4 * kg + g);
    const u32x4 v = *reinterpret_cast<const u32x4 *>(at);
    const uint32_t next = *reinterpret_cast<const uint32_t *>(at + 16);
    u32x4 x{__builtin_amdgcn_alignbit(v[1], v[0], (uint32_t)shift),
            __builtin_amdgcn_alignbit(v[2], v[1], (uint32_t)shift),
            __builtin_amdgcn_alignbit(v[3], v[2], (uint32_t)shift),
            __builtin_amdgcn_alignbit(next, v[3], (uint32_t)shift)};
    if (left < kStepK) {  // uniform
      const int keep = left - 32 * kg - 8 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = keep >= 2 * i + 2 ? x[i] : keep == 2 * i + 1 ? x[i] & 0xffffu : 0u;
    }
    return __builtin_bit_cast(i16x8, x);
  }
}

template <int FMT, int RB, int KS, bool WORDS>
__global__ void __launch_bounds__(kThinThreads) adapters_rounds_kernel(AdaptersProblem all) {
  typedef Rounds<RB, KS, WORDS> R;
  const AdaptersProblem p = rows_of(all, blockIdx.y);
  __shared__ __attribute__((aligned(16))) unsigned char lds[R::LDS];
  __shared__ int order[64], ids[64];
  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t *)lds;
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15;
  order_rows(p, order, ids);
  const int first = wave % KS;
  const int columns = 16 * ((int)blockIdx.x * (kThinWaves / KS) + wave / KS);
  const int have = p.N - columns < 16 ? p.N - columns : 16;  // columns, or none
  // The words that the matrices' values are in; the wave's rows of W from the word of the first.
  const uintptr_t w_at = reinterpret_cast<uintptr_t>(p.W + (have > 0 ? columns : 0) * p.ldw);
  const int w_odd = (int)(w_at & 2), x_odd = (int)(reinterpret_cast<uintptr_t>(p.X) & 2);
  auto words = [](long long bytes) { return records_of((bytes + 3) & ~3LL); };
  const rsrc_t xs = buffer_of(reinterpret_cast<const char *>(p.X) - x_odd,
                              words(x_odd + 2 * ((p.T - 1) * p.ldx + p.K)));
  const rsrc_t ws = buffer_of(reinterpret_cast<const void *>(w_at - w_odd),
                              have > 0 ? words(w_odd + 2 * ((have - 1) * p.ldw + p.K)) : 0);
  // Offset of a row's chunk 0, and of the first value in it.
  auto w_row = [&](int r) __attribute__((always_inline)) { return w_odd + (int)(2 * r * p.ldw); };
  __syncthreads();
  auto x_row = [&](int r) __attribute__((always_inline)) {
    return x_odd + (int)(2 * order[r] * p.ldx);
  };
  int wv[R::W_LOADS], wk[R::W_LOADS];  // offsets, and the first k of the chunk in the step
#pragma unroll
  for (int h = 0; h < R::W_LOADS; ++h) {
    const int n = 64 * h + lane, r = R::row_of(n), c = R::chunk_of(n), at = w_row(r);
    wk[h] = 8 * c - (at & 2) / 2;
    wv[h] = r < have && r < 16 ? (at & ~3) + 16 * c : kOutside;
  }
  // x's loads are dealt to the waves, some twice where they do not come out even.
  int xv[R::X_LOADS], xk[R::X_LOADS], part[R::X_LOADS], place[R::X_LOADS];
#pragma unroll
  for (int q = 0; q < R::X_LOADS; ++q) {
    const int i = (wave + kThinWaves * q) % (R::X_ALL * KS), in = i % R::X_ALL;
    const int n = 64 * in + lane, r = R::row_of(n), c = R::chunk_of(n);
    const int at = x_row(r < 64 ? r : 0);
    part[q] = i / R::X_ALL;
    place[q] = part[q] * R::X + in * 1024;
    xk[q] = 8 * c - (at & 2) / 2;
    xv[q] = r < p.T && r < 16 * RB ? (at & ~3) + 16 * c : kOutside;
  }
  const int steps = (p.K + kStepK - 1) / kStepK, rounds = (steps + KS - 1) / KS;
  // A workgroup's n-th round, past the end the one after the last.  Workgroups begin at
  // places spread over K and go round: rows a power of two apart lie in few channels
  // of the memory at any one k (64 rows, 16384 x 8192: 104 us from the first round, 90 so; one row,
  // 4096 x 4096: 16.3 and 15.8).
  const int shift = (int)((long long)blockIdx.x * rounds / gridDim.x);
  auto round_of = [&](int n) __attribute__((always_inline)) {
    const int r = n + shift;
    return uniform(n >= rounds ? rounds : r < rounds ? r : r - rounds);
  };
  auto issue = [&](int n, int stage) __attribute__((always_inline)) {
    const unsigned to = lds_u + stage * R::STAGE;
    const int round = round_of(n);
#pragma unroll
    for (int q = 0; q < R::X_LOADS; ++q) {
      const int k0 = kStepK * (round * KS + part[q]);
      buffer_load_to_lds16(k0 + xk[q] < p.K ? xv[q] : kOutside, xs, uniform(2 * k0),
                           (unsigned)uniform((int)(to + place[q])));
    }
    const int k0 = kStepK * (round * KS + first);
#pragma unroll
    for (int h = 0; h < R::W_LOADS; ++h)
      buffer_load_to_lds16(k0 + wk[h] < p.K ? wv[h] : kOutside, ws, uniform(2 * k0),
                           (unsigned)uniform((int)(to + KS * R::X + wave * R::W + h * 1024)));
  };
#pragma unroll
  for (int i = 0; i < R::STAGES - 1; ++i) issue(i, i);
  // Bits that a lane's rows are into their words.
  int ws_shift = 8 * (w_row(l16) & 2), xs_shift[RB];
  f32x4 acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    xs_shift[b] = 8 * (x_row(16 * b + l16) & 2);
    acc[b] = f32x4{0, 0, 0, 0};
  }
  int stage = 0, ahead = R::STAGES - 1;
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(R::LOADS * (R::STAGES - 2)));  // round i's, own
    ks_lds_barrier();  // everyone's; the stage of round i - 1 is free
    issue(i + R::STAGES - 1, ahead);  // past the end: zeros
    const unsigned char *st = lds + stage * R::STAGE;
    const int left = p.K - kStepK * (round_of(i) * KS + first);
#pragma unroll
    for (int kg = 0; kg < 2; ++kg) {
      const i16x8 wf = read_round<WORDS>(st + KS * R::X + wave * R::W, 0, kg, lane, ws_shift, left);
#pragma unroll
      for (int b = 0; b < RB; ++b)
        acc[b] = mfma_rows<FMT>(
            wf, read_round<WORDS>(st + first * R::X, b, kg, lane, xs_shift[b], left), acc[b]);
    }
    stage = stage + 1 == R::STAGES ? 0 : stage + 1;
    ahead = ahead + 1 == R::STAGES ? 0 : ahead + 1;
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(0));
  add_adapters<FMT, RB>(p, order, ids, columns, KS, first, acc);
  store_rows<FMT, RB>(p, lds, order, columns, KS, first, acc);
}

// ---- matrices that start in the middle of a word, and pitches past the ring's offsets ------
// x waits in LDS, the weights of two pieces of 128 values are on their way while a third
// is used.
constexpr int kThinLds = 74 * 1024;  // of x: two workgroups to a compute unit

template <int FMT, int RB, int ROWS>
__global__ void __launch_bounds__(kThinThreads, 2) adapters_thin_kernel(AdaptersProblem all,
                                                                        Tile tile, int ks) {
  const AdaptersProblem p = rows_of(all, blockIdx.y);
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
                         dim3((unsigned)ceil_div(groups, kThinWaves / ks),
                              (unsigned)ceil_div(p.T, kAdaptersThin)),
                         dim3(kThinThreads), args,
                         (size_t)lds, s);
}
// Whether `rows` rows of a matrix that starts on a word are within 32-bit offsets.
bool on_words(const uint16_t *p, long long ld, long long rows) {
  return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && 2 * rows * ld + 64 <= kMostRecords;
}
template <int FMT, int RB, int KS, bool WORDS>
hipError_t launch_rounds(const AdaptersProblem &p, hipStream_t s) {
  return launch_kernel(adapters_rounds_kernel<FMT, RB, KS, WORDS>,
                       dim3((unsigned)ceil_div(p.N, 16 * kThinWaves / KS),
                            (unsigned)ceil_div(p.T, kAdaptersThin)),
                       dim3(kThinThreads), s, p);
}
// Waves to a block of columns: until there is a workgroup to each compute unit.
template <int FMT, int RB, bool WORDS>
hipError_t launch_direct(const AdaptersProblem &p, hipStream_t s) {
  const long long groups = ceil_div(p.N, 16);
  if (groups >= 4 * 256) return launch_rounds<FMT, RB, 1, WORDS>(p, s);
  if (groups >= 2 * 256) return launch_rounds<FMT, RB, 2, WORDS>(p, s);
  return launch_rounds<FMT, RB, 4, WORDS>(p, s);
}
template <int FMT, bool WORDS>
hipError_t launch_blocks(const AdaptersProblem &p, hipStream_t s) {
  if (p.T <= 16) return launch_direct<FMT, 1, WORDS>(p, s);
  return p.T <= 32 ? launch_direct<FMT, 2, WORDS>(p, s) : launch_direct<FMT, 4, WORDS>(p, s);
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
  if (direct(p.X, p.ldx, p.K, kAdaptersThin) && direct(p.W, p.ldw, p.K, 16))
    return launch_blocks<FMT, false>(p, s);
  if (on_words(p.X, p.ldx, kAdaptersThin) && on_words(p.W, p.ldw, 16))
    return launch_blocks<FMT, true>(p, s);
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
