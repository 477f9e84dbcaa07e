// Products of 16-bit matrices in tiles whose rows are chosen by a list (gfx950):
// the experts' products and the adapters'.
//
// A tile is WGM x WGN waves of WTM / 16 x WTN / 16 blocks of v_mfma_f32_16x16x32,
// in 64-deep k steps and two or more LDS stages.  The waves that share columns
// take the tile's blocks of 16 rows in turn, so that a tile
// with few rows costs every wave the same, and blocks without rows are passed
// over.  An operand lies in memory in one of two ways, and in LDS likewise:
//   * k along its rows (KcSide): rows of 64 k, 8 chunks of 16 bytes, at m16_a_pos;
//     a lane's operand is one 16-byte read;
//   * k down its rows (KmSide): rows of W columns in 32-byte slots, at m16_b_slot;
//     a lane's operand is two transposing reads (mixed16.hip).
// Rows that are not there, columns past the width and k past the end are zeros.
//
// S says how operands come to LDS.  kDirect: by buffer loads straight into it; a
// lane with nothing to load takes an offset past the buffer's record count.  Needs
// 16-byte aligned rows, widths of whole 16 bytes and 32-bit offsets.  Else
// through registers with 64-bit addresses: kByWords: rows that may start in the middle
// of a 4-byte word, of 8 values at least, in a matrix that starts on one; kAnyRows:
// anything.
#pragma once

#include "addr_math16.hpp"
#include "buffer_lds.hpp"
#include "mx_thin.hpp"
#include "w16_tiles.hpp"

namespace gemm_f32_impl {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

enum { kDirect, kByWords, kAnyRows };
constexpr int kStepK = 64;
constexpr int kMostRecords = 0x7ffffff0;
constexpr int kNever = 0x7fffffff;

// WGM x WGN waves of WTM x WTN, and LDS stages: two, or more for tiles that each have a
// compute unit to themselves (then what bounds a step is how long its loads take).
template <int WTM_, int WTN_, int WGM_, int WGN_, int STAGES_ = 2>
struct RowTile {
  static constexpr int STAGES = STAGES_;
  static constexpr int WTM = WTM_, WTN = WTN_, WGM = WGM_, WGN = WGN_, WAVES = WGM_ * WGN_;
  static constexpr int BM = WGM_ * WTM_, BN = WGN_ * WTN_, THREADS = 64 * WAVES;
  static constexpr int TBM = WTM_ / 16, TBN = WTN_ / 16;
  static constexpr int A_BYTES = BM * kStepK * 2, B_BYTES = BN * kStepK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int A_LOADS = BM / 8 / WAVES, B_LOADS = BN / 8 / WAVES;  // per wave and step, 1 KB each
  static_assert(A_LOADS % 2 == 0 && B_LOADS % 2 == 0, "whole pairs of loads (KcSide)");
  static constexpr int LDS = STAGES * STAGE;
  static_assert(LDS <= kLdsBytes && (STAGES - 2) * (A_LOADS + B_LOADS) < 64, "the stages");
};

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline const void *uniform(const void *p) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return reinterpret_cast<const void *>((uintptr_t)(uint32_t)uniform((int)(a >> 32)) << 32 |
                                        (uint32_t)uniform((int)a));
}
// (Made again for each step: the compiler may carry what all lanes share in vector
// registers from one to the next.)
__device__ inline int records_of(long long bytes) {
  return (int)(bytes < kMostRecords ? bytes : kMostRecords);
}
__device__ inline rsrc_t buffer_of(const void *p, int records) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(uniform(p)), 0, uniform(records),
                                           0x00020000);
}

// 8 codes on their way through registers, in memory order along the lanes of a row.
// kByWords: the words around them, from 2 bytes before the first on where that is in
// the middle of one (the row before, or its padding: only rows after the first can be,
// because the matrix starts on a word); the last code is the first of the next lane's
// words, or `last`.  In a step that passes the end of the rows (`tail`, the same for all
// lanes) the 8 codes that end there at the latest, moved into place when they are put
// to LDS, each lane with a `last` of its own.
template <int S>
struct Chunk {
  u32x4 v;
  uint32_t last;
  int shift, drop;
  // Codes k .. k + 7 of `row`, of which there are `width`; the lane that holds the
  // row's last chunk of the step ends at `end`.
  __device__ __forceinline__ void load(const uint16_t *row, int k, int width, int end, bool tail) {
    if constexpr (S == kByWords) {
      int from = k, stop = end - 1;
      if (tail) {  // uniform
        from = k < width - 8 ? k : width - 8;
        drop = k - from;
        stop = from + 7;
      }
      const uint16_t *at = row + from;
      const uintptr_t odd = reinterpret_cast<uintptr_t>(at) & 2;
      v = *reinterpret_cast<const u32x4w *>(reinterpret_cast<const char *>(at) - odd);
      last = row[stop];
      shift = 8 * (int)odd;
    } else {
      v = load_guarded(reinterpret_cast<const unsigned char *>(row), k < width ? k : width, width);
    }
  }
  __device__ __forceinline__ u32x4 get(bool ends, bool tail) const {
    if constexpr (S != kByWords) return v;
    const uint32_t next =
        (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[0], 0x101, 0xf, 0xf, true);  // lane + 1's
    const uint32_t word = ends || tail ? last : next;
    u32x4 x{__builtin_amdgcn_alignbit(v[1], v[0], (uint32_t)shift),
            __builtin_amdgcn_alignbit(v[2], v[1], (uint32_t)shift),
            __builtin_amdgcn_alignbit(v[3], v[2], (uint32_t)shift),
            __builtin_amdgcn_alignbit(word, v[3], (uint32_t)shift)};
    if (tail) x = drop_first(x, drop);
    return x;
  }
};

// An operand with k along its rows, W rows of it, loaded by NW waves.  `row(r, q)`: row r's first element,
// or null (then nothing that is read of the result depends on it); q, the number of
// the load that brings it, row_of its r.  K values to a row; from step `half` on (for rows of two
// parts, each of whole steps and K values) the second part.
template <int W, int S, int NW>
struct KcSide {
  static constexpr bool kDown = false, kListed = false;
  static constexpr int kLoads = W / 8 / NW;
  const void *base;
  int records;
  rsrc_t rsrc;
  int voff[S == kDirect ? kLoads : 1];
  const uint16_t *rows[S == kDirect ? 1 : kLoads];
  Chunk<S == kDirect ? kAnyRows : S> held[S == kDirect ? 1 : kLoads];
  int c0, K, half, step, left;

  static __device__ __forceinline__ int row_of(int q, int wave, int lane) {
    return 8 * (kLoads * wave + q) + (lane >> 3);
  }
  // `base`, `bytes`: what the rows lie in (kDirect).
  template <class RowOf>
  __device__ __forceinline__ void init(const void *base_, long long bytes, RowOf row, int K_,
                                       int half_, int wave, int lane) {
    K = K_;
    half = half_;
    c0 = (lane & 7) ^ (lane >> 4);
    base = base_;
    records = records_of(bytes);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const uint16_t *r = row(row_of(q, wave, lane), q);
      if constexpr (S == kDirect)
        voff[q] = r ? (int)(reinterpret_cast<const char *>(r) - static_cast<const char *>(base)) +
                          16 * (c0 ^ (4 * (q & 1)))
                    : kOutside;
      else
        rows[q] = r ? r : static_cast<const uint16_t *>(base);
    }
  }
  __device__ __forceinline__ void begin(int kk) {
    turn(kk);
    seal();
  }
  // In two parts, for steps that may be of different rows.
  __device__ __forceinline__ void turn(int kk) {
    step = kk;
    left = K - kStepK * (kk >= half ? kk - half : kk);  // values from the step's first on
  }
  __device__ __forceinline__ void seal() {
    if constexpr (S == kDirect) rsrc = buffer_of(base, records);
  }
  __device__ __forceinline__ void issue(int q, unsigned stage, int wave) {
    const int v = 8 * (c0 ^ (4 * (q & 1))) < left ? voff[q] : kOutside;
    buffer_load_to_lds16(v, rsrc, uniform(2 * kStepK * step), (unsigned)uniform((int)(stage + (kLoads * wave + q) * 1024)));
  }
  __device__ __forceinline__ bool tail() const { return left < kStepK; }
  __device__ __forceinline__ void load(int q, int, int lane) {
    const int k0 = K - left;
    held[q].load(rows[q] + (kStepK * step - k0), k0 + 8 * (lane & 7), K, k0 + kStepK, tail());
  }
  __device__ __forceinline__ void put(char *st, int q, int wave, int lane) const {
    *reinterpret_cast<u32x4 *>(st + 16 * m16_a_pos(row_of(q, wave, lane), lane & 7)) =
        held[q].get((lane & 7) == 7, tail());
  }
};

// Chunk c of k row r, to where side_issue's loads would bring it; zeros where it is not `in`.
template <int W>
__device__ __forceinline__ void put_down(char *st, int r, int c, u32x4 v, bool in) {
  *reinterpret_cast<u32x4 *>(st + r * (2 * W) + 32 * m16_b_slot(r, c >> 1) + 16 * (c & 1)) =
      in ? v : u32x4{0, 0, 0, 0};
}

// An operand with k down its rows, `width` (at most W) columns of it: n rows from
// `first` on, ld elements apart.  From step `half` on the second part: n rows
// from `second` on.
template <int W, int S, int NW>
struct KmSide {
  static constexpr bool kDown = true, kListed = false;
  static constexpr int kLoads = W / 8 / NW, kChunks = W / 8;
  rsrc_t rsrc;
  int voff[S == kDirect ? kLoads : 1];
  Chunk<S == kDirect ? kAnyRows : S> held[S == kDirect ? 1 : kLoads];
  const uint16_t *first, *second, *at;
  long long ld;
  int n, half, width, left;

  static __device__ __forceinline__ int row_of(int q, int wave, int lane) {
    return (64 * (kLoads * wave + q) + lane) / kChunks;
  }
  static __device__ __forceinline__ int column_of(int q, int wave, int lane) {
    const int pos = lane % kChunks;  // 64 is a multiple of kChunks
    return 8 * (2 * m16_b_slot(row_of(q, wave, lane), pos >> 1) + (pos & 1));
  }
  __device__ __forceinline__ void init(const uint16_t *first_, const uint16_t *second_,
                                       long long ld_, int n_, int half_, int width_, int wave,
                                       int lane) {
    first = first_;
    second = second_;
    ld = ld_;
    n = n_;
    half = half_;
    width = width_;
    if constexpr (S == kDirect)
#pragma unroll
      for (int q = 0; q < kLoads; ++q) {
        const int c = column_of(q, wave, lane);
        voff[q] = c < width ? (int)(2 * (row_of(q, wave, lane) * ld + c)) : kOutside;
      }
  }
  __device__ __forceinline__ void begin(int kk) {
    const int k0 = kStepK * (kk >= half ? kk - half : kk);
    left = n - k0;
    at = (kk >= half ? second : first) + k0 * ld;
    if constexpr (S == kDirect)  // rows past the end are past the record count
      rsrc = buffer_of(at, left > 0 ? records_of(2 * ((left - 1) * ld + width)) : 0);
  }
  __device__ __forceinline__ void issue(int q, unsigned stage, int wave) {
    buffer_load_to_lds16(voff[q], rsrc, 0, (unsigned)uniform((int)(stage + (kLoads * wave + q) * 1024)));
  }
  __device__ __forceinline__ bool tail() const { return left < kStepK || width < W; }
  __device__ __forceinline__ void load(int q, int wave, int lane) {
    const int r = row_of(q, wave, lane);  // (width - 8 may be negative: columns before the tile's)
    held[q].load(at + (r < left ? r : left - 1) * ld, 8 * (lane % kChunks), width, W, tail());
  }
  __device__ __forceinline__ void put(char *st, int q, int wave, int lane) const {
    const int r = row_of(q, wave, lane);
    put_down<W>(st, r, lane % kChunks, held[q].get(lane % kChunks == kChunks - 1, tail()), r < left);
  }
};

// The same with its rows chosen by a list: row k is row list[k] of `base`.  The list
// is read a step ahead.
template <int W, int S, int NW>
struct KmListSide {
  static constexpr bool kDown = true, kListed = true;  // (its steps come in order)
  static constexpr int kLoads = W / 8 / NW, kChunks = W / 8;
  rsrc_t rsrc;
  int records;
  Chunk<S == kDirect ? kAnyRows : S> held[S == kDirect ? 1 : kLoads];
  const uint16_t *base;
  const int *list;
  long long ld;
  int n, last, width, k0;
  int now[kLoads], next[kLoads];

  __device__ __forceinline__ void fetch(int kk, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int k = kStepK * kk + KmSide<W, S, NW>::row_of(q, wave, lane);
      now[q] = next[q];
      next[q] = list[k < n ? k : last];
    }
  }
  // `list` has a readable place if n is 0.  Before begin(0).
  __device__ __forceinline__ void init(const uint16_t *base_, long long bytes, long long ld_,
                                       const int *list_, int n_, int width_, int wave, int lane) {
    base = base_;
    ld = ld_;
    list = list_;
    n = n_;
    last = n > 0 ? n - 1 : 0;
    width = width_;
    records = records_of(bytes);
    fetch(0, wave, lane);
  }
  __device__ __forceinline__ void begin(int kk, int wave, int lane) {
    k0 = kStepK * kk;
    if constexpr (S == kDirect) rsrc = buffer_of(base, records);
    fetch(kk + 1, wave, lane);
  }
  __device__ __forceinline__ void issue(int q, unsigned stage, int wave, int lane) {
    const int c = KmSide<W, S, NW>::column_of(q, wave, lane);
    const bool in = k0 + KmSide<W, S, NW>::row_of(q, wave, lane) < n && c < width;
    buffer_load_to_lds16(in ? (int)(2 * (now[q] * ld + c)) : kOutside, rsrc, 0,
                         (unsigned)uniform((int)(stage + (kLoads * wave + q) * 1024)));
  }
  __device__ __forceinline__ bool tail() const { return k0 + kStepK > n || width < W; }
  __device__ __forceinline__ void load(int q, int, int lane) {
    held[q].load(base + now[q] * ld, 8 * (lane % kChunks), width, W, tail());
  }
  __device__ __forceinline__ void put(char *st, int q, int wave, int lane) const {
    const int r = KmSide<W, S, NW>::row_of(q, wave, lane);
    put_down<W>(st, r, lane % kChunks, held[q].get(lane % kChunks == kChunks - 1, tail()),
                k0 + r < n);
  }
};

// One set of calls for all sides.
template <int W, int S, int NW>
__device__ __forceinline__ void side_begin(KcSide<W, S, NW> &x, int kk, int, int) { x.begin(kk); }
template <int W, int S, int NW>
__device__ __forceinline__ void side_begin(KmSide<W, S, NW> &x, int kk, int, int) { x.begin(kk); }
template <int W, int S, int NW>
__device__ __forceinline__ void side_begin(KmListSide<W, S, NW> &x, int kk, int wave, int lane) {
  x.begin(kk, wave, lane);
}
template <int W, int S, int NW>
__device__ __forceinline__ void side_issue(KcSide<W, S, NW> &x, int q, unsigned stage, int wave, int) {
  x.issue(q, stage, wave);
}
template <int W, int S, int NW>
__device__ __forceinline__ void side_issue(KmSide<W, S, NW> &x, int q, unsigned stage, int wave, int) {
  x.issue(q, stage, wave);
}
template <int W, int S, int NW>
__device__ __forceinline__ void side_issue(KmListSide<W, S, NW> &x, int q, unsigned stage, int wave,
                                           int lane) {
  x.issue(q, stage, wave, lane);
}
// A lane's operand: block `block` of 16 rows (columns), 32-deep group kg.
template <bool DOWN, int W>
__device__ __forceinline__ i16x8 read_operand(const char *st, int block, int kg, int lane) {
  const int l16 = lane & 15, g = lane >> 4;
  if constexpr (!DOWN) {
    return *reinterpret_cast<const i16x8 *>(st + 16 * m16_a_pos(16 * block + l16, 4 * kg + g));
  } else {
    i16x4 h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 32 * kg + 8 * g + 4 * i + (l16 >> 2);
      const char *at = st + k * (W * 2) + 32 * m16_b_slot(k, block) + 8 * (l16 & 3);
      h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at));
    }
    return i16x8{h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
  }
}

template <int FMT>
__device__ inline f32x4 mfma_rows(i16x8 b, i16x8 a, f32x4 acc) {
  if constexpr (FMT == kBf16)
    return mfma_bf16(__builtin_bit_cast(u32x4, b), __builtin_bit_cast(u32x4, a), acc);
  else
    return mfma_f16(__builtin_bit_cast(u32x4, b), __builtin_bit_cast(u32x4, a), acc);
}

// How many of a wave's row blocks have any of n rows.
template <class T>
__device__ inline int blocks_of(int n, int wm) {
  return (((n + 15) >> 4) - wm + T::WGM - 1) / T::WGM;
}

// Two column blocks' four values of a lane, in 16 bits, as eight of one: lanes of
// even groups of 16 get theirs of block a, with the next group's, odd ones of block b.
// So a row's 64 bytes are stored by four lanes, 16 bytes each.
struct Eights {
  u32x4 v;
  int at;  // of 32 columns
};
template <int FMT>
__device__ inline Eights eights(f32x4 a, f32x4 b, int lane) {
  const auto lo = __builtin_amdgcn_permlane16_swap(pack2<FMT>(a[0], a[1]), pack2<FMT>(b[0], b[1]),
                                                   false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(pack2<FMT>(a[2], a[3]), pack2<FMT>(b[2], b[3]),
                                                   false, false);
  const int g = lane >> 4;
  return {u32x4{lo[0], hi[0], lo[1], hi[1]}, 16 * (g & 1) + 8 * (g >> 1)};
}
// Stored to a row of `left` values, of any alignment.
__device__ inline void store_eights(uint16_t *row, const Eights &e, int left) {
  left -= e.at;
  if (left >= 8) {
    *reinterpret_cast<u32x4h *>(row + e.at) = e.v;
    return;
  }
#pragma unroll
  for (int c = 0; c < 7; ++c)
    if (c < left) row[e.at + c] = (uint16_t)(e.v[c >> 1] >> (16 * (c & 1)));
}

// The first of a workgroup's n steps: each begins at another place in k and goes round
// (next_step).  Rows a power of two apart lie in few channels of an L2 at any one k, and of the
// memory: workgroups of one XCD begin up to three steps apart (what they share is still
// in its L2), XCDs an eighth of k.  (All from the first step, and so, us: 16,384 pairs of 8
// experts, 4096 / 4096 1,585 and 1,502; a training step of 64 experts, 2048 / 1024 1,385
// and 1,373; of 7, 1000 / 517 164 and 166; 8,192 rows with adapters, 4096 x 4096 253 and 255.)
template <class Op>
__device__ __forceinline__ int first_of(int n) {
  if constexpr (Op::A::kListed || Op::B::kListed) return 0;
  if (n < 4) return 0;  // uniform
  const int from = n * (int)(blockIdx.x & 7) / 8 + (int)(blockIdx.x >> 3 & 3);
  return uniform(from < n ? from : from - n);
}
__device__ __forceinline__ int next_step(int kk, int n) { return kk + 1 == n ? 0 : kk + 1; }

// tile_loop with more than two stages: the loads of STAGES - 1 steps are on their way.
template <class T, int FMT, int S, class Op>
__device__ __forceinline__ void deep_tiles(char *lds, Op &op, int count, int wave, int lane) {
  static_assert(S == kDirect, "direct loads");
  constexpr int kLoads = T::A_LOADS + T::B_LOADS, kAhead = T::STAGES - 1;
  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t *)lds;
  const int wm = wave / T::WGN, wn = wave % T::WGN;
  int place = 0;
  auto issue = [&](int n, int at) __attribute__((always_inline)) {
    const unsigned stage = (unsigned)uniform((int)(lds_u + at * T::STAGE));
    side_begin(op.a, place, wave, lane);
    side_begin(op.b, place, wave, lane);
    place = next_step(place, n);
#pragma unroll
    for (int q = 0; q < T::A_LOADS; ++q) side_issue(op.a, q, stage, wave, lane);
#pragma unroll
    for (int q = 0; q < T::B_LOADS; ++q) side_issue(op.b, q, stage + T::A_BYTES, wave, lane);
  };
#pragma unroll 1
  for (int t = 0; t < count; ++t) {
    const typename Op::Job job = op.job(t);
    const int nk = job.steps, blocks = blocks_of<T>(job.rows, wm);
    op.fetch(job);
    op.begin(job);
    place = first_of<Op>(nk);
#pragma unroll 1
    for (int kk = 0; kk < kAhead && kk < nk; ++kk) issue(nk, kk);
    f32x4 acc[T::TBM][T::TBN];
#pragma unroll
    for (int i = 0; i < T::TBM; ++i)
#pragma unroll
      for (int j = 0; j < T::TBN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int stage = 0;
    auto step = [&](auto more) __attribute__((always_inline)) {
      constexpr bool MORE = decltype(more)::value;
      // This step's own loads, which at least those of kAhead - 1 steps follow.
      __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(MORE ? kLoads * (kAhead - 1) : 0));
      ks_lds_barrier();  // everyone's; the stage of the step before is free
      if constexpr (MORE) issue(nk, stage == 0 ? kAhead : stage - 1);
      const char *st = lds + stage * T::STAGE;
#pragma unroll
      for (int kg = 0; kg < kStepK / 32; ++kg) {
        i16x8 fa[T::TBM], fb[T::TBN];
#pragma unroll
        for (int j = 0; j < T::TBN; ++j)
          fb[j] = read_operand<Op::B::kDown, T::BN>(st + T::A_BYTES, wn * T::TBN + j, kg, lane);
#pragma unroll
        for (int i = 0; i < T::TBM; ++i)
          fa[i] = read_operand<Op::A::kDown, T::BM>(st, T::WGM * i + wm, kg, lane);
#pragma unroll
        for (int i = 0; i < T::TBM; ++i)
          if (i < blocks) {  // uniform
#pragma unroll
            for (int j = 0; j < T::TBN; ++j) acc[i][j] = mfma_rows<FMT>(fb[j], fa[i], acc[i][j]);
          }
      }
      stage = stage + 1 == T::STAGES ? 0 : stage + 1;
    };
    int kk = 0;
#pragma unroll 1
    for (; kk + kAhead < nk; ++kk) step(std::true_type{});
#pragma unroll 1
    for (; kk < nk; ++kk) step(std::false_type{});
    op.store(job, acc, wave, lane);
    ks_lds_barrier();  // the next tile's loads overwrite the LDS
  }
}

// A workgroup's tiles, one after the other.  `Op` has
//   Job       what a tile is: `steps` of k, `rows` (of the tile's that there are), ...
//   A, B      the operands' sides, members a and b
//   job(t)    the job of this workgroup's t-th tile; t < count
//   fetch(j)  starts the loads that the sides of job j need to begin
//   begin(j)  makes the sides those of job j
//   store(j, acc, wave, lane)
// In store's acc[i][m] lane l has row l % 16 of the wave's row block i (block WGM i +
// wave / WGN of the tile) and columns 4 (l / 16) .. + 3 of its column block m (block
// TBN (wave % WGN) + m).
//
// The loads of a tile's first step are issued under the end of the tile before, so
// that they are on their way while its results are stored.
template <class T, int FMT, int S, class Op>
__device__ __forceinline__ void tile_loop(char *lds, Op &op, int count, int wave, int lane) {
  if (count <= 0) return;  // uniform
  if constexpr (T::STAGES > 2) {
    deep_tiles<T, FMT, S>(lds, op, count, wave, lane);
    return;
  }
  const unsigned lds_u = (unsigned)(uintptr_t)(lds_void_t *)lds;
  const int wm = wave / T::WGN, wn = wave % T::WGN;
  constexpr int kLoads = T::A_LOADS + T::B_LOADS;

  auto issue = [&](unsigned to, int q0, int q1) __attribute__((always_inline)) {
    const unsigned stage = (unsigned)uniform((int)to);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      if (q < q0 || q >= q1) continue;
      if (q < T::A_LOADS) side_issue(op.a, q, stage, wave, lane);
      else side_issue(op.b, q - T::A_LOADS, stage + T::A_BYTES, wave, lane);
    }
  };
  auto load = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < T::A_LOADS; ++q) op.a.load(q, wave, lane);
#pragma unroll
    for (int q = 0; q < T::B_LOADS; ++q) op.b.load(q, wave, lane);
  };
  auto put = [&](char *stage) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < T::A_LOADS; ++q) op.a.put(stage, q, wave, lane);
#pragma unroll
    for (int q = 0; q < T::B_LOADS; ++q) op.b.put(stage + T::A_BYTES, q, wave, lane);
  };
  int stage = 0, place = 0;
  // The first step of a job that has one.
  auto first_step = [&](const typename Op::Job &j) __attribute__((always_inline)) {
    op.begin(j);
    place = first_of<Op>(j.steps);
    side_begin(op.a, place, wave, lane);
    side_begin(op.b, place, wave, lane);
    if constexpr (S == kDirect) {
      issue(lds_u + stage * T::STAGE, 0, kLoads);
    } else {
      load();
      put(lds + stage * T::STAGE);
    }
  };

  typename Op::Job job = op.job(0);
  op.fetch(job);
  if (job.steps > 0) first_step(job);
#pragma unroll 1
  for (int t = 0; t < count; ++t) {
    const bool next = t + 1 < count;
    typename Op::Job after = job;
    if (next) after = op.job(t + 1);
    const int blocks = blocks_of<T>(job.rows, wm), nk = job.steps;
    f32x4 acc[T::TBM][T::TBN];
#pragma unroll
    for (int i = 0; i < T::TBM; ++i)
#pragma unroll
      for (int j = 0; j < T::TBN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // A step; MORE: another of this tile follows; FULL: every row block has rows (a
    // branch to each block costs a lone wave a tenth of its rate).
    auto step = [&](auto more, auto full) __attribute__((always_inline)) {
      constexpr bool MORE = decltype(more)::value, FULL = decltype(full)::value;
      if constexpr (S == kDirect) __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(0));  // own loads
      ks_lds_barrier();  // everyone's; the other stage is free
      const char *st = lds + stage * T::STAGE;
      stage ^= 1;
      const unsigned nst = lds_u + stage * T::STAGE;
      if constexpr (MORE) {
        place = next_step(place, nk);
        side_begin(op.a, place, wave, lane);
        side_begin(op.b, place, wave, lane);
        if constexpr (S != kDirect) load();
      } else if (next) {
        op.fetch(after);
      }
      // One group's operands, or two where there are registers for them.
      constexpr int kAhead = S == kDirect && T::TBM * T::TBN <= 16 ? 1 : 0;
      i16x8 fa[1 + kAhead][T::TBM], fb[1 + kAhead][T::TBN];
      auto read = [&](int kg) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < T::TBN; ++j)
          fb[kg & kAhead][j] =
              read_operand<Op::B::kDown, T::BN>(st + T::A_BYTES, wn * T::TBN + j, kg, lane);
#pragma unroll
        for (int i = 0; i < T::TBM; ++i)
          fa[kg & kAhead][i] = read_operand<Op::A::kDown, T::BM>(st, T::WGM * i + wm, kg, lane);
      };
      // The first group's in the order of their use.
      fb[0][0] = read_operand<Op::B::kDown, T::BN>(st + T::A_BYTES, wn * T::TBN, 0, lane);
      __builtin_amdgcn_sched_barrier(0);
      fa[0][0] = read_operand<Op::A::kDown, T::BM>(st, wm, 0, lane);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 1; j < T::TBN; ++j)
        fb[0][j] = read_operand<Op::B::kDown, T::BN>(st + T::A_BYTES, wn * T::TBN + j, 0, lane);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 1; i < T::TBM; ++i) {
        fa[0][i] = read_operand<Op::A::kDown, T::BM>(st, T::WGM * i + wm, 0, lane);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int kg = 0; kg < kStepK / 32; ++kg) {
#pragma unroll
        for (int i = 0; i < T::TBM; ++i) {
          if (FULL || i < blocks) {  // uniform
#pragma unroll
            for (int j = 0; j < T::TBN; ++j)
              acc[i][j] = mfma_rows<FMT>(fb[kg & kAhead][j], fa[kg & kAhead][i], acc[i][j]);
          }
          // Loads after each row of products: 4 against 2, long prompt's first product 1016
          // against 1027 us.
          constexpr int kPerRow = 4;
          const int row = kg * T::TBM + i;
          if (MORE && S == kDirect && row * kPerRow < kLoads) {
            __builtin_amdgcn_sched_barrier(0);
            issue(nst, row * kPerRow, (row + 1) * kPerRow);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (kg + 1 < kStepK / 32 && i == (kAhead ? T::TBM / 2 - 1 : T::TBM - 1)) {
            __builtin_amdgcn_sched_barrier(0);
            read(kg + 1);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      if constexpr (S != kDirect && MORE) put(lds + stage * T::STAGE);
      if constexpr (T::TBM * T::TBN == 64) {  // accumulation registers (see big16_kernel)
#pragma unroll
        for (int i = 0; i < T::TBM; ++i)
#pragma unroll
          for (int j = 0; j < T::TBN; ++j) asm volatile("" : "+a"(acc[i][j]));
      }
    };
    if (blocks == T::TBM) {
#pragma unroll 1
      for (int kk = 0; kk + 1 < nk; ++kk) step(std::true_type{}, std::true_type{});
    } else {
#pragma unroll 1
      for (int kk = 0; kk + 1 < nk; ++kk) step(std::true_type{}, std::false_type{});
    }
    if (nk > 0) step(std::false_type{}, std::false_type{});
    if (next) {
      if (nk <= 0) op.fetch(after);
      if (after.steps > 0) first_step(after);
    }
    op.store(job, acc, wave, lane);
    job = after;
  }
  if constexpr (S == kDirect) __builtin_amdgcn_s_waitcnt(vmcnt_wait_imm(0));
}

}  // namespace
}  // namespace gemm_f32_impl
