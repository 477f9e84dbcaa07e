// Pieces of the products of few rows of activations with weights that are read
// once from memory, which is what bounds them (gemm_mx_a16, the
// mixture-of-experts layer).
//
// A wave multiplies blocks of 16 activation rows with blocks of 16 weight
// rows ("columns" of C) and takes K in pieces of 256 bytes of weight row:
// four 128-deep steps of MX weights, one of 16-bit ones.  The weights go from
// memory into registers, the next piece's while one is used; the activations,
// which a workgroup's waves share, wait in LDS.  Loads complete in order, so
// activations loaded from memory between the pieces would make each wave wait
// for the next piece's weights as well (measured: twice the time).
//
// Lane l multiplies row l % 16 of each operand; which k a lane holds is free
// as long as both operands agree, so it follows how the weights are stored,
// with g = l / 16:
//   MX weights: block 4 s + g of a piece in step s; MFMA j of the step takes
//     its values 8 j .. 8 j + 7, widened with their scale (exact: an element
//     has two significant bits);
//   16-bit weights: load j is k = 32 j + 8 g .. + 7, the operand of MFMA j.
#pragma once

#include "mx_values.hpp"

#include <type_traits>

namespace gemm_f32_impl {
namespace {

// Kinds of operands: the formats of mx_plan.hpp (kF32: activations split into
// two bf16 terms, hi + lo, 16 significant bits), and MX rows.
constexpr int kMx = 3;

template <int W>
constexpr int kPieceK = W == kMx ? 512 : 128;
// 128-deep steps of a piece.
template <int W>
constexpr int kPieceSteps = kPieceK<W> / 128;

__device__ inline f32x4 mfma_bf16(u32x4 b, u32x4 a, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b),
                                                 __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
}
__device__ inline f32x4 mfma_f16(u32x4 b, u32x4 a, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b),
                                                __builtin_bit_cast(f16x8, a), acc, 0, 0, 0);
}

// hi + lo, in bf16, of 8 fp16 values: exact (11 significant bits, lo at most
// 128).  An infinity or a NaN is hi alone.
__device__ inline void split_f16(u32x4 x, u32x4 &hi, u32x4 &lo) {
  const f16x8 v = __builtin_bit_cast(f16x8, x);
  bf16x8 h, l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = (float)v[i];
    h[i] = (__bf16)f;
    const float d = f - (float)h[i];
    l[i] = (__bf16)(__builtin_fabsf(d) < 256.f ? d : 0.f);
  }
  hi = __builtin_bit_cast(u32x4, h);
  lo = __builtin_bit_cast(u32x4, l);
}

// hi + lo of 8 fp32 values, 16 significant bits; an infinity or a NaN is hi
// alone.
__device__ inline void split_f32(u32x4 a, u32x4 b, u32x4 &hi, u32x4 &lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float h[2], l[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float v = __builtin_bit_cast(float, i < 2 ? a[2 * i + q] : b[2 * i + q - 4]);
      h[q] = (float)(__bf16)v;
      l[q] = mag_bits(h[q]) < 0x7f800000u ? v - h[q] : 0.f;
    }
    hi[i] = pack2<kBf16>(h[0], h[1]);
    lo[i] = pack2<kBf16>(l[0], l[1]);
  }
}

// The 16-bit codes of x from number `drop` on, then zeros.
__device__ inline u32x4 drop_first(u32x4 x, long long drop) {
  uint64_t lo = x[0] | (uint64_t)x[1] << 32, hi = x[2] | (uint64_t)x[3] << 32;
  const int bits = drop < 8 ? (int)drop * 16 : 128;
  if (bits >= 64) {
    lo = bits < 128 ? hi >> (bits - 64) : 0;
    hi = 0;
  } else if (bits > 0) {
    lo = lo >> bits | hi << (64 - bits);
    hi >>= bits;
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Values k .. k + 7 of a row of K 16-bit codes, zeros past K: the eight that
// end at K at the latest, moved into place.  (One load and a shift: guarded
// element loads, inlined everywhere, made kernels of 60 KB that spent their
// time on fetching instructions.)
__device__ inline u32x4 load_guarded(const unsigned char *row, long long k, int K) {
  const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
  if (K >= 8) {
    const long long from = k < K - 8 ? k : K - 8;
    return drop_first(*reinterpret_cast<const u32x4h *>(p + from), k - from);
  }
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int i = 0; k + i < K; ++i) {
    const uint64_t v = (uint64_t)p[k + i] << (16 * (i & 3));
    if (i < 4) lo |= v;
    else hi |= v;
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// 8 values of a row of 16-bit codes.  ODD: rows that may start in the middle
// of a 4-byte word, where a 16-byte load costs a multiple of an aligned one:
// the words around them are loaded, from 2 bytes before the first value on
// (the row before, or its padding: only rows after the first can be odd,
// because the matrix starts on a word), with the last value on its own.
template <bool ODD>
struct Eight {
  u32x4 v;
  __device__ __forceinline__ void load(const unsigned char *at) {
    v = *reinterpret_cast<const u32x4h *>(at);
  }
  __device__ __forceinline__ u32x4 get(const unsigned char *) const { return v; }
  __device__ __forceinline__ void set(u32x4 x, const unsigned char *) { v = x; }
};
template <>
struct Eight<true> {
  u32x4 v;
  uint32_t last;
  static __device__ __forceinline__ uint32_t shift(const unsigned char *at) {
    return ((uint32_t)(uintptr_t)at & 2u) * 8u;
  }
  __device__ __forceinline__ void load(const unsigned char *at) {
    const uintptr_t odd = reinterpret_cast<uintptr_t>(at) & 2;
    v = *reinterpret_cast<const u32x4w *>(at - odd);
    last = *reinterpret_cast<const uint16_t *>(at + 14);
  }
  __device__ __forceinline__ void set(u32x4 x, const unsigned char *at) {
    const bool odd = shift(at) != 0;
    v = odd ? u32x4{x[0] << 16, x[0] >> 16 | x[1] << 16, x[1] >> 16 | x[2] << 16,
                    x[2] >> 16 | x[3] << 16}
            : x;
    last = x[3] >> 16;
  }
  // `at`: any address of the row, for its alignment.
  __device__ __forceinline__ u32x4 get(const unsigned char *at) const {
    const uint32_t s = shift(at);
    return u32x4{__builtin_amdgcn_alignbit(v[1], v[0], s), __builtin_amdgcn_alignbit(v[2], v[1], s),
                 __builtin_amdgcn_alignbit(v[3], v[2], s), __builtin_amdgcn_alignbit(last, v[3], s)};
  }
};

// How the values of MX weights become matrix operands.  As bf16 or fp16 by
// one conversion per two values where every scale of the piece allows it:
// bf16 holds every element under scale bytes 1 to 254 (0.5 2^-126 is a
// subnormal that it holds exactly), fp16 under 104 to 140 (0.5 2^-23 is its
// smallest step, 6 2^13 below its largest value).  Otherwise through fp32.
enum Widen { kToBf16, kToF16, kThroughF32 };
template <Widen HOW>
__device__ inline u32x4 widen(uint32_t codes, uint32_t sb) {
  if constexpr (HOW == kToBf16) {
    const float unit = __builtin_bit_cast(float, sb << 23);
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 0);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 1);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 2);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 3);
    return u32x4{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                 __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
  } else if constexpr (HOW == kToF16) {
    const float unit = __builtin_bit_cast(float, sb << 23);
    const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, unit, 0);
    const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, unit, 1);
    const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, unit, 2);
    const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, unit, 3);
    return u32x4{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                 __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
  } else {
    float v[8];
    decode8(codes, sb, v);
    return u32x4{pack2<kBf16>(v[0], v[1]), pack2<kBf16>(v[2], v[3]), pack2<kBf16>(v[4], v[5]),
                 pack2<kBf16>(v[6], v[7])};
  }
}

// The wave's number in its workgroup, as a scalar.
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// ---- weights -----------------------------------------------------------------
//
// Lane l loads 16 bytes number l % 4 of 64 of row l / 4: lanes that each read
// the row they need, l % 16, cost the L1 an access each, four that read one
// line of a row one between them (gemm_mx_a16, 32 x 16384 x 8192: 27.7 us
// against 21.7).  What lane l needs, number l / 16 of row l % 16, then comes
// from lane 4 (l % 16) + l / 16.

__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * lane, (int)v);
}
__device__ __forceinline__ u32x4 from_lane(u32x4 v, int lane) {
  return u32x4{from_lane(v[0], lane), from_lane(v[1], lane), from_lane(v[2], lane),
               from_lane(v[3], lane)};
}
// The lane whose load holds this lane's operand.
__device__ __forceinline__ int loader(int lane) { return 4 * (lane & 15) + (lane >> 4); }

// Row l / 4 of a block of 16 rows: 2-byte values or MX codes, and MX scales.
struct Row {
  const unsigned char *p;
  const unsigned char *q;
};

// A piece of 16 MX rows as loaded: blocks 16 piece + 4 i + l % 4, and scales
// 4 (l % 4) .. + 3 of the piece.  Blocks past the row's are read from its last.
struct MxPiece {
  u32x4 c[4];
  uint32_t s;
  __device__ __forceinline__ void load(const Row &r, int piece, int lane, int nb) {
    s = *reinterpret_cast<const uint32_t *>(r.q + 16LL * piece + 4 * (lane & 3));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kb = 16 * piece + 4 * i + (lane & 3);
      c[i] = *reinterpret_cast<const u32x4 *>(r.p + 16LL * (kb < nb ? kb : nb - 1));
    }
  }
};
// Its operands: blocks 16 piece + 4 i + l / 16 of row l % 16 and their scales;
// blocks past the row's are zeros with scale 1.
struct MxBlocks {
  u32x4 c[4];
  uint32_t s[4];
  __device__ __forceinline__ MxBlocks(const MxPiece &x, int piece, int lane, int nb) {
    const int g = lane >> 4, from = loader(lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = from_lane(x.c[i], from);
      s[i] = from_lane(x.s, 4 * (lane & 15) + i) >> (8 * g) & 255u;
    }
    if (16 * (piece + 1) > nb) {  // uniform
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * piece + 4 * i + g >= nb) {
          c[i] = u32x4{0, 0, 0, 0};
          s[i] = 127u;
        }
    }
  }
  // Whether all of the lane's blocks have scales within (blocks of zeros allow any).
  template <uint32_t LOW, uint32_t HIGH>
  __device__ __forceinline__ bool within() const {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ok &= s[i] - LOW <= HIGH - LOW || (s[i] != 255 && (c[i][0] | c[i][1] | c[i][2] | c[i][3]) == 0);
    return ok;
  }
};

// ---- activations in LDS --------------------------------------------------------
//
// Blocks of up to 16 rows, `rows` of them kept (4 or 16), of kc values: for
// each operand of a matrix instruction (piece, step, MFMA j) and lane group,
// the rows' 16 bytes one after the other, and 16 bytes of padding, so that
// neither the writes (neighbouring threads take neighbouring k of a row) nor
// the reads (16 lanes take 16 rows) meet on a bank.  kF32: a second such
// plane for lo.

struct Tile {
  int rows, kc;
  __host__ __device__ int group() const { return 16 * rows + 16; }
};
// LDS bytes of a block of rows of kind A: linear in kc (whole pieces).
template <int A>
__host__ __device__ inline int act_bytes(const Tile &t) {
  return t.kc / 8 * t.group() * (A == kF32 ? 2 : 1);
}

// Fills a block with values k0 .. k0 + kc - 1 of rows 0 .. n - 1, zeros past K;
// `row(r)` gives row r's start.  All THREADS
// threads of the workgroup take part; each issues four loads before it writes
// any (one at a time, their latencies alone took 30 us of a first product).
// Rows of kind kF32 hold zeros from K to a multiple of 8.
template <int A, int W, bool ODD, int THREADS, class RowOf>
__device__ __forceinline__ void stage_acts(unsigned char *lds, const Tile &t, RowOf row, int n,
                                           int k0, int K) {
  constexpr int kBatch = 4;
  const int G = t.group();
  const int per = t.kc / 8, all = n * per, eights = (int)ceil_div(K, 8);
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < all; i0 += kBatch * THREADS) {
    u32x4 c[kBatch], d[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * THREADS < all ? i0 + u * THREADS : all - 1;
      const int r = i / per, x = i % per;
      const Row src = row(r);
      if constexpr (A == kF32) {
        const int e = k0 / 8 + x, in = e < eights ? e : eights - 1;
        const u32x4w *q = reinterpret_cast<const u32x4w *>(src.p + 32LL * in);
        c[u] = q[0];
        d[u] = q[1];
      } else {
        const long long k = k0 + 8LL * x;
        if constexpr (ODD) {
          if (k + 8 <= K) {
            Eight<true> v;
            v.load(src.p + 2 * k);
            c[u] = v.v;
            d[u][0] = v.last;
          }
        } else if (k + 8 <= K) {
          c[u] = *reinterpret_cast<const u32x4h *>(src.p + 2 * k);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * THREADS;
      if (i >= all) continue;
      const int r = i / per, x = i % per;
      {
        // Operand and lane group of values 8 x .. 8 x + 7: the MX order of k
        // is (step, g, j), the 16-bit one (j, g).
        const int group = W == kMx ? (x & ~15) | (x & 3) << 2 | (x >> 2 & 3) : x;
        u32x4 *to = reinterpret_cast<u32x4 *>(lds + group * G + 16 * r);
        if constexpr (A == kF32) {
          const bool in = k0 / 8 + x < eights;
          u32x4 hi, lo;
          split_f32(c[u], d[u], hi, lo);
          *to = in ? hi : u32x4{0, 0, 0, 0};
          *reinterpret_cast<u32x4 *>(lds + per * G + group * G + 16 * r) =
              in ? lo : u32x4{0, 0, 0, 0};
        } else {
          const long long k = k0 + 8LL * x;
          if (k + 8 > K) {
            c[u] = load_guarded(row(r).p, k < K ? k : K, K);
          } else if constexpr (ODD) {
            Eight<true> v;
            v.v = c[u];
            v.last = d[u][0];
            c[u] = v.get(row(r).p);
          }
          *to = c[u];
        }
      }
    }
  }
}

// ---- the product -----------------------------------------------------------------

// MB blocks of rows of kind A in LDS by NB blocks of 16 rows of weights of
// kind W in registers.
template <int W, int A, int MB, int NB, bool ODD>
struct Thin {
  static constexpr int kK = kPieceK<W>, kSteps = kPieceSteps<W>;
  struct Weights {
    MxPiece mx[W == kMx ? NB : 1];
    Eight<ODD> half[W == kMx ? 1 : NB][4];
  };
  f32x4 acc[MB][NB];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // A piece's weights, zeros past K.
  static __device__ __forceinline__ void load(Weights &x, const Row (&w)[NB], int piece, int lane,
                                              int K) {
    const int nb = (int)mx_blocks(K);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (W == kMx) {
        x.mx[b].load(w[b], piece, lane, nb);
      } else {
        const long long k0 = (long long)kK * piece + 8 * (lane & 3);
        if (piece < K / kK) {  // uniform
#pragma unroll
          for (int j = 0; j < 4; ++j) x.half[b][j].load(w[b].p + 2 * (k0 + 32 * j));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const long long k = k0 + 32 * j;
            x.half[b][j].set(load_guarded(w[b].p, k < K ? k : K, K), w[b].p);
          }
        }
      }
    }
  }

  // The products of a loaded piece, number `local` of the tile.
  __device__ __forceinline__ void use(const Weights &x, const Row (&w)[NB],
                                      const unsigned char *lds, const Tile &t, int local, int piece,
                                      int lane, int K) {
    const int g = lane >> 4, r = lane & (t.rows - 1), G = t.group(), block = act_bytes<A>(t);
    constexpr Widen kHow = W == kF16 || (W == kMx && A == kF16) ? kToF16 : kToBf16;
    const unsigned char *from = lds + (local * kSteps * 16 + g) * G + 16 * r;
    const int lo = t.kc / 8 * G;
    if constexpr (W != kMx) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 wv[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) wv[b] = from_lane(x.half[b][j].get(w[b].p), loader(lane));
        multiply<kHow>(wv, from + j * 4 * G, block, lo);
      }
    } else {
      const MxBlocks y0(x.mx[0], piece, lane, (int)mx_blocks(K));
      const MxBlocks y1(x.mx[NB - 1], piece, lane, (int)mx_blocks(K));
      const MxBlocks *y[2] = {&y0, &y1};
      bool ok = true;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        ok &= A == kF16 ? y[b]->template within<104, 140>() : y[b]->template within<1, 254>();
      if (__all(ok)) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            u32x4 wv[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) wv[b] = widen<kHow>(y[b]->c[s][j], y[b]->s[s]);
            multiply<kHow>(wv, from + (4 * s + j) * 4 * G, block, lo);
          }
      } else {
        // Rare, and kept short: a loop over the piece's words.
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          u32x4 wv[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t c = 0, sb = 0;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              if (q == i) c = y[b]->c[q >> 2][q & 3];
              if (q == i) sb = y[b]->s[q >> 2];
            }
            wv[b] = widen<kThroughF32>(c, sb);
          }
          multiply<kThroughF32>(wv, from + i * 4 * G, block, lo);
        }
      }
    }
  }

  // One matrix operand's products; `at`: the lane's activations in LDS.  HOW:
  // the format that the weights come in or were brought to.
  template <Widen HOW>
  __device__ __forceinline__ void multiply(const u32x4 (&wv)[NB], const unsigned char *at,
                                           int block, int lo_plane) {
    constexpr bool kSplitHere = A == kF16 && HOW != kToF16;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      u32x4 v = *reinterpret_cast<const u32x4 *>(at + i * block), lo{};
      if constexpr (A == kF32) lo = *reinterpret_cast<const u32x4 *>(at + i * block + lo_plane);
      if constexpr (kSplitHere) split_f16(v, v, lo);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (A == kF32 && HOW == kToF16) {
          // fp16 weights are split too; the product of the two low parts,
          // 2^-18 of the whole, is left out
          u32x4 wh, wl;
          split_f16(wv[b], wh, wl);
          acc[i][b] = mfma_bf16(wh, v, acc[i][b]);
          acc[i][b] = mfma_bf16(wh, lo, acc[i][b]);
          acc[i][b] = mfma_bf16(wl, v, acc[i][b]);
        } else if constexpr (HOW == kToF16) {
          acc[i][b] = mfma_f16(wv[b], v, acc[i][b]);
        } else {
          acc[i][b] = mfma_bf16(wv[b], v, acc[i][b]);
          if constexpr (A == kF32 || kSplitHere) acc[i][b] = mfma_bf16(wv[b], lo, acc[i][b]);
        }
      }
    }
  }

  // How a workgroup's waves go through K.
  struct Walk {
    int first, ks;  // this wave takes pieces first, first + ks, ...
    bool any;       // whether this wave has columns at all
    bool staged;    // the tile already holds all of K
  };
  // Adds all K values, from `x`, which holds the wave's first piece, on.  At
  // the end `x` holds the first piece of the rows `next`.  `row(r)` gives row
  // r of n activations.  Every wave of the workgroup makes the call.
  template <int THREADS, class RowOf>
  __device__ __forceinline__ void run(unsigned char *lds, const Tile &t, RowOf row, int n,
                                      const Row (&w)[NB], const Row (&next)[NB], Weights &x,
                                      const Walk &at, int K, int lane) {
    const int pieces = (int)ceil_div(K, kK);
    const int rounds = (int)ceil_div(pieces, at.ks), per = t.kc / (kK * at.ks);
    const int block = act_bytes<A>(t);
#pragma unroll 1
    for (int i0 = 0; i0 < rounds; i0 += per) {
      if (!at.staged) {
        __syncthreads();
#pragma unroll 1
        for (int m = 0; m < MB && n > 16 * m; ++m)
          stage_acts<A, W, ODD, THREADS>(
              lds + m * block, t, [&](int r) { return row(16 * m + r); },
              n - 16 * m < 16 ? n - 16 * m : 16, i0 * at.ks * kK, K);
        __syncthreads();
      }
      if (!at.any) continue;
      const int end = i0 + per < rounds ? i0 + per : rounds;
#pragma unroll 1
      for (int i = i0; i < end; ++i) {
        const int p = at.first + i * at.ks;
        const bool last = i + 1 == rounds;
        const int q = last ? (at.first < pieces ? at.first : 0) : p + at.ks < pieces ? p + at.ks : 0;
        Row from[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) from[b] = last ? next[b] : w[b];
        Weights y;
        load(y, from, q, lane, K);
        if (p < pieces) use(x, w, lds, t, (i - i0) * at.ks + at.first, p, lane, K);
        x = y;  // the next piece, needed at once
      }
    }
  }
  static __device__ __forceinline__ void load_first(Weights &x, const Row (&w)[NB], const Walk &at,
                                                    int K, int lane) {
    const int pieces = (int)ceil_div(K, kK);
    if (at.any) load(x, w, at.first < pieces ? at.first : 0, lane, K);
  }
};

// The same product of one block of rows with the activations straight from
// memory, for products so small that what counts is the latency: a piece's
// weights and activations are asked for together, both by four lanes to a
// line.  MFMA m of step s takes block 4 s + m of the piece here, lane l its
// values 8 (l / 16) .. + 7, so that one lane's load holds one lane's operand.
template <int A, bool ODD>
struct Direct {
  f32x4 acc;
  // The products of 8 values per lane, of MX words that allow `kHow` or not.
  template <Widen HOW>
  __device__ __forceinline__ void add(uint32_t codes, uint32_t sb, u32x4 v) {
    const u32x4 wv = widen<HOW>(codes, sb);
    if constexpr (HOW == kToF16) {
      acc = mfma_f16(wv, v, acc);
    } else {
      u32x4 lo{};
      if constexpr (A == kF16) split_f16(v, v, lo);
      acc = mfma_bf16(wv, v, acc);
      if constexpr (A == kF16) acc = mfma_bf16(wv, lo, acc);
    }
  }
  // `w`, `a`: rows l / 4 of the weights and the activations.
  __device__ __forceinline__ void piece(const Row &w, const unsigned char *a, int piece, int lane,
                                        int K) {
    const int from = loader(lane), part = lane & 3, nb = (int)mx_blocks(K);
    const uint32_t s = *reinterpret_cast<const uint32_t *>(w.q + 16LL * piece + 4 * part);
    if (512LL * (piece + 1) <= K) {  // uniform
      uint32_t c[16], sc[4];
      Eight<ODD> v[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        c[q] = *reinterpret_cast<const uint32_t *>(w.p + 16 * (16LL * piece + q) + 4 * part);
        v[q].load(a + 2 * (32 * (16LL * piece + q) + 8 * part));
      }
      bool ok = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[i] = from_lane(s, 4 * (lane & 15) + i);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t sb = sc[i] >> (8 * m) & 255u;
          ok &= A == kF16 ? sb - 104u <= 140u - 104u : sb - 1u <= 253u;
        }
      }
      if (__all(ok)) {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          add<A == kF16 ? kToF16 : kToBf16>(from_lane(c[q], from), sc[q >> 2] >> (8 * (q & 3)) & 255u,
                                            from_lane(v[q].get(a), from));
        return;
      }
    }
    // K's end, or scales far from 1: block by block, through fp32.
#pragma unroll 1
    for (int q = 0; q < 16; ++q) {
      const int kb = 16 * piece + q;
      if (kb >= nb) break;
      const uint32_t c = *reinterpret_cast<const uint32_t *>(w.p + 16LL * kb + 4 * part);
      const long long k = 32LL * kb + 8 * part;
      add<kThroughF32>(from_lane(c, from),
                       from_lane(s, 4 * (lane & 15) + (q >> 2)) >> (8 * (q & 3)) & 255u,
                       from_lane(load_guarded(a, k < K ? k : K, K), from));
    }
  }
};

// Waves per group of columns: until the groups' waves fill the chip (`want`),
// or each has a piece.
inline int waves_per_group(long long groups, int K, int piece, int most, int want) {
  int ks = 1;
  while (ks < most && groups * ks < want && (long long)2 * ks * piece <= K) ks *= 2;
  return ks;
}
// Values of the activations' tile: all of K where it fits `bytes`, else as many
// whole rounds (pieces of all waves that share columns) as do, one at least.
template <int A>
__host__ __device__ inline int tile_values(int rows, int K, int round, int bytes) {
  const int all = (int)ceil_div(K, round), fit = bytes / act_bytes<A>(Tile{rows, round});
  return round * (all < fit ? all : fit > 1 ? fit : 1);
}

}  // namespace
}  // namespace gemm_f32_impl
