// Pieces of the thin products (few rows of gemm_mx, gemm_mx_a16, the
// mixture-of-experts layer): up to 32 rows of activations against weights
// read once from memory, which is what bounds them.
//
// A wave multiplies blocks of 16 activation rows with blocks of 16 weight
// rows ("columns" of C) and takes K in pieces of four 128-deep steps (MX
// weights) or one (16-bit ones).  A piece's weights are loaded at once, the
// activations step by step, a step ahead of their use.  Rows past the last
// are not loaded: with the usual few rows most lanes are spared the L1
// traffic, of which 16-bit activations need four times what MX weights do.
//
// Lane l holds row l % 16 of each operand; which k a lane holds is free as
// long as both operands agree, so it follows how the weights are stored, with
// g = l / 16:
//   MX weights: load s of a piece is block 4 s + g of it; MFMA j of step s
//     takes its values 8 j .. 8 j + 7, widened with their scale (exact: an
//     element has two significant bits);
//   16-bit weights: load j of a step is k = 32 j + 8 g .. + 7, the operand of
//     MFMA j.
#pragma once

#include "mx_values.hpp"

namespace gemm_f32_impl {
namespace {

// Kinds of operands: the formats of mx_plan.hpp, MX rows, and activations
// kept as a sum of two bf16 terms.
constexpr int kMx = 3, kSplit = 4;

// One row of an operand: 2-byte values or MX codes; scales of an MX row; the
// second term of a split one.
struct Row {
  const unsigned char *p;
  const unsigned char *q;
};

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

// 8 values of a row of 16-bit codes from k, the first `n` of them (others 0).
__device__ inline u32x4 load_guarded(const unsigned char *row, long long k, long long n) {
  const uint16_t *p = reinterpret_cast<const uint16_t *>(row) + k;
  if (n >= 8) return *reinterpret_cast<const u32x4h *>(p);
  u32x4 w{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return w;
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

// A piece of an MX row as it is stored: blocks 16 piece + 4 s + g and the 16
// scales.  Blocks past the row's are read from its last; mask_mx_piece makes
// them zeros with scale 1.
struct MxPiece {
  u32x4 c[4];
  u32x4 s;
};
__device__ __forceinline__ void load_mx_piece(MxPiece &x, const Row &r, int piece, int g, int nb) {
  x.s = *reinterpret_cast<const u32x4 *>(r.q + 16LL * piece);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int kb = 16 * piece + 4 * s + g < nb ? 16 * piece + 4 * s + g : nb - 1;
    x.c[s] = *reinterpret_cast<const u32x4 *>(r.p + 16LL * kb);
  }
}
__device__ __forceinline__ void mask_mx_piece(MxPiece &x, int piece, int g, int nb) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (16 * piece + 4 * s + g >= nb) {
      x.c[s] = u32x4{0, 0, 0, 0};
      x.s[s] = 0x7f7f7f7fu;
    }
}
// Lane group g's scale byte of step s.
__device__ inline uint32_t piece_scale(const MxPiece &x, int s, int g) {
  return (x.s[s] >> (8 * g)) & 255u;
}

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
// Whether all of a lane's blocks allow it (blocks of zeros allow any).
template <uint32_t LOW, uint32_t HIGH>
__device__ inline bool scales_within(const MxPiece &x, int g) {
  bool ok = true;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const u32x4 c = x.c[s];
    const uint32_t sb = piece_scale(x, s, g);
    ok &= sb - LOW <= HIGH - LOW || (sb != 255 && (c[0] | c[1] | c[2] | c[3]) == 0);
  }
  return ok;
}

// The wave's number in its workgroup, as a scalar.
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// First k (from the piece's first) of lane group g's operand of MFMA j of
// step s.
template <int W>
__device__ inline int piece_k(int g, int s, int j) {
  return 128 * s + (W == kMx ? 32 * g + 8 * j : 32 * j + 8 * g);
}

// One product of thin operands: MB blocks of 16 rows of kind A by NB blocks
// of 16 rows of weights of kind W.
template <int W, int A, int MB, int NB, bool ODD = false>
struct Thin {
  static constexpr int kK = kPieceK<W>, kSteps = kPieceSteps<W>;
  struct Weights {
    MxPiece mx[W == kMx ? NB : 1];
    Eight<ODD> half[W == kMx ? 1 : NB][4];
  };
  // Activations of one step (16-bit or split), or of a piece (MX).
  struct Acts {
    MxPiece mx[A == kMx ? MB : 1];
    Eight<ODD && A != kSplit> v[A == kMx ? 1 : MB][4];
    Eight<false> lo[A == kSplit ? MB : 1][4];
  };
  f32x4 acc[MB][NB];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // A piece's weights; with TAIL it reaches past K: zeros there.
  template <bool TAIL>
  static __device__ __forceinline__ void load_weights(Weights &x, const Row (&w)[NB], int piece,
                                                      int g, int K, int nb) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (W == kMx) {
        load_mx_piece(x.mx[b], w[b], piece, g, nb);
        if constexpr (TAIL) mask_mx_piece(x.mx[b], piece, g, nb);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const long long k = (long long)kK * piece + piece_k<W>(g, 0, j);
          if constexpr (TAIL) x.half[b][j].set(load_guarded(w[b].p, k, K - k), w[b].p);
          else x.half[b][j].load(w[b].p + 2 * k);
        }
      }
    }
  }
  // Step s of a piece's activations.  Rows that `valid` leaves out are not
  // loaded: their results are not used.  Split ones are padded with zeros to
  // whole pieces.
  template <bool TAIL>
  static __device__ __forceinline__ void load_acts(Acts &y, const Row (&a)[MB],
                                                   const bool (&valid)[MB], int piece, int s,
                                                   int g, int K, int nb) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
      if (valid[i]) {
        if constexpr (A == kMx) {
          load_mx_piece(y.mx[i], a[i], piece, g, nb);
          if constexpr (TAIL) mask_mx_piece(y.mx[i], piece, g, nb);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const long long k = (long long)kK * piece + piece_k<W>(g, s, j);
            if constexpr (A == kSplit) {
              y.v[i][j].load(a[i].p + 2 * k);
              y.lo[i][j].load(a[i].q + 2 * k);
            } else if constexpr (TAIL) {
              y.v[i][j].set(load_guarded(a[i].p, k, K - k), a[i].p);
            } else {
              y.v[i][j].load(a[i].p + 2 * k);
            }
          }
        }
      }
  }

  // The products of a piece whose weights are loaded.
  template <bool TAIL>
  __device__ __forceinline__ void use(const Weights &x, const Row (&w)[NB], const Row (&a)[MB],
                                      const bool (&valid)[MB], int piece, int g, int K, int nb) {
    if constexpr (A == kMx) {
      Acts y;
      load_acts<TAIL>(y, a, valid, piece, 0, g, K, nb);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[i][b] = mfma_mx(x.mx[b].c[s], (int)piece_scale(x.mx[b], s, g), y.mx[i].c[s],
                                (int)piece_scale(y.mx[i], s, g), acc[i][b]);
    } else {
      Acts y[2];
      load_acts<TAIL>(y[0], a, valid, piece, 0, g, K, nb);
      bool ok = true;
      if constexpr (W == kMx) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          ok &= A == kF16 ? scales_within<104, 140>(x.mx[b], g) : scales_within<1, 254>(x.mx[b], g);
        ok = __all(ok);
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s + 1 < kSteps) load_acts<TAIL>(y[(s + 1) & 1], a, valid, piece, s + 1, g, K, nb);
        __builtin_amdgcn_sched_barrier(0);
        constexpr Widen kHow = W == kF16 || (W == kMx && A == kF16) ? kToF16 : kToBf16;
        if (W != kMx || ok) multiply<kHow>(x, y[s & 1], w, a, s, g);
        else multiply<kThroughF32>(x, y[s & 1], w, a, s, g);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // One step's products.  HOW: the format the weights come in or are brought to.
  template <Widen HOW>
  __device__ __forceinline__ void multiply(const Weights &x, const Acts &y, const Row (&w)[NB],
                                           const Row (&a)[MB], int s, int g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 wv[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (W == kMx) wv[b] = widen<HOW>(x.mx[b].c[s][j], piece_scale(x.mx[b], s, g));
        else wv[b] = x.half[b][j].get(w[b].p);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        u32x4 v = y.v[i][j].get(a[i].p), lo{};
        if constexpr (A == kSplit) lo = y.lo[i][j].get(a[i].q);
        constexpr bool kSplitHere = A == kF16 && HOW != kToF16;
        if constexpr (kSplitHere) split_f16(v, v, lo);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (A == kSplit && HOW == kToF16) {
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
            if constexpr (A == kSplit || kSplitHere) acc[i][b] = mfma_bf16(wv[b], lo, acc[i][b]);
          }
        }
      }
    }
  }

  // Adds the products of pieces first, first + step, ... of the K values.
  __device__ __forceinline__ void run(const Row (&a)[MB], const bool (&valid)[MB],
                                      const Row (&w)[NB], int first, int step, int K, int g) {
    const int nb = (int)mx_blocks(K), last = K / kK;  // whole pieces
    int p = first;
#pragma unroll 1
    for (; p < last; p += step) {
      Weights x;
      load_weights<false>(x, w, p, g, K, nb);
      use<false>(x, w, a, valid, p, g, K, nb);
    }
    if (p == last && (long long)last * kK < K) {
      Weights x;
      load_weights<true>(x, w, p, g, K, nb);
      use<true>(x, w, a, valid, p, g, K, nb);
    }
  }
};

}  // namespace
}  // namespace gemm_f32_impl
