// Pieces of the thin products (few rows of gemm_mx, gemm_mx_a16, the
// mixture-of-experts layer): up to 64 rows of activations against weights
// read once from memory, which is what bounds them.
//
// A wave multiplies blocks of 16 activation rows with blocks of 16 weight
// rows ("columns" of C) and takes K in pieces of four 16-byte loads per
// weight row: 512 k of MX weights, 128 k of 16-bit ones.  A piece's weights
// are loaded whole before any is used and the next piece's while it is used,
// so a wave keeps 4 KB or more per 16 weight rows in flight.
//
// Lane l holds row l % 16 of each operand; which k a lane holds is free as
// long as both operands agree, so it follows how the weights are stored, with
// g = l / 16:
//   MX weights: load s of a piece is block 4 s + g of the row; MFMA j of the
//     128-deep step s takes its values 8 j .. 8 j + 7, widened with their
//     scale (exact: an element has two significant bits);
//   16-bit weights: load j is k = 32 j + 8 g .. + 7, the operand of MFMA j.
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

// A piece of an MX row as it is stored: blocks 16 piece + 4 s + g and the 16
// scales.  Blocks past the row's are read from its last and made zeros with
// scale 1.
struct MxPiece {
  u32x4 c[4];
  u32x4 s;
};
__device__ inline MxPiece load_mx_piece(const Row &r, int piece, int g, int nb) {
  MxPiece x;
  const int kb0 = 16 * piece + g;
  x.s = *reinterpret_cast<const u32x4 *>(r.q + 16LL * piece);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int kb = kb0 + 4 * s < nb ? kb0 + 4 * s : nb - 1;
    x.c[s] = *reinterpret_cast<const u32x4 *>(r.p + 16LL * kb);
  }
  return x;
}
__device__ inline void mask_mx_piece(MxPiece &x, int piece, int g, int nb) {
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
// Whether all of a lane's four blocks allow it (blocks of zeros allow any).
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

// A piece of 16-bit weights: operands of MFMA 0 .. 3.
struct HalfPiece {
  u32x4 c[4];
};
__device__ inline HalfPiece load_half_piece(const Row &r, int piece, int g) {
  HalfPiece x;
  const uint16_t *p = reinterpret_cast<const uint16_t *>(r.p) + 128LL * piece + 8 * g;
#pragma unroll
  for (int j = 0; j < 4; ++j) x.c[j] = *reinterpret_cast<const u32x4h *>(p + 32 * j);
  return x;
}
__device__ inline HalfPiece load_half_guarded(const Row &r, int piece, int g, int K) {
  HalfPiece x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long k = 128LL * piece + 32 * j + 8 * g;
    x.c[j] = load_guarded(r.p, k, K - k);
  }
  return x;
}

template <int W>
struct PieceOf {
  typedef HalfPiece type;
};
template <>
struct PieceOf<kMx> {
  typedef MxPiece type;
};

// First k (from the piece's first) of lane group g's operand of MFMA j of
// step s.
template <int W>
__device__ inline int piece_k(int g, int s, int j) {
  return W == kMx ? 128 * s + 32 * g + 8 * j : 32 * j + 8 * g;
}

// The wave's number in its workgroup, as a scalar.
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// One product of thin operands: MB blocks of 16 rows of kind A by NB blocks
// of 16 rows of weights of kind W.  `mine` says which pieces this wave takes:
// first, first + step, ... below `pieces`.
template <int W, int A, int MB, int NB>
struct Thin {
  typedef typename PieceOf<W>::type Piece;
  f32x4 acc[MB][NB];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  static __device__ __forceinline__ void load(Piece (&x)[NB], const Row (&w)[NB], int piece, int g,
                                              int K, int nb) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (W == kMx) x[b] = load_mx_piece(w[b], piece, g, nb);
      else x[b] = load_half_piece(w[b], piece, g);
    }
  }

  // The products of one piece.  With GUARD it may reach past K.
  template <bool GUARD>
  __device__ __forceinline__ void use(Piece (&x)[NB], const Row (&a)[MB], int piece, int g, int K,
                                      int nb) {
    if constexpr (W == kMx && GUARD) {
#pragma unroll
      for (int b = 0; b < NB; ++b) mask_mx_piece(x[b], piece, g, nb);
    }
    if constexpr (A == kMx) {
      MxPiece y[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        y[i] = load_mx_piece(a[i], piece, g, nb);
        if constexpr (GUARD) mask_mx_piece(y[i], piece, g, nb);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[i][b] = mfma_mx(x[b].c[s], (int)piece_scale(x[b], s, g), y[i].c[s],
                                (int)piece_scale(y[i], s, g), acc[i][b]);
    } else if constexpr (W == kMx) {
      bool wide = true, half = A == kF16;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        wide &= scales_within<1, 254>(x[b], g);
        if constexpr (A == kF16) half &= scales_within<104, 140>(x[b], g);
      }
      if (A == kF16 && __all(half)) multiply<GUARD, kToF16>(x, a, piece, g, K);
      else if (A != kF16 && __all(wide)) multiply<GUARD, kToBf16>(x, a, piece, g, K);
      else multiply<GUARD, kThroughF32>(x, a, piece, g, K);
    } else {
      multiply<GUARD, W == kF16 ? kToF16 : kToBf16>(x, a, piece, g, K);
    }
  }

  // HOW: the format the weights come in or are brought to.
  template <bool GUARD, Widen HOW>
  __device__ __forceinline__ void multiply(const Piece (&x)[NB], const Row (&a)[MB], int piece,
                                           int g, int K) {
#pragma unroll
    for (int s = 0; s < kPieceSteps<W>; ++s) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 w[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (W == kMx) w[b] = widen<HOW>(x[b].c[s][j], piece_scale(x[b], s, g));
          else w[b] = x[b].c[j];
        }
        const long long k = (long long)kPieceK<W> * piece + piece_k<W>(g, s, j);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          u32x4 v, lo;
          if constexpr (A == kSplit) {  // rows padded with zeros to whole 512 k
            v = *reinterpret_cast<const u32x4 *>(a[i].p + 2 * k);
            lo = *reinterpret_cast<const u32x4 *>(a[i].q + 2 * k);
          } else {
            if constexpr (GUARD) v = load_guarded(a[i].p, k, K - k);
            else v = *reinterpret_cast<const u32x4h *>(a[i].p + 2 * k);
            if constexpr (A == kF16 && HOW != kToF16) split_f16(v, v, lo);
          }
          constexpr bool kTwo = A == kSplit || (A == kF16 && HOW != kToF16);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if constexpr (kTwo && HOW == kToF16) {
              // fp16 weights are split too; the product of the two low
              // parts, 2^-18 of the whole, is left out
              u32x4 wh, wl;
              split_f16(w[b], wh, wl);
              acc[i][b] = mfma_bf16(wh, v, acc[i][b]);
              acc[i][b] = mfma_bf16(wh, lo, acc[i][b]);
              acc[i][b] = mfma_bf16(wl, v, acc[i][b]);
            } else if constexpr (HOW == kToF16) {
              acc[i][b] = mfma_f16(w[b], v, acc[i][b]);
            } else {
              acc[i][b] = mfma_bf16(w[b], v, acc[i][b]);
              if constexpr (kTwo) acc[i][b] = mfma_bf16(w[b], lo, acc[i][b]);
            }
          }
        }
      }
      // One step's activations at a time: hoisted all together their
      // registers would cost the waves that hide their latency.
      if constexpr (kPieceSteps<W> > 1) __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Adds this wave's pieces first, first + step, ... below `end` of the K
  // values of rows `a` and `w`.
  __device__ __forceinline__ void run(const Row (&a)[MB], const Row (&w)[NB], int first, int step,
                                      int end, int K, int g) {
    const int nb = (int)mx_blocks(K), whole = K / kPieceK<W>;
    const int last = end < whole ? end : whole;  // whole pieces below `end`
    int p = first;
    Piece x[NB];
    if (p < last) load(x, w, p, g, K, nb);
    if constexpr (W == kMx && NB > 1) {  // 8 KB or more in flight; registers for waves instead
      for (; p < last; p += step) {
        use<false>(x, a, p, g, K, nb);
        load(x, w, p + step < last ? p + step : p, g, K, nb);
      }
    } else {
      // Two pieces by turns: handing the loaded one on in registers would
      // wait for it.
      Piece y[NB];
      while (p < last) {
        load(y, w, p + step < last ? p + step : p, g, K, nb);
        use<false>(x, a, p, g, K, nb);
        p += step;
        if (p >= last) break;
        load(x, w, p + step < last ? p + step : p, g, K, nb);
        use<false>(y, a, p, g, K, nb);
        p += step;
      }
    }
    if (p < end) {  // the piece that reaches past K
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (W == kMx) x[b] = load_mx_piece(w[b], p, g, nb);
        else x[b] = load_half_guarded(w[b], p, g, K);
      }
      use<true>(x, a, p, g, K, nb);
    }
  }
};

}  // namespace
}  // namespace gemm_f32_impl
