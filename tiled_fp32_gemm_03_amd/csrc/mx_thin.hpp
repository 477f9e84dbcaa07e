// Pieces of the thin products (few rows of gemm_mx, gemm_mx_a16, the
// mixture-of-experts layer): up to 32 rows of activations against weights
// read once from memory, which is what bounds them.
//
// A wave multiplies blocks of 16 activation rows with blocks of 16 weight
// rows ("columns" of C) and takes K in pieces of 256 bytes of weight row:
// four 128-deep steps of MX weights, one of 16-bit ones.  A piece's weights
// are loaded at once, the activations step by step, a step ahead of their
// use.
//
// The matrix instructions want lane l to hold row l % 16, but four
// neighbouring lanes that read four rows cost the L1 four accesses where
// four that read 64 bytes of one row cost it one, and the L1's accesses were
// what bounded these kernels (a second product of 143 MB took 70 us with 21
// accesses per load).  So lane l loads 16 bytes number l % 4 (of group g = l /
// 16) of rows 4 (l / 4 % 4) + t, t = 0 .. 3, and a 4 x 4 transpose inside each
// four lanes brings row l % 16's four into the lane: 32 ALU operations per
// 4 KB.  Lane l then holds 64 consecutive bytes of its row, which decides the
// order of k (any order is as good as both operands agree):
//   MX weights: blocks 4 g + s of a piece's 16, s its step; MFMA j takes the
//     block's values 8 j .. 8 j + 7, widened with their scale (exact: an
//     element has two significant bits);
//   16-bit weights: MFMA j takes k = 32 g + 8 j .. + 7.
// The activations are read as their lanes hold them, valid rows alone; with
// few rows that is few accesses.  The layer's inner values, which its first
// product writes for its second, are kept in the order of these loads.
#pragma once

#include "mx_values.hpp"

#include <type_traits>

namespace gemm_f32_impl {
namespace {

// Kinds of operands: the formats of mx_plan.hpp, MX rows, and activations
// kept as a sum of two bf16 terms.
constexpr int kMx = 3, kSplit = 4;

// Where lane l loads 16 rows of weights: rows 4 (l / 4 % 4) + t, as 2-byte
// values or MX codes, and the scales of row l % 16 (MX).
struct Rows {
  const unsigned char *p[4];
  const unsigned char *q;
};
// Activations: the lane's row l % 16 of 2-byte values; of MX rows as weights;
// of a split operand the lane's place in its two planes.
struct Row {
  const unsigned char *p;
  const unsigned char *q;
};
template <int A>
struct ActRow {
  typedef Row type;
};
template <>
struct ActRow<kMx> {
  typedef Rows type;
};
// Row t of those that this lane loads, and the row it holds.
__device__ inline int load_row(int lane, int t) { return (lane & 12) + t; }

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

// The 4 x 4 transpose inside each four lanes: lane i's r[t] goes to lane t's
// r[i].
template <int CTRL>
__device__ inline uint32_t quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ void quad_transpose(u32x4 (&r)[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
#pragma unroll
    for (int t = 0; t < 4; t += 2) {  // lanes i, i ^ 1 and registers t, t + 1
      const uint32_t a = r[t][d], b = r[t + 1][d], fa = quad<0xB1>(a), fb = quad<0xB1>(b);
      r[t][d] = odd ? fb : a;
      r[t + 1][d] = odd ? b : fa;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {  // lanes i, i ^ 2 and registers t, t + 2
      const uint32_t a = r[t][d], b = r[t + 2][d], fa = quad<0x4E>(a), fb = quad<0x4E>(b);
      r[t][d] = high ? fb : a;
      r[t + 2][d] = high ? b : fa;
    }
  }
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

// A piece of 16 MX rows: after `turn`, lane l holds blocks 16 piece + 4 g + s of
// row l % 16 and their scales, byte s of the word.  Blocks past the row's are
// read from its last; mask makes them zeros with scale 1.
struct MxPiece {
  u32x4 c[4];
  uint32_t s;
  __device__ __forceinline__ void load(const Rows &r, int piece, int lane, int nb) {
    const int kb = 16 * piece + 4 * (lane >> 4) + (lane & 3), in = kb < nb ? kb : nb - 1;
    s = *reinterpret_cast<const uint32_t *>(r.q + 16LL * piece + 4 * (lane >> 4));
#pragma unroll
    for (int t = 0; t < 4; ++t) c[t] = *reinterpret_cast<const u32x4 *>(r.p[t] + 16LL * in);
  }
  __device__ __forceinline__ void turn(int lane) { quad_transpose(c, lane); }
  __device__ __forceinline__ void mask(int piece, int lane, int nb) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (16 * piece + 4 * (lane >> 4) + i >= nb) {
        c[i] = u32x4{0, 0, 0, 0};
        s = (s & ~(255u << (8 * i))) | 127u << (8 * i);
      }
  }
  __device__ __forceinline__ uint32_t scale(int i) const { return (s >> (8 * i)) & 255u; }
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
// Whether all of a lane's blocks allow it (blocks of zeros allow any).
template <uint32_t LOW, uint32_t HIGH>
__device__ inline bool scales_within(const MxPiece &x) {
  bool ok = true;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const u32x4 c = x.c[s];
    const uint32_t sb = x.scale(s);
    ok &= sb - LOW <= HIGH - LOW || (sb != 255 && (c[0] | c[1] | c[2] | c[3]) == 0);
  }
  return ok;
}

// The wave's number in its workgroup, as a scalar.
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Four 16-byte parts of 16-bit rows: 64 consecutive bytes of row l % 16 after
// `turn`, from byte `at` of group g = 0 on.
template <bool ODD>
struct Half {
  Eight<ODD> e[4];
  u32x4 v[4];
  __device__ __forceinline__ void load(const unsigned char *const (&p)[4], long long at) {
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t].load(p[t] + at);
  }
  // Values k .. k + 7 of each row as far as they are below K, else 0.
  __device__ __forceinline__ void load_tail(const unsigned char *const (&p)[4], long long k, int K) {
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t].set(load_guarded(p[t], k, K - k), p[t]);
  }
  __device__ __forceinline__ void turn(const unsigned char *const (&p)[4], int lane) {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = e[t].get(p[t]);
    quad_transpose(v, lane);
  }
};

// Split activations (two bf16 planes, hi and lo): 4 rows together, in the
// order of the second product's loads.  For a load (piece, step, MFMA j) and
// 4 rows: 256 bytes, lane group g's 64 at 64 g, row r's 16 at 16 (r % 4).
// Values per row are padded with zeros to whole pieces (`pitch`).
template <int W>
__device__ inline long long split_at(int row, int k, long long pitch) {
  const int kSteps = kPieceSteps<W>;
  const int piece = k / kPieceK<W>, in = k % kPieceK<W>;
  const int g = in / (32 * kSteps), s = in / 32 % kSteps, j = in / 8 % 4, b = in % 8;
  return 2 * ((row >> 2) * 4 * pitch) + ((piece * kSteps + s) * 4 + j) * 256LL + 64 * g +
         16 * (row & 3) + 2 * b;
}

// One product of thin operands: MB blocks of 16 rows of kind A by NB blocks
// of 16 rows of weights of kind W.
template <int W, int A, int MB, int NB, bool ODD = false>
struct Thin {
  static constexpr int kK = kPieceK<W>, kSteps = kPieceSteps<W>;
  typedef typename ActRow<A>::type Act;
  struct Weights {
    MxPiece mx[W == kMx ? NB : 1];
    Half<ODD> half[W == kMx ? 1 : NB];
  };
  f32x4 acc[MB][NB];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // A piece's weights; with TAIL it may reach past K.
  template <bool TAIL>
  static __device__ __forceinline__ void load_weights(Weights &x, const Rows (&w)[NB], int piece,
                                                      int lane, int K, int nb) {
    const long long k = (long long)kK * piece + 32 * (lane >> 4) + 8 * (lane & 3);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (W == kMx) x.mx[b].load(w[b], piece, lane, nb);
      else if constexpr (TAIL) x.half[b].load_tail(w[b].p, k, K);
      else x.half[b].load(w[b].p, 2 * k);
    }
  }
  template <bool TAIL>
  static __device__ __forceinline__ void turn_weights(Weights &x, const Rows (&w)[NB], int piece,
                                                      int lane, int nb) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (W == kMx) {
        x.mx[b].turn(lane);
        if constexpr (TAIL) x.mx[b].mask(piece, lane, nb);
      } else {
        x.half[b].turn(w[b].p, lane);
      }
    }
  }

  // The products of a piece whose weights are loaded and turned, with the
  // activation rows that `valid` has.
  template <bool TAIL>
  __device__ __forceinline__ void use(const Weights &x, const Act (&a)[MB],
                                      const bool (&valid)[MB], int piece, int lane, int K, int nb) {
    if constexpr (A == kMx) {
      MxPiece y[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if (valid[i]) y[i].load(a[i], piece, lane, nb);
        y[i].turn(lane);
        if constexpr (TAIL) y[i].mask(piece, lane, nb);
      }
      auto step = [&](auto sel) __attribute__((always_inline)) {
        constexpr int s = decltype(sel)::value;
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[i][b] = mfma_mx<s>(x.mx[b].c[s], (int)x.mx[b].s, y[i].c[s], (int)y[i].s, acc[i][b]);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
    } else {
      constexpr Widen kHow = W == kF16 || (W == kMx && A == kF16) ? kToF16 : kToBf16;
      bool ok = true;
      if constexpr (W == kMx) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          ok &= A == kF16 ? scales_within<104, 140>(x.mx[b]) : scales_within<1, 254>(x.mx[b]);
        ok = __all(ok);
      }
      if (W != kMx || ok) multiply<TAIL, kHow>(x, a, valid, piece, lane, K);
      else multiply<TAIL, kThroughF32>(x, a, valid, piece, lane, K);
    }
  }

  // HOW: the format the weights come in or are brought to.
  template <bool TAIL, Widen HOW>
  __device__ __forceinline__ void multiply(const Weights &x, const Act (&a)[MB],
                                           const bool (&valid)[MB], int piece, int lane, int K) {
    constexpr bool kSplitHere = A == kF16 && HOW != kToF16;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Eight<ODD && A != kSplit> y[MB][4];
      u32x4 z[A == kSplit ? MB : 1][4];
#pragma unroll
      for (int i = 0; i < MB; ++i)
        if (valid[i]) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (A == kSplit) {
              const long long at = ((piece * kSteps + s) * 4 + j) * 256LL;
              y[i][j].load(a[i].p + at);
              z[i][j] = *reinterpret_cast<const u32x4 *>(a[i].q + at);
            } else {
              const long long k =
                  (long long)kK * piece + 32 * kSteps * (lane >> 4) + 32 * s + 8 * j;
              if constexpr (TAIL) y[i][j].set(load_guarded(a[i].p, k, K - k), a[i].p);
              else y[i][j].load(a[i].p + 2 * k);
            }
          }
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 wv[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (W == kMx) wv[b] = widen<HOW>(x.mx[b].c[s][j], x.mx[b].scale(s));
          else wv[b] = x.half[b].v[j];
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          u32x4 v = y[i][j].get(a[i].p), lo{};
          if constexpr (A == kSplit) lo = z[i][j];
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
      // One step's activations at a time: all of them together would cost the
      // registers of the waves that hide their latency.
      if constexpr (kSteps > 1) __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Adds the products of pieces first, first + step, ... of the K values.
  __device__ __forceinline__ void run(const Act (&a)[MB], const bool (&valid)[MB],
                                      const Rows (&w)[NB], int first, int step, int K, int lane) {
    const int nb = (int)mx_blocks(K), last = K / kK;  // whole pieces
    int p = first;
#pragma unroll 1
    for (; p < last; p += step) {
      Weights x;
      load_weights<false>(x, w, p, lane, K, nb);
      turn_weights<false>(x, w, p, lane, nb);
      use<false>(x, a, valid, p, lane, K, nb);
    }
    if (p == last && (long long)last * kK < K) {
      Weights x;
      load_weights<true>(x, w, p, lane, K, nb);
      turn_weights<true>(x, w, p, lane, nb);
      use<true>(x, a, valid, p, lane, K, nb);
    }
  }
};

}  // namespace
}  // namespace gemm_f32_impl
