// Pieces of the products of few rows of activations with weights that are read
// once from memory, which is what bounds them (gemm_mx_a16, the
// mixture-of-experts layer).
//
// A wave multiplies blocks of 16 activation rows with blocks of 16 weight
// rows ("columns" of C) and takes K in pieces of 256 bytes of weight row:
// four 128-deep steps of MX weights, one of 16-bit ones.  The weights go from
// memory into registers, the next two pieces' while one is used; the activations,
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

// Kinds of operands: the formats of mx_plan.hpp (kF32: activations that enter
// as three bf16 terms, all their 24 bits), and MX rows.
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

// The same of finite weights, by truncation, which leaves lo's bits where the
// packing takes them (an infinity's lo is a NaN).
__device__ inline void split_f16_weights(u32x4 x, u32x4 &hi, u32x4 &lo) {
  const f16x8 v = __builtin_bit_cast(f16x8, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = (float)v[2 * i], b = (float)v[2 * i + 1];
    const uint32_t ua = __builtin_bit_cast(uint32_t, a), ub = __builtin_bit_cast(uint32_t, b);
    const float la = a - __builtin_bit_cast(float, ua & 0xffff0000u);
    const float lb = b - __builtin_bit_cast(float, ub & 0xffff0000u);
    hi[i] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
    lo[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, lb), __builtin_bit_cast(uint32_t, la),
                                  0x07060302u);
  }
}

// Three bf16 terms whose sum is each of 8 fp32 values: exact down to bf16's
// smallest step, 2^-133 (each takes the next 8 of 24 bits, by truncation).  An
// infinity or a NaN is the first alone.
__device__ inline void split_f32(u32x4 a, u32x4 b, u32x4 (&term)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u[3][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float v = __builtin_bit_cast(float, i < 2 ? a[2 * i + q] : b[2 * i + q - 4]);
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        u[t][q] = __builtin_bit_cast(uint32_t, v);
        const float rest = v - __builtin_bit_cast(float, u[t][q] & 0xffff0000u);
        v = mag_bits(v) < 0x7f800000u ? rest : 0.f;
      }
    }
#pragma unroll
    for (int t = 0; t < 3; ++t) term[t][i] = __builtin_amdgcn_perm(u[t][1], u[t][0], 0x07060302u);
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

// How the rows of 16-bit codes lie: kWords: a 16-byte load of 8 of them is
// cheap, or as cheap as any.  kOdd: rows that may start in the middle of a 4-byte
// word, where a 16-byte load costs a multiple of an aligned one.  kShort: of
// fewer than 8 codes.
enum { kWords, kOdd, kShort };

// Values k .. k + 7 of a row of K codes, or the last 8 where those pass K:
// `end` then moves them into place and adds the zeros.
template <int ROWS>
struct Eight {
  u32x4 v;
  static __device__ __forceinline__ long long first(long long k, int K) {
    return k < K - 8 ? k : K - 8;
  }
  __device__ __forceinline__ void load(const unsigned char *row, long long k, int K) {
    v = *reinterpret_cast<const u32x4h *>(row + 2 * first(k, K));
  }
  __device__ __forceinline__ u32x4 get() const { return v; }
  static __device__ __forceinline__ u32x4 end(u32x4 x, long long k, int K) {
    return drop_first(x, k - first(k, K));
  }
};
// The words around the values, from 2 bytes before the first on where that is
// in the middle of one (the row before, or its padding: only rows after the
// first can be odd, because the matrix starts on a word), with the last value on
// its own.
template <>
struct Eight<kOdd> : Eight<kWords> {
  uint32_t last, shift;
  __device__ __forceinline__ void load(const unsigned char *row, long long k, int K) {
    const unsigned char *at = row + 2 * first(k, K);
    const uintptr_t odd = reinterpret_cast<uintptr_t>(at) & 2;
    v = *reinterpret_cast<const u32x4w *>(at - odd);
    last = *reinterpret_cast<const uint16_t *>(at + 14);
    shift = 8 * (uint32_t)odd;
  }
  __device__ __forceinline__ u32x4 get() const {
    return u32x4{__builtin_amdgcn_alignbit(v[1], v[0], shift),
                 __builtin_amdgcn_alignbit(v[2], v[1], shift),
                 __builtin_amdgcn_alignbit(v[3], v[2], shift),
                 __builtin_amdgcn_alignbit(last, v[3], shift)};
  }
};
template <>
struct Eight<kShort> : Eight<kWords> {
  __device__ __forceinline__ void load(const unsigned char *row, long long k, int K) {
    v = load_guarded(row, k < K ? k : K, K);
  }
  static __device__ __forceinline__ u32x4 end(u32x4 x, long long, int) { return x; }
};

// How the values of MX weights become matrix operands.  As bf16 or fp16 by
// one conversion per two values where every scale of the piece allows it:
// bf16 holds every element under scale bytes 0 to 252 (0.5 2^-127 is a
// subnormal that it holds exactly, 6 2^125 below its largest value; the conversion
// takes a scale's exponent bits alone, 0 as 2^-127), fp16 under 104 to 140 (0.5
// 2^-23 is its smallest step, 6 2^13 below its largest value) and zeros under all
// but 255: a block of them has byte 0.  Otherwise through fp32, over 2^down (see
// Quartered).
enum Widen { kToBf16, kToF16, kThroughF32 };
template <Widen HOW>
__device__ inline u32x4 widen(uint32_t codes, uint32_t sb, int down = 0) {
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
    decode8(codes, sb, v, down);
    return u32x4{pack2<kBf16>(v[0], v[1]), pack2<kBf16>(v[2], v[3]), pack2<kBf16>(v[4], v[5]),
                 pack2<kBf16>(v[6], v[7])};
  }
}

// Elements under scale bytes 253 and 254 can be past bf16's largest value, their
// products need not be.  A piece that has such a byte is multiplied at a quarter of
// its size, which bf16 holds of the smallest elements too, onto a quarter of the sums
// so far.  `bytes`: the lane's, through top_scale, or'ed (255, a NaN, counts too,
// and stays one).
constexpr uint32_t kTopScale = 252;
__device__ inline uint32_t top_scale(uint32_t sb) { return sb + (255 - kTopScale); }  // bit 8: past it
struct Quartered {
  int down;
  __device__ __forceinline__ explicit Quartered(uint32_t bytes) : down(__any((bytes & 256) != 0) ? 2 : 0) {}
  __device__ __forceinline__ void before(f32x4 &acc) const { scale(acc, -down); }
  __device__ __forceinline__ void after(f32x4 &acc) const { scale(acc, down); }
  static __device__ __forceinline__ void scale(f32x4 &acc, int e) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_amdgcn_ldexpf(acc[i], e);
  }
};

// Whether codes under scale byte `sb` can be widened to bf16, or to fp16 (A ==
// kF16), by conversion.
template <int A>
__device__ inline bool widens_fast(uint32_t sb, uint32_t codes) {
  return A == kF16 ? sb - 104u <= 140u - 104u || (codes == 0 && sb != 255) : sb <= kTopScale;
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
// Exchanges inside each four lanes.
template <int CTRL>
__device__ inline uint32_t quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
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
  template <int A>
  __device__ __forceinline__ bool widens_fast() const {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ok &= gemm_f32_impl::widens_fast<A>(s[i], c[i][0] | c[i][1] | c[i][2] | c[i][3]);
    return ok;
  }
};

// A piece of 16 rows of 16-bit weights as loaded: values 32 j + 8 (l % 4) ..
// + 7 of it, j = 0 .. 3; or the last 8 of the row where those pass K.
template <int ROWS>
struct HalfPiece {
  Eight<ROWS> x[4];
  static __device__ __forceinline__ long long at(int piece, int j, int lane) {
    return 128LL * piece + 32 * j + 8 * (lane & 3);
  }
  __device__ __forceinline__ void load(const unsigned char *row, int piece, int lane, int K) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j].load(row, at(piece, j, lane), K);
  }
  // For the piece that passes K: moves what it holds into place.
  __device__ __forceinline__ void end(const unsigned char *, int piece, int lane, int K) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j].v = x[j].end(x[j].v, at(piece, j, lane), K);
  }
  __device__ __forceinline__ u32x4 get(int j, int) const { return x[j].get(); }
};
// The words around the values, as in Eight<kOdd>; the last value is the first
// of the next lane's words, and the piece's last a load of its own (one of each
// lane's: 71 us for the loads of a first product of 268 MB, against 53 of even
// rows).
template <>
struct HalfPiece<kOdd> {
  u32x4 v[4];
  uint32_t last, shift;
  __device__ __forceinline__ void load(const unsigned char *row, int piece, int lane, int K) {
    const uintptr_t odd = reinterpret_cast<uintptr_t>(row) & 2;
    shift = 8 * (uint32_t)odd;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long k = HalfPiece<kWords>::at(piece, j, lane), most = (K - 8) & ~1;
      v[j] = *reinterpret_cast<const u32x4w *>(row - odd + 2 * (k < most ? k : most));
    }
    const long long k = 128LL * piece + 127;
    last = *reinterpret_cast<const uint16_t *>(row + 2 * (k < K ? k : K - 1));
  }
  // What it holds is of no use there, but its lines are at hand.
  __device__ __forceinline__ void end(const unsigned char *row, int piece, int lane, int K) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long k = HalfPiece<kWords>::at(piece, j, lane);
      v[j] = load_guarded(row, k < K ? k : K, K);
    }
    shift = 0;
  }
  __device__ __forceinline__ u32x4 get(int j, int lane) const {
    const uint32_t next = j < 3 ? v[j < 3 ? j + 1 : j][0] : last;
    const uint32_t word = (lane & 3) == 0 ? next : v[j][0];
    // of lane + 1, in each four
    const uint32_t w4 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0x39, 0xf, 0xf, false);
    return u32x4{__builtin_amdgcn_alignbit(v[j][1], v[j][0], shift),
                 __builtin_amdgcn_alignbit(v[j][2], v[j][1], shift),
                 __builtin_amdgcn_alignbit(v[j][3], v[j][2], shift),
                 __builtin_amdgcn_alignbit(w4, v[j][3], shift)};
  }
};

// ---- activations in LDS --------------------------------------------------------
//
// Blocks of up to 16 rows, `rows` of them kept (4, 8 or 16), of kc values: for
// each operand of a matrix instruction (piece, step, MFMA j) and lane group,
// the rows' 16 bytes one after the other, and 16 bytes of padding, so that
// neither the writes (neighbouring threads take neighbouring k of a row) nor
// the reads (16 lanes take 16 rows) meet on a bank.  kF32: three such planes,
// one for each term (splitting the values where they are used, by every wave that
// does, took 64 tokens on 64 experts from 123 to 159 us, the planes to 124).

struct Tile {
  int rows, kc;
  __host__ __device__ int group() const { return 16 * rows + 16; }
};
// LDS bytes of a block of rows of kind A: linear in kc (whole pieces).
template <int A>
__host__ __device__ inline int act_bytes(const Tile &t) {
  return t.kc / 8 * t.group() * (A == kF32 ? 3 : 1);
}

// Fills a block with values k0 .. k0 + kc - 1 of rows 0 .. n - 1, zeros past K;
// `row(r)` gives row r's start.  Threads 0 .. threads - 1 (`tid`) take part; each
// issues eight loads before it writes any (one at a time, their
// latencies alone took 30 us of a first product).  Rows of kind kF32 hold
// zeros from K to a multiple of 8.
template <int A, int W, int ROWS, class RowOf>
__device__ __forceinline__ void stage_acts(unsigned char *lds, const Tile &t, RowOf row, int n,
                                           int k0, int K, int tid, int threads) {
  constexpr int kBatch = A == kF32 ? 4 : 8;
  const int G = t.group();
  const int per = t.kc / 8, all = n * per, eights = (int)ceil_div(K, 8);
#pragma unroll 1
  for (int i0 = tid; i0 < all; i0 += kBatch * threads) {
    Eight<ROWS> c[kBatch];
    u32x4 d[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * threads < all ? i0 + u * threads : all - 1;
      const int r = i / per, x = i % per;
      if constexpr (A == kF32) {
        const int e = k0 / 8 + x, in = e < eights ? e : eights - 1;
        const u32x4w *q = reinterpret_cast<const u32x4w *>(row(r) + 32LL * in);
        c[u].v = q[0];
        d[u] = q[1];
      } else {
        c[u].load(row(r), k0 + 8LL * x, K);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * threads;
      if (i >= all) continue;
      const int r = i / per, x = i % per;
      // Operand and lane group of values 8 x .. 8 x + 7: the MX order of k
      // is (step, g, j), the 16-bit one (j, g).
      const int group = W == kMx ? (x & ~15) | (x & 3) << 2 | (x >> 2 & 3) : x;
      if constexpr (A == kF32) {
        const bool in = k0 / 8 + x < eights;
        u32x4 term[3];
        split_f32(c[u].v, d[u], term);
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *reinterpret_cast<u32x4 *>(lds + (q * per + group) * G + 16 * r) =
              in ? term[q] : u32x4{0, 0, 0, 0};
      } else {
        const long long k = k0 + 8LL * x;
        u32x4 v = c[u].get();
        if (k + 8 > K) v = c[u].end(v, k, K);
        *reinterpret_cast<u32x4 *>(lds + group * G + 16 * r) = v;
      }
    }
  }
}

// ---- the product -----------------------------------------------------------------

// A block of rows of kind A in LDS by NB blocks of 16 rows of weights of kind
// W in registers.  No load stands behind a branch: one that may or may not
// have been issued makes the compiler wait for all, the next piece's too.
template <int W, int A, int NB, int ROWS>
struct Thin {
  static constexpr int kK = kPieceK<W>, kSteps = kPieceSteps<W>;
  struct Weights {
    MxPiece mx[W == kMx ? NB : 1];
    HalfPiece<ROWS> half[W == kMx ? 1 : NB];
  };
  f32x4 acc[NB];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // A piece's weights.
  static __device__ __forceinline__ void load(Weights &x, const Row (&w)[NB], int piece, int lane,
                                              int K) {
    const int nb = (int)mx_blocks(K);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (W == kMx) {
        x.mx[b].load(w[b], piece, lane, nb);
      } else {
        x.half[b].load(w[b].p, piece, lane, K);
      }
    }
  }

  // The products of a loaded piece, number `local` of the tile; zeros past K.
  // `rows` gives the rows w once more.
  template <class RowsOf>
  __device__ __forceinline__ void use(Weights &x, RowsOf rows, const unsigned char *lds,
                                      const Tile &t, int local, int piece, int lane, int K) {
    const int g = lane >> 4, r = lane & (t.rows - 1), G = t.group();
    constexpr Widen kHow = W == kF16 || (W == kMx && A == kF16) ? kToF16 : kToBf16;
    const unsigned char *from = lds + (local * kSteps * 16 + g) * G + 16 * r;
    const int plane = t.kc / 8 * G;
    if constexpr (W != kMx) {
      if (piece >= K / kK) {  // uniform
        Row w[NB];
        rows(w);
#pragma unroll
        for (int b = 0; b < NB; ++b) x.half[b].end(w[b].p, piece, lane, K);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 wv[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) wv[b] = from_lane(x.half[b].get(j, lane), loader(lane));
        multiply<kHow>(wv, from + j * 4 * G, plane);
      }
    } else {
      const MxBlocks y0(x.mx[0], piece, lane, (int)mx_blocks(K));
      const MxBlocks y1(x.mx[NB - 1], piece, lane, (int)mx_blocks(K));
      const MxBlocks *y[2] = {&y0, &y1};
      bool ok = true;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        ok &= y[b]->template widens_fast<A>();
      if (__builtin_expect(__all(ok), 1)) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            u32x4 wv[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) wv[b] = widen<kHow>(y[b]->c[s][j], y[b]->s[s]);
            multiply<kHow>(wv, from + (4 * s + j) * 4 * G, plane);
          }
      } else {
        // Rare, and kept short: a loop over the piece's words.
        uint32_t top = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int s = 0; s < 4; ++s) top |= top_scale(y[b]->s[s]);
        const Quartered quarter(top);
#pragma unroll
        for (int b = 0; b < NB; ++b) quarter.before(acc[b]);
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
            wv[b] = widen<kThroughF32>(c, sb, quarter.down);
          }
          multiply<kThroughF32>(wv, from + i * 4 * G, plane);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) quarter.after(acc[b]);
      }
    }
  }

  // One matrix operand's products; `at`: the lane's activations in LDS.  HOW:
  // the format that the weights come in or were brought to.
  template <Widen HOW>
  __device__ __forceinline__ void multiply(const u32x4 (&wv)[NB], const unsigned char *at,
                                           int plane) {
    u32x4 v = *reinterpret_cast<const u32x4 *>(at);
    if constexpr (A == kF32) {
      const u32x4 term[3] = {v, *reinterpret_cast<const u32x4 *>(at + plane),
                             *reinterpret_cast<const u32x4 *>(at + 2 * plane)};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4 w = wv[b];
        if constexpr (HOW == kToF16) {  // fp16 weights are split too
          u32x4 rest;
          split_f16_weights(wv[b], w, rest);
#pragma unroll
          for (int i = 0; i < 3; ++i) acc[b] = mfma_bf16(rest, term[i], acc[b]);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) acc[b] = mfma_bf16(w, term[i], acc[b]);
      }
    } else {
      constexpr bool kSplitHere = A == kF16 && HOW != kToF16;
      u32x4 lo{};
      if constexpr (kSplitHere) split_f16(v, v, lo);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (HOW == kToF16) {
          acc[b] = mfma_f16(wv[b], v, acc[b]);
        } else {
          acc[b] = mfma_bf16(wv[b], v, acc[b]);
          if constexpr (kSplitHere) acc[b] = mfma_bf16(wv[b], lo, acc[b]);
        }
      }
    }
  }
};

// The same product of one block of rows with the activations straight from
// memory, for products so small that what counts is the latency: a piece's
// weights and activations are asked for together, both by four lanes to a
// line.  MFMA m of step s takes block 4 s + m of the piece here, lane l its
// values 8 (l / 16) .. + 7, so that one lane's load holds one lane's operand.
template <int A, int ROWS>
struct Direct {
  f32x4 acc;
  // The products of 8 values per lane, of MX words that allow `kHow` or not.
  template <Widen HOW>
  __device__ __forceinline__ void add(uint32_t codes, uint32_t sb, u32x4 v, int down = 0) {
    const u32x4 wv = widen<HOW>(codes, sb, down);
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
      Eight<ROWS> v[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        c[q] = *reinterpret_cast<const uint32_t *>(w.p + 16 * (16LL * piece + q) + 4 * part);
        v[q].load(a, 32 * (16LL * piece + q) + 8 * part, K);
      }
      // Looked at as loaded: the lane's codes are of row l / 4, whose scales the
      // quad's lanes have (with the operands' codes, 1 x 4096 x 4096 took 0.4 us more).
      bool ok = true;
      const uint32_t row[4] = {quad<0x00>(s), quad<0x55>(s), quad<0xAA>(s), quad<0xFF>(s)};
#pragma unroll
      for (int q = 0; q < 16; ++q)
        ok &= widens_fast<A>(row[q >> 2] >> (8 * (q & 3)) & 255u, c[q]);
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = from_lane(s, 4 * (lane & 15) + i);
      if (__all(ok)) {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          add<A == kF16 ? kToF16 : kToBf16>(from_lane(c[q], from), sc[q >> 2] >> (8 * (q & 3)) & 255u,
                                            from_lane(v[q].get(), from));
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
      const uint32_t sb = from_lane(s, 4 * (lane & 15) + (q >> 2)) >> (8 * (q & 3)) & 255u;
      const Quartered quarter(top_scale(sb));
      quarter.before(acc);
      add<kThroughF32>(from_lane(c, from), sb, from_lane(load_guarded(a, k < K ? k : K, K), from),
                       quarter.down);
      quarter.after(acc);
    }
  }
};

// Rows of the tile for n rows.
__host__ __device__ inline int tile_rows(int n) { return n <= 4 ? 4 : n <= 8 ? 8 : 16; }
// The activations' tile: all of K where it fits `bytes`, else as many pairs of
// rounds (pieces of all waves that share columns) as do, one at least.
template <int A>
__host__ __device__ inline Tile tile_of(int rows, int K, int round, int bytes) {
  const int all = (int)ceil_div(K, round), fit = bytes / act_bytes<A>(Tile{rows, round});
  return Tile{rows, round * (all <= fit ? all : fit > 3 ? fit & ~1 : all < 2 ? all : 2)};
}

}  // namespace
}  // namespace gemm_f32_impl
