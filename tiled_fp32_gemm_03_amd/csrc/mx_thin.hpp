// Pieces of the thin products (gemm_mx_a16, the mixture-of-experts layer):
// 16 to 64 rows of activations against weights read once from memory.
//
// A wave multiplies blocks of 16 activation rows with blocks of 16 weight
// rows, 128 k at a time, four v_mfma_f32_16x16x32_bf16 (or _f16) per pair.
// Lane l holds row l % 16 of each operand; which k a lane holds is free as
// long as both operands agree, so it follows how the weights are stored:
//   MX weights: lane group g = l / 16 holds block g of the 128 k (one 16-byte
//     load) and MFMA j takes the block's values 8 j .. 8 j + 7, widened to
//     bf16 with their scale (exact: an element has two significant bits);
//   16-bit weights: MFMA j takes k = 32 j + 8 g .. + 7 (one 16-byte load).
// Activations of another type than the weights' are split into a bf16 sum
// hi + lo whose two terms are multiplied separately: exact for fp16 (11
// significant bits), 16 bits or more of an fp32 value.
#pragma once

#include "mx_values.hpp"

namespace gemm_f32_impl {
namespace {

constexpr int kWBf16 = 0, kWF16 = 1, kWMx = 2;  // kinds of weights

// First k (within a 128-deep step) of lane group g's operand of MFMA j.
template <int W>
__device__ inline int thin_k(int g, int j) {
  return W == kWMx ? 32 * g + 8 * j : 32 * j + 8 * g;
}

// The 32 values of a block as four bf16 operands.  v_cvt_scalef32_pk_bf16_fp4
// takes a normal float as its scale: byte 0 (2^-127) goes as 2^-126 times
// halved elements through fp32, and byte 255 makes NaN.
__device__ inline void widen_block(u32x4 codes, uint32_t sb, bf16x8 (&w)[4]) {
  if (sb - 1u < 254u) {
    const float unit = __builtin_bit_cast(float, sb << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], unit, 0);
      const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], unit, 1);
      const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], unit, 2);
      const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j], unit, 3);
      w[j] = bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      decode8(codes[j], sb, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[j][i] = (__bf16)v[i];
    }
  }
}

// hi + lo of 8 fp16 values; an infinity or a NaN is hi alone.
__device__ inline void split_f16(f16x8 x, bf16x8 &hi, bf16x8 &lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = (float)x[i];
    hi[i] = (__bf16)v;
    lo[i] = mag_bits(v) < 0x7f800000u ? (__bf16)(v - (float)hi[i]) : (__bf16)0.f;
  }
}

__device__ inline f32x4 mfma_bf16(bf16x8 b, bf16x8 a, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, acc, 0, 0, 0);
}
__device__ inline f32x4 mfma_f16(f16x8 b, f16x8 a, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a, acc, 0, 0, 0);
}

// 8 values of a row of 16-bit codes from k, the first `n` of them (others 0).
__device__ inline u32x4 load_act(const uint16_t *row, long long k, long long n) {
  if (n >= 8) return *reinterpret_cast<const u32x4h *>(row + k);
  u32x4 w{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
  return w;
}

// One row of weights of kind W and K values.
struct WRow {
  const unsigned char *p;       // 2-byte values or codes
  const unsigned char *scales;  // MX
};

// Lane group g's operands of step `step` (128 k): four of 8 values, 16-bit
// codes as they are or MX blocks widened to bf16; zeros past K.
template <int W>
__device__ inline void load_weights(const WRow &r, int step, int g, int K, u32x4 (&w)[4]) {
  if constexpr (W == kWMx) {
    const long long kb = 4LL * step + g;
    u32x4 c{0, 0, 0, 0};
    uint32_t sb = 127;
    if (kb < mx_blocks(K)) {
      c = *reinterpret_cast<const u32x4 *>(r.p + 16 * kb);
      sb = r.scales[kb];
    }
    bf16x8 v[4];
    widen_block(c, sb, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __builtin_bit_cast(u32x4, v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long k = 128LL * step + thin_k<W>(g, j);
      w[j] = load_act(reinterpret_cast<const uint16_t *>(r.p), k, K - k);
    }
  }
}

// acc += w a for one MFMA's operands: weights of kind W (MX ones widened to
// bf16), activations of format AF.
template <int W, int AF>
__device__ inline f32x4 thin_mfma(u32x4 w, u32x4 a, f32x4 acc) {
  if constexpr (W == kWF16) {
    static_assert(AF == kF16, "fp16 weights take fp16 activations");
    return mfma_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, a), acc);
  } else if constexpr (AF == kBf16) {
    return mfma_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a), acc);
  } else {
    bf16x8 hi, lo;
    split_f16(__builtin_bit_cast(f16x8, a), hi, lo);
    acc = mfma_bf16(__builtin_bit_cast(bf16x8, w), hi, acc);
    return mfma_bf16(__builtin_bit_cast(bf16x8, w), lo, acc);
  }
}

// The same for an activation given as hi + lo.  fp16 weights are split as
// well and the product of the two low parts, 2^-18 of the whole, is left out.
template <int W>
__device__ inline f32x4 thin_mfma_split(u32x4 w, u32x4 hi, u32x4 lo, f32x4 acc) {
  const bf16x8 h = __builtin_bit_cast(bf16x8, hi), l = __builtin_bit_cast(bf16x8, lo);
  if constexpr (W == kWF16) {
    bf16x8 wh, wl;
    split_f16(__builtin_bit_cast(f16x8, w), wh, wl);
    acc = mfma_bf16(wh, h, acc);
    acc = mfma_bf16(wh, l, acc);
    return mfma_bf16(wl, h, acc);
  } else {
    acc = mfma_bf16(__builtin_bit_cast(bf16x8, w), h, acc);
    return mfma_bf16(__builtin_bit_cast(bf16x8, w), l, acc);
  }
}

}  // namespace
}  // namespace gemm_f32_impl
