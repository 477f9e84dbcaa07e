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

}  // namespace
}  // namespace gemm_f32_impl
