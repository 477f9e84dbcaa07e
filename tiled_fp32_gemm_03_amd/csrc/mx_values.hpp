// Device pieces shared by the MX kernels (gfx950): vector types, loads and
// stores of the unquantised formats, block scales and codes.  Everything
// here has internal linkage.
#pragma once

#include "gemm_internal.hpp"
#include "launch_util.hpp"
#include "mx_plan.hpp"

#include <cstdint>

namespace gemm_f32_impl {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4w __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32h __attribute__((aligned(2)));
typedef f32x2 f32x2u __attribute__((aligned(4)));

// An element of format FMT as fp32 (exact), and back (nearest even).
template <int FMT>
__device__ inline float to_f32(uint16_t h) {
  if constexpr (FMT == kBf16) return __builtin_bit_cast(float, (uint32_t)h << 16);
  else return (float)__builtin_bit_cast(_Float16, h);
}
template <int FMT>
__device__ inline uint16_t from_f32(float v) {
  if constexpr (FMT == kBf16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}
template <int FMT>
__device__ inline uint32_t pack2(float a, float b) {
  return (uint32_t)from_f32<FMT>(a) | (uint32_t)from_f32<FMT>(b) << 16;
}

template <int FMT>
__device__ inline float load1(const void *p, long long i) {
  if constexpr (FMT == kF32) return static_cast<const float *>(p)[i];
  else return to_f32<FMT>(static_cast<const uint16_t *>(p)[i]);
}
template <int FMT>
__device__ inline void store1(void *p, long long i, float v) {
  if constexpr (FMT == kF32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = from_f32<FMT>(v);
}

// 8 consecutive elements from element i, the first `n` of them (others 0).
template <int FMT>
__device__ inline void load8(const void *p, long long i, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (FMT == kF32) {
      const f32x4u *q = reinterpret_cast<const f32x4u *>(static_cast<const float *>(p) + i);
      const f32x4 a = q[0], b = q[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4h *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = to_f32<FMT>((uint16_t)a[j]);
        v[2 * j + 1] = to_f32<FMT>((uint16_t)(a[j] >> 16));
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < n ? load1<FMT>(p, i + j) : 0.f;
}
template <int FMT>
__device__ inline void store8(void *p, long long i, int n, const float (&v)[8]) {
  if (n >= 8) {
    if constexpr (FMT == kF32) {
      f32x4u *q = reinterpret_cast<f32x4u *>(static_cast<float *>(p) + i);
      q[0] = f32x4{v[0], v[1], v[2], v[3]};
      q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *reinterpret_cast<u32x4h *>(static_cast<uint16_t *>(p) + i) =
          u32x4{pack2<FMT>(v[0], v[1]), pack2<FMT>(v[2], v[3]), pack2<FMT>(v[4], v[5]),
                pack2<FMT>(v[6], v[7])};
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) store1<FMT>(p, i + j, v[j]);
}
// 4 consecutive elements to element i, the first `n` of them.
template <int FMT>
__device__ inline void store4(void *p, long long i, int n, f32x4 v) {
  if (n >= 4) {
    if constexpr (FMT == kF32)
      *reinterpret_cast<f32x4u *>(static_cast<float *>(p) + i) = v;
    else
      *reinterpret_cast<u32x2h *>(static_cast<uint16_t *>(p) + i) =
          u32x2{pack2<FMT>(v[0], v[1]), pack2<FMT>(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) store1<FMT>(p, i + j, v[j]);
}

// The magnitude bits of a float: ordered like the magnitudes, with
// infinities and NaN above every finite value.
__device__ inline uint32_t mag_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

// Scale byte of a block whose largest magnitude has these bits.  The fp32
// exponent field x stands for floor(log2 m) + 127, so the byte is x - 2,
// clamped at 0 (subnormal m has x = 0); x = 255 is an infinity or a NaN.
__device__ inline uint32_t scale_byte(uint32_t mbits) {
  const uint32_t x = mbits >> 23;
  return x == 255 ? 255u : (x > 2 ? x - 2 : 0u);
}

// Codes of 8 values under scale byte `sb`, value j in bits 4j .. 4j + 3.
// v_cvt_scalef32_pk_fp4_f32 divides by a power of two and rounds to nearest
// even with saturation; its scale has to be a normal float, so blocks with
// small scales are lifted by 2^64 first (exact).
__device__ inline uint32_t encode8(const float (&v)[8], uint32_t sb) {
  if (sb == 255) return 0;
  const bool low = sb < 64;
  const float lift = low ? 0x1p64f : 1.f;
  const float unit = __builtin_bit_cast(float, (sb + (low ? 64u : 0u)) << 23);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * lift, v[1] * lift, unit, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * lift, v[3] * lift, unit, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * lift, v[5] * lift, unit, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * lift, v[7] * lift, unit, 3);
  return r;
}

// The 8 values of a word of codes under scale byte `sb`: the elements, then
// one exact scaling by v_ldexp_f32 (rounded only below fp32's subnormals,
// which no element reaches; past its range an infinity), over 2^down.
__device__ inline void decode8(uint32_t w, uint32_t sb, float (&v)[8], int down = 0) {
  f32x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
  const int e = (int)sb - 127 - down;
  const float nan = __builtin_nanf("");
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = sb == 255 ? nan : __builtin_amdgcn_ldexpf(p[j >> 1][j & 1], e);
}

// 4 consecutive elements of a row of C in a format known at run time.
__device__ inline void store4_fmt(int fmt, void *p, long long i, int n, f32x4 v) {
  if (fmt == kF32) store4<kF32>(p, i, n, v);
  else if (fmt == kBf16) store4<kBf16>(p, i, n, v);
  else store4<kF16>(p, i, n, v);
}

// One v_mfma_scale_f32_16x16x128_f8f6f4 on 4-bit elements: lane l holds 32
// values (one block) of row l % 16 of each operand, the k of block l / 16,
// with that block's scale byte: byte SEL of the words sb and sa.  The accumulator's 4 values are row l % 16
// of `a` (C's row) and rows 4 (l / 16) .. + 3 of `b` (C's columns).
template <int SEL = 0>
__device__ inline f32x4 mfma_mx(u32x4 b, int sb, u32x4 a, int sa, f32x4 acc) {
  const i32x8 x{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8 y{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, SEL, sb, SEL, sa);
}

}  // namespace
}  // namespace gemm_f32_impl
