// The MXFP4 format on the device: e2m1 codes, two to a byte (the first in the low half), one e8m0 scale
// byte b per 32 consecutive elements; a value is code * 2^(b - 127), and NaN for b = 255. Codes of
// [rows, d] are rows of d / 2 bytes. Scales lie in blocks of 256 elements, [ceil(d/256)][rows][8]: a
// tile of a product takes 256 elements of neighbouring rows at a time, and so finds their scales in one piece
// (row by row they would be 8 bytes of a cache line each).
#pragma once

#include "rows.h"

namespace moe {

constexpr int kMxGroup = 32, kMxBlock = 256;
constexpr int kMxMaxExp = 125;  // scales that are written: 2^-125 .. 2^125, so that values are normal bf16 numbers
constexpr int kMxNan = 255;

__host__ __device__ inline int mx_blocks(int d) { return (d + kMxBlock - 1) / kMxBlock; }
// Where the 8 scales of row r of matrix e, block b lie (matrices of n rows and `blocks` blocks).
__device__ __forceinline__ size_t mx_scale_at(size_t e, int blocks, int b, size_t n, size_t r) {
  return ((e * blocks + b) * n + r) * 8;
}

// The scale byte of a group whose largest magnitude has the bits `top`: the smallest power of two with
// which it is at most 6, the largest code, so that nothing saturates (but from 6 * 2^125 on, where codes
// stop at 6) and value / scale is exact: the one rounding is the code's. 1 for a group of zeros; NaN for
// a group that holds a NaN or an infinity, which no code stands for.
__device__ __forceinline__ int mx_scale(unsigned top) {
  if (top >= 0x7f800000u) return kMxNan;
  const int e = (int)(top >> 23) - 127 - 2 + ((top & 0x7fffffu) > 0x400000u ? 1 : 0);  // 6 = 1.5 * 2^2
  return top == 0 ? 127 : min(max(e, -kMxMaxExp), kMxMaxExp) + 127;
}
// 1 / scale (0 for NaN, so that the codes of such a group are 0 or whatever NaN becomes)
__device__ __forceinline__ float mx_inverse(int scale) { return __uint_as_float((unsigned)(254 - min(scale, 254)) << 23); }

// Codes of 8 scaled elements, rounded to nearest even, beyond 6 to 6.
__device__ __forceinline__ unsigned mx_codes8(const float (&q)[8]) {
  unsigned c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, q[0], q[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[2], q[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[4], q[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[6], q[7], 1.0f, 3);
}
// The scale as the conversions take it (its exponent bits; 255 gives NaN).
__device__ __forceinline__ float mx_scale_f32(unsigned byte) { return __uint_as_float(byte << 23); }

// The values of 8 codes, exact but for the ends of the formats.
__device__ __forceinline__ F8 mx_values8(unsigned c, float scale) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
  return F8{{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]}};
}
__device__ __forceinline__ bf16x8 mx_bf16x8(unsigned c, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2), e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

}  // namespace moe
