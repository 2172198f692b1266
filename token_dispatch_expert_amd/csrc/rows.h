// Device helpers for the row-wise kernels of the training step: 8 elements of a row per thread.
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kRowThreads = 256;

// Threads of a workgroup over rows of `units` 8-element units: 2^shift threads per row (so
// several short rows share a workgroup), `slices` workgroups per long row. The width is the
// one, of 16 to 256, that leaves the fewest threads idle.
struct RowMap {
  int shift, slices;
};
inline RowMap row_map(int units) {
  RowMap best{4, 0};
  long long waste = -1;
  for (int s = 8; s >= 4; --s) {
    const int slices = (units + (1 << s) - 1) >> s;
    const long long w = ((long long)slices << s) - units;
    if (waste < 0 || w < waste) {
      waste = w;
      best = RowMap{s, slices};
    }
  }
  return best;
}
inline long long row_grid(const RowMap& m, long long rows) {
  const long long per = kRowThreads >> m.shift;
  return (rows + per - 1) / per * m.slices;
}
__device__ __forceinline__ void row_unit(const RowMap& m, unsigned& row, int& unit) {
  const unsigned rb = blockIdx.x / (unsigned)m.slices, slice = blockIdx.x - rb * (unsigned)m.slices;
  row = rb * (unsigned)(kRowThreads >> m.shift) + (threadIdx.x >> m.shift);
  unit = (int)((slice << m.shift) + (threadIdx.x & ((1u << m.shift) - 1)));
}

struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 load8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ F8 load8(const __bf16* p) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(a[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
  return r;
}
// The rounding of a result to bf16 (nearest even) is the output format's.
__device__ __forceinline__ void store8(float* p, const F8& r) {
  *reinterpret_cast<f32x4*>(p) = f32x4{r.v[0], r.v[1], r.v[2], r.v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{r.v[4], r.v[5], r.v[6], r.v[7]};
}
__device__ __forceinline__ void store8(__bf16* p, const F8& r) {
  bf16x8 b;
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = (__bf16)r.v[i];
  *reinterpret_cast<bf16x8*>(p) = b;
}

// ---------------------------------------------------------------------------------------
// 8-bit rows: e4m3fn codes and one fp32 scale per 128 elements, a power of two
// ---------------------------------------------------------------------------------------
constexpr int kHeldGroup = 128;
constexpr int kHeldMinExp = -117, kHeldMaxExp = 120;

// Codes of this thread's 8 elements; `scale` is that of the 16 threads (one aligned group of
// 128 elements) that call together. The scale is the smallest power of two with which the
// group's largest finite magnitude is at most 448, the largest code, so nothing saturates and
// value / scale is exact: the one rounding is the code's, to nearest even. It is at least
// 2^-117, so that every code times its scale is a normal bf16 number. At the largest scale,
// 2^120, codes stop at 240: the next one up would stand for 2^128. NaN and infinities become
// the NaN code and do not enter the scale.
__device__ __forceinline__ uint2 hold8(const F8& x, float& scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x.v[i]);
    top = fmaxf(top, a <= 3.402823466e38f ? a : 0.f);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const unsigned bits = __float_as_uint(top);
  int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  e = top == 0.f ? 0 : min(max(e, kHeldMinExp), kHeldMaxExp);
  scale = __uint_as_float((unsigned)(e + 127) << 23);
  const float inv = __uint_as_float((unsigned)(127 - e) << 23);
  const float most = e == kHeldMaxExp ? 240.f : 448.f;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x.v[i]);
    q[i] = a <= 3.402823466e38f ? fminf(fmaxf(x.v[i] * inv, -most), most) : __uint_as_float(0x7fc00000u);
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return make_uint2((unsigned)lo, (unsigned)hi);
}
// The values that 8 codes stand for (exact).
__device__ __forceinline__ F8 held8(uint2 c, float scale) {
  F8 r;
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, true);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, false), f = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, true);
  const float v[8] = {a[0], a[1], b[0], b[1], d[0], d[1], f[0], f[1]};
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = v[i] * scale;
  return r;
}

}  // namespace moe
