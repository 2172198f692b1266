// Device helpers for the row-wise kernels of the training step: 8 elements of a row per thread.
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kRowThreads = 256;
constexpr long long kCacheBytes = 256LL << 20;  // the last-level cache

// Workgroups over rows of `units` 8-element units: 2^shift threads and `slices` workgroups per
// row. Rows of at least 64 units have workgroups of their own (of 2^shift threads, so the row and
// what goes with it are the same for a whole workgroup and come through scalar loads); shorter
// ones share workgroups of kRowThreads. The width is the one that leaves the fewest threads idle.
struct RowMap {
  int shift, slices;
  __host__ __device__ int threads() const { return shift >= 6 ? 1 << shift : kRowThreads; }
};
inline RowMap row_map(int units) {
  RowMap best{4, 0};
  long long waste = -1;
  for (int s = 8; s >= (units >= 64 ? 6 : 4); --s) {
    const int slices = (units + (1 << s) - 1) >> s;
    const long long w = ((long long)slices << s) - units;
    if (waste < 0 || w < waste) {
      waste = w;
      best = RowMap{s, slices};
    }
  }
  return best;
}
// All workgroups of a row run on one XCD (workgroup b runs on XCD b % 8).
inline long long row_grid(const RowMap& m, long long rows) {
  const long long per = m.threads() >> m.shift, groups = (rows + per - 1) / per;
  return (m.slices > 1 ? (groups + 7) / 8 * 8 : groups) * m.slices;
}
// WIDE: m.shift >= 6. The row is then the same for a whole workgroup, and the compiler knows it: summing
// 8 rows of 14 KB for each of 8192 tokens took 231 us with the row's number (and so its map entries)
// per lane, 176 us like this.
template <bool WIDE = false>
__device__ __forceinline__ void row_unit(const RowMap& m, unsigned& row, int& unit) {
  unsigned group = blockIdx.x, slice = 0;
  if (m.slices > 1) {
    const unsigned i = blockIdx.x >> 3, q = i / (unsigned)m.slices;
    slice = i - q * (unsigned)m.slices;
    group = q * 8 + (blockIdx.x & 7);
  }
  row = group;
  if (!WIDE && m.shift < 6) row = group * (unsigned)(kRowThreads >> m.shift) + (threadIdx.x >> m.shift);
  unit = (int)((slice << m.shift) + (threadIdx.x & ((1u << m.shift) - 1)));
}

struct F8 {
  float v[8];
};
// ..._once: non-temporal, for data that the kernel reads or writes once: its lines leave the caches
// first. At 65,536 rows of 2048 the SwiGLU gradient took 239 us without and 199 us with them; loads of rows
// that several workgroups read stay plain, and stores where a kernel says why.
__device__ __forceinline__ F8 load8_once(const float* p) {
  const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
  const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
  return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ F8 widen8(u32x4 a) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(a[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ F8 load8_once(const __bf16* p) {
  return widen8(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
}
__device__ __forceinline__ F8 load8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ F8 load8(const __bf16* p) { return widen8(*reinterpret_cast<const u32x4*>(p)); }
// The rounding of a result to bf16 (nearest even) is the output format's.
__device__ __forceinline__ bf16x8 narrow8(const F8& r) {
  bf16x8 b;
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = (__bf16)r.v[i];
  return b;
}
__device__ __forceinline__ void store8(float* p, const F8& r) {
  *reinterpret_cast<f32x4*>(p) = f32x4{r.v[0], r.v[1], r.v[2], r.v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{r.v[4], r.v[5], r.v[6], r.v[7]};
}
__device__ __forceinline__ void store8(__bf16* p, const F8& r) { *reinterpret_cast<bf16x8*>(p) = narrow8(r); }
__device__ __forceinline__ void store8_once(float* p, const F8& r) {
  __builtin_nontemporal_store(f32x4{r.v[0], r.v[1], r.v[2], r.v[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{r.v[4], r.v[5], r.v[6], r.v[7]}, reinterpret_cast<f32x4*>(p + 4));
}
__device__ __forceinline__ void store8_once(__bf16* p, const F8& r) {
  __builtin_nontemporal_store(narrow8(r), reinterpret_cast<bf16x8*>(p));
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
__device__ __forceinline__ unsigned dpp_max16(unsigned v) {  // over the 16 lanes of a row
  v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));   // lanes 1 0 3 2
  v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));   // lanes 2 3 0 1
  v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));  // mirrored within 8
  return max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));  // within 16
}
__device__ __forceinline__ uint2 hold8(const F8& x, float& scale) {
  // magnitudes compare as their bits do; infinity and NaN are the largest
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x.v[i]) & 0x7fffffffu);
  top = dpp_max16(top);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = x.v[i];
  const bool ends = top >= 0x7f000000u;  // non-finite values, or some of at least 2^127
  if (ends) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned a = __float_as_uint(q[i]) & 0x7fffffffu;
      if (a < 0x7f800000u) top = max(top, a);
      else q[i] = __uint_as_float(0x7fc00000u);
    }
    top = dpp_max16(top);
  }
  int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  e = top == 0 ? 0 : min(max(e, kHeldMinExp), kHeldMaxExp);
  scale = __uint_as_float((unsigned)(e + 127) << 23);
  const float inv = __uint_as_float((unsigned)(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] *= inv;
  if (ends && e == kHeldMaxExp)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = q[i] > 240.f ? 240.f : (q[i] < -240.f ? -240.f : q[i]);
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
