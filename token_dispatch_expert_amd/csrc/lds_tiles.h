// Device helpers for tiles loaded from HBM straight into LDS: buffer loads, the swizzled LDS
// image, and waits on one memory counter alone.
#pragma once

#include <utility>

#include "moe_internal.h"

namespace moe {

// Word 3 of a raw buffer descriptor (32-bit data format, bounds-checked offsets): loads at or
// past num_records bytes return zeros.
constexpr int kBufferWord3 = 0x00020000;

// 16 bytes per lane from a buffer into LDS at lds + 16 * lane (the loads are wrapped in a device
// function: called directly from a kernel template, the host compilation pass drops the
// kernel's launch stub)
// AUX is the load's cache policy; kNonTemporal marks data read once (streamed weights), so its
// lines are the first to leave the L2 and do not push out the operands other tiles reuse.
constexpr int kNonTemporal = 2;  // the nt bit of the gfx950 cache-policy field
template <int AUX = 0>
__device__ __forceinline__ void buffer_load_lds16(__amdgpu_buffer_rsrc_t rsrc, void* lds, int voffset,
                                                  int soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)lds, 16,
                                           voffset, soffset, 0, AUX);
}

// LDS image of a tile row of CPR chunks of 16 bytes: chunk c of row r sits at chunk c ^ x(r),
// x(r) = (r >> 2) & 3 for 4 chunks, (r >> 1) & 7 for 8 and r & 15 for 16, so that the 16 rows
// read by one fragment load (same chunk) fall on distinct banks.
template <int CPR>
__device__ __forceinline__ int dswz(int row, int chunk) {
  static_assert(CPR == 4 || CPR == 8 || CPR == 16, "row width");
  if constexpr (CPR == 4) return row * 4 + (chunk ^ ((row >> 2) & 3));
  else if constexpr (CPR == 8) return row * 8 + (chunk ^ ((row >> 1) & 7));
  else return row * 16 + (chunk ^ (row & 15));
}

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding: vmcnt in bits
// 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8; the others are left at their maxima).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// f(integral_constant<int, 0>), ..., f(integral_constant<int, N - 1>), in order
template <typename F, int... Is>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}
// s_waitcnt lgkmcnt(0) alone (vmcnt and expcnt at their maxima)
__device__ __forceinline__ void wait_lgkmcnt0() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
}
// the same with a wave-uniform runtime count in [0, MAX] (a scalar branch per candidate)
template <int... Ns>
__device__ __forceinline__ void wait_vmcnt_dyn_impl(int n, std::integer_sequence<int, Ns...>) {
  ((n == Ns ? (wait_vmcnt<Ns>(), 0) : 0), ...);
}
template <int MAX>
__device__ __forceinline__ void wait_vmcnt_dyn(int n) {
  wait_vmcnt_dyn_impl(n, std::make_integer_sequence<int, MAX + 1>{});
}

}  // namespace moe
