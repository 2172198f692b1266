// Rows and weights to MXFP4 and back (the format is in mxfp4.h).
#include "mxfp4.h"
#include "mxfp4_internal.h"

namespace moe {

namespace {

struct QuantizeArgs {
  const void* x;
  const int32_t* f2s;  // the sorted row of each of a row's k assignments, or null: the row itself
  uint8_t *codes, *scales;
  int rows, k, d;      // rows of all matrices
  int n;               // output rows of a matrix
};

// 8 elements a thread: 4 threads share a scale, 32 a block of 8 scales. With a map the 4 threads of a group hand the group's 16 bytes
// round and store them for an assignment each, and the threads of a block its scales. WIDE: see row_unit.
// HBM bounds it: 8,192 bf16 rows of 7168 go to their 65,536 sorted rows in 79 us (367 MB, 4.7 TB/s; 105 with 4 bytes a thread and
// copy), 32 x 2048 such rows of weights in 230 us (1.19 GB, 5.2 TB/s).
template <typename T, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void quantize_kernel(RowMap m, QuantizeArgs p) {
  unsigned row;
  int unit;
  row_unit<WIDE>(m, row, unit);
  if (row >= (unsigned)p.rows) return;  // whole blocks of 32 threads
  const bool in = unit * 8 < p.d;
  const F8 x = in ? load8_once(static_cast<const T*>(p.x) + (size_t)row * p.d + unit * 8) : F8{};
  unsigned top = 0;  // magnitudes compare as their bits do; infinity and NaN are the largest
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x.v[i]) & 0x7fffffffu);
  top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
  top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
  const int scale = mx_scale(top);
  const float inv = mx_inverse(scale);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = x.v[i] * inv;
  const unsigned c = scale == kMxNan ? 0u : mx_codes8(q);
  // the block's 8 scales, of threads 0, 4, .. 28 of its 32, in every thread: 4 of each 16 threads, then the two 16s'
  unsigned four = (unsigned)scale << ((unit & 12) * 2);
  four |= (unsigned)__builtin_amdgcn_mov_dpp((int)four, 0x141, 0xf, 0xf, true);  // mirrored within 8
  four |= (unsigned)__builtin_amdgcn_mov_dpp((int)four, 0x140, 0xf, 0xf, true);  // within 16
  const auto both = __builtin_amdgcn_permlane16_swap(four, four, false, false);
  const u32x2 eight{both[0], both[1]};
  const int blocks = mx_blocks(p.d), b = unit >> 5;
  if (!p.f2s) {
    const size_t e = row / (unsigned)p.n, r = row - e * p.n;
    if (in) reinterpret_cast<unsigned*>(p.codes)[((size_t)row * p.d >> 3) + unit] = c;
    if ((unit & 31) == 0 && b < blocks)
      *reinterpret_cast<u32x2*>(p.scales + mx_scale_at(e, blocks, b, p.n, r)) = eight;
    return;
  }
  u32x4 group;
  group[0] = (unsigned)__builtin_amdgcn_mov_dpp((int)c, 0x00, 0xf, 0xf, true);
  group[1] = (unsigned)__builtin_amdgcn_mov_dpp((int)c, 0x55, 0xf, 0xf, true);
  group[2] = (unsigned)__builtin_amdgcn_mov_dpp((int)c, 0xaa, 0xf, 0xf, true);
  group[3] = (unsigned)__builtin_amdgcn_mov_dpp((int)c, 0xff, 0xf, 0xf, true);
  const int32_t* const map = p.f2s + (size_t)row * p.k;
  const int lead = unit & 31;
  if (lead < p.k && b < blocks) {
    const int to = map[lead];
    if ((unsigned)to < (unsigned)p.n)
      *reinterpret_cast<u32x2*>(p.scales + mx_scale_at(0, blocks, b, p.n, to)) = eight;
  }
  if (!in) return;
  for (int j = unit & 3; j < p.k; j += 4) {
    const int to = map[j];
    if ((unsigned)to < (unsigned)p.n) *reinterpret_cast<u32x4*>(p.codes + ((size_t)to * p.d >> 1) + (unit >> 2) * 16) = group;
  }
}

template <typename T, bool STREAM, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void dequantize_kernel(RowMap m, const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int rows, int n,
                                                                int d, T* __restrict__ out) {
  unsigned row;
  int unit;
  row_unit<WIDE>(m, row, unit);
  if (row >= (unsigned)rows || unit * 8 >= d) return;
  const size_t e = row / (unsigned)n, r = row - e * n;
  const unsigned c = reinterpret_cast<const unsigned*>(codes)[((size_t)row * d >> 3) + unit];
  const unsigned s = scales[mx_scale_at(e, mx_blocks(d), unit >> 5, n, r) + (unit >> 2 & 7)];
  const F8 v = mx_values8(c, mx_scale_f32(s));
  if constexpr (STREAM) store8_once(out + (size_t)row * d + unit * 8, v);
  else store8(out + (size_t)row * d + unit * 8, v);
}

RowMap block_map(int d) { return row_map(mx_blocks(d) * 32); }

}  // namespace

long long mx_row_grid(long long rows, int d) {
  const long long blocks = row_grid(block_map(d), rows), plain = row_grid(row_map(d / 8), rows);
  return blocks > plain ? blocks : plain;
}

hipError_t launch_mx_quantize(const void* x, bool bf16, int E, int rows, int k, int d, const int32_t* f2s,
                              void* codes, void* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const RowMap m = block_map(d);
  const QuantizeArgs p{x, f2s, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), E * rows, k, d, rows * k};
  const unsigned grid = (unsigned)row_grid(m, p.rows);
  const bool wide = m.shift >= 6;
  auto kern = bf16 ? (wide ? &quantize_kernel<__bf16, true> : &quantize_kernel<__bf16, false>)
                   : (wide ? &quantize_kernel<float, true> : &quantize_kernel<float, false>);
  kern<<<grid, m.threads(), 0, stream>>>(m, p);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_mx_dequantize_t(const void* codes, const void* scales, int E, int rows, int d, void* out,
                                         hipStream_t stream) {
  const RowMap m = row_map(d / 8);
  const unsigned grid = (unsigned)row_grid(m, (long long)E * rows);
  // Non-temporal stores where an instruction writes whole lines and the rows do not fit the last-level cache.
  const bool past_cache = sizeof(T) == 2 && d % 64 == 0 && (long long)E * rows * d * 2 >= kCacheBytes;
  auto kern = m.shift < 6 ? &dequantize_kernel<T, false, false>
                          : (past_cache ? &dequantize_kernel<T, true, true> : &dequantize_kernel<T, false, true>);
  kern<<<grid, m.threads(), 0, stream>>>(m, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                                         E * rows, rows, d, static_cast<T*>(out));
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void* codes, const void* scales, int E, int rows, int d, void* out,
                                bool bf16, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return (bf16 ? &launch_mx_dequantize_t<__bf16> : &launch_mx_dequantize_t<float>)(codes, scales, E, rows, d, out, stream);
}

}  // namespace moe
