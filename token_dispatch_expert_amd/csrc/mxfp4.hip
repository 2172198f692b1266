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

// 8 elements a thread: 4 threads share a scale, 32 a block of 8 scales.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void quantize_kernel(RowMap m, QuantizeArgs p) {
  unsigned row;
  int unit;
  row_unit(m, row, unit);
  if (row >= (unsigned)p.rows) return;  // whole blocks of 32 threads (RowMap rows are whole blocks)
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
  // the block's 8 scales, of threads 0, 4, .. 28 of its 32, in every thread
  unsigned lo = (unsigned)scale << ((unit & 12) * 2), hi = 0;
  lo |= (unsigned)__shfl_xor((int)lo, 4);
  lo |= (unsigned)__shfl_xor((int)lo, 8);
  hi = (unsigned)__shfl_xor((int)lo, 16);
  if (unit & 16) {
    const unsigned t = lo;
    lo = hi;
    hi = t;
  }
  const int blocks = mx_blocks(p.d), b = unit >> 5;
  const bool lead = (unit & 31) == 0 && b < blocks;
  if (!p.f2s) {
    const size_t e = row / (unsigned)p.n, r = row - e * p.n;
    if (in) reinterpret_cast<unsigned*>(p.codes)[((size_t)row * p.d >> 3) + unit] = c;
    if (lead) *reinterpret_cast<u32x2*>(p.scales + mx_scale_at(e, blocks, b, p.n, r)) = u32x2{lo, hi};
    return;
  }
  for (int j = 0; j < p.k; ++j) {
    const int to = p.f2s[(size_t)row * p.k + j];
    if ((unsigned)to >= (unsigned)p.n) continue;
    if (in) reinterpret_cast<unsigned*>(p.codes)[((size_t)to * p.d >> 3) + unit] = c;
    if (lead) *reinterpret_cast<u32x2*>(p.scales + mx_scale_at(0, blocks, b, p.n, to)) = u32x2{lo, hi};
  }
}

template <typename T>
__global__ __launch_bounds__(kRowThreads) void dequantize_kernel(RowMap m, const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int rows, int n,
                                                                int d, T* __restrict__ out) {
  unsigned row;
  int unit;
  row_unit(m, row, unit);
  if (row >= (unsigned)rows || unit * 8 >= d) return;
  const size_t e = row / (unsigned)n, r = row - e * n;
  const unsigned c = reinterpret_cast<const unsigned*>(codes)[((size_t)row * d >> 3) + unit];
  const unsigned s = scales[mx_scale_at(e, mx_blocks(d), unit >> 5, n, r) + (unit >> 2 & 7)];
  store8(out + (size_t)row * d + unit * 8, mx_values8(c, mx_scale_f32(s)));
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
  if (bf16) quantize_kernel<__bf16><<<grid, m.threads(), 0, stream>>>(m, p);
  else quantize_kernel<float><<<grid, m.threads(), 0, stream>>>(m, p);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void* codes, const void* scales, int E, int rows, int d, void* out,
                                bool bf16, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const RowMap m = row_map(d / 8);
  const unsigned grid = (unsigned)row_grid(m, (long long)E * rows);
  const uint8_t *c = static_cast<const uint8_t*>(codes), *s = static_cast<const uint8_t*>(scales);
  if (bf16)
    dequantize_kernel<__bf16><<<grid, m.threads(), 0, stream>>>(m, c, s, E * rows, rows, d, static_cast<__bf16*>(out));
  else
    dequantize_kernel<float><<<grid, m.threads(), 0, stream>>>(m, c, s, E * rows, rows, d, static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace moe
