// Activations held in 8 bits between the forward and the backward pass, and the SwiGLU
// activation with its gradient on the held values.
//
// A held row is its e4m3fn codes and one fp32 scale per 128 elements, always a power of two
// (hold8 in rows.h): a value is code * scale, with a relative error of at most 2^-4 above the
// code's subnormal range, and exact in bf16, so nothing is rounded a second time on the way
// back. Every kernel here is bound by HBM: one pass, 16 bytes a thread and operand. 8,192 rows of 7168
// (bf16) are packed in 28 us (6.3 TB/s) and unpacked into their 65,536 sorted rows in 174 - 183 us
// (1.0 GB, 5.5 - 5.8 TB/s; a fill reaches 6.8); 65,536 rows of 2048 go through moe_swiglu in 161 us
// (6.7 TB/s) and its gradient in 199 - 230 us (1.35 GB, 5.9 - 6.8 TB/s).
//
// With s = 1 / (1 + e^-g), in fp32, and in 64 bits where s is no normal fp32 number (far_sigmoid):
//   h  = g s u
//   du = dh g s
//   dg = dh u s (1 + g (1 - s))
#include <math.h>

#include "grouped.h"
#include "rows.h"

namespace moe {

namespace {

template <typename T>
__global__ __launch_bounds__(kRowThreads) void pack_kernel(RowMap m, const T* __restrict__ x, int rows,
                                                          int d, uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  unsigned row;
  int unit;
  row_unit(m, row, unit);
  if (row >= (unsigned)rows) return;  // whole groups of 16 threads
  const bool in = unit * 8 < d;
  const size_t at = (size_t)row * d + unit * 8;
  float scale;
  const uint2 c = hold8(in ? load8(x + at) : F8{}, scale);
  if (!in) return;
  *reinterpret_cast<uint2*>(codes + at) = c;
  if ((unit & 15) == 0) scales[(size_t)row * ((d + kHeldGroup - 1) / kHeldGroup) + unit / 16] = scale;
}

// Row t of the codes to each of its k rows of the output (flat_to_sorted; entries that name no
// row are skipped), or to row t itself without a map. The codes are read once, for all k.
// STREAM: out is stored non-temporally.
template <typename T, bool WIDE, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void unpack_kernel(RowMap m, const uint8_t* __restrict__ codes,
                                                            const float* __restrict__ scales, int T_,
                                                            int k, int d,
                                                            const int32_t* __restrict__ f2s,
                                                            T* __restrict__ out) {
  unsigned t;
  int unit;
  row_unit<WIDE>(m, t, unit);
  if (t >= (unsigned)T_ || unit * 8 >= d) return;
  const uint2 c = *reinterpret_cast<const uint2*>(codes + (size_t)t * d + unit * 8);
  const float scale = scales[(size_t)t * ((d + kHeldGroup - 1) / kHeldGroup) + unit / 16];
  const F8 v = held8(c, scale);
  if (!f2s) {
    if constexpr (STREAM) store8_once(out + (size_t)t * d + unit * 8, v);
    else store8(out + (size_t)t * d + unit * 8, v);
    return;
  }
  const int R = T_ * k;
  for (int j = 0; j < k; ++j) {
    const int p = f2s[(size_t)t * k + j];
    if ((unsigned)p < (unsigned)R) {
      if constexpr (STREAM) store8_once(out + (size_t)p * d + unit * 8, v);
      else store8(out + (size_t)p * d + unit * 8, v);
    }
  }
}

struct SwigluArgs {
  const void *g, *u, *dh;
  const float *gs, *us;  // scales of held g and u
  void *h, *dg, *du;
  uint8_t *gc, *uc;
  float *gso, *uso;
  const int32_t* offsets;
  int E, rows, f;
};

// 1 / (1 + e^-g) for g >= kFar. For bf16 results the hardware's exp2 and reciprocal (each within
// one unit of fp32, and the product with log2 e within |g| 2^-24) are far inside the result's
// rounding.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896f));
  else return 1.0f / (1.0f + expf(-g));
}

// Below kFar s = e^g leaves the normal fp32 numbers (2^-126 at g = -87.3): the reciprocal would flush
// it to 0 and, from -88.7 on, e^-g would overflow, however large the factors that s meets. There the
// products are taken in 64 bits and rounded to fp32 once, with s = (e^(g/4))^4: a quarter's power
// is a normal fp32 number down to g = -349, where s is under 2^-503 and every product with fp32
// factors is 0. One comparison per 8 elements where no g is that low; these results are stored over
// the ordinary ones, which need not wait for them then (65,536 rows of 2048 forward and back: 387.2 us
// without this, 388.0 with it, 389.4 where one store comes after the branch).
constexpr float kFar = -87.0f;
__device__ __forceinline__ bool any_far(const F8& g) {
  float low = g.v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) low = fminf(low, g.v[i]);  // (NaN is passed over: it needs no care)
  return low < kFar;
}
template <typename T>
__device__ __forceinline__ double far_sigmoid(float g) {
  // bf16: the hardware's exp2 and the product with log2 e leave s within 2^-15 of itself, inside the rounding
  const double q = sizeof(T) == 2 ? __builtin_amdgcn_exp2f(g * (0.25f * 1.44269504088896f)) : expf(0.25f * g);
  return (q * q) * (q * q);
}

template <typename T>
__global__ __launch_bounds__(kRowThreads) void swiglu_kernel(RowMap m, SwigluArgs p) {
  unsigned row;
  int unit;
  row_unit(m, row, unit);
  if (row >= (unsigned)rows_in_use(p.offsets, p.E, p.rows)) return;
  const bool in = unit * 8 < p.f;
  const size_t at = (size_t)row * p.f + unit * 8;
  const F8 g = in ? load8_once(static_cast<const T*>(p.g) + at) : F8{};
  const F8 u = in ? load8_once(static_cast<const T*>(p.u) + at) : F8{};
  if (p.gc) {
    float gs, us;
    const uint2 cg = hold8(g, gs), cu = hold8(u, us);
    if (in) {
      *reinterpret_cast<uint2*>(p.gc + at) = cg;
      *reinterpret_cast<uint2*>(p.uc + at) = cu;
      if ((unit & 15) == 0) {
        const size_t s = (size_t)row * ((p.f + kHeldGroup - 1) / kHeldGroup) + unit / 16;
        p.gso[s] = gs;
        p.uso[s] = us;
      }
    }
  }
  if (!in) return;
  F8 h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h.v[i] = g.v[i] * sigmoid<T>(g.v[i]) * u.v[i];
  store8_once(static_cast<T*>(p.h) + at, h);
  if (any_far(g)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g.v[i] < kFar) h.v[i] = (float)(g.v[i] * far_sigmoid<T>(g.v[i]) * u.v[i]);
    store8_once(static_cast<T*>(p.h) + at, h);
  }
}

template <typename T, bool HELD>
__global__ __launch_bounds__(kRowThreads) void swiglu_backward_kernel(RowMap m, SwigluArgs p) {
  unsigned row;
  int unit;
  row_unit(m, row, unit);
  if (row >= (unsigned)rows_in_use(p.offsets, p.E, p.rows) || unit * 8 >= p.f) return;
  const size_t at = (size_t)row * p.f + unit * 8;
  F8 g, u;
  if constexpr (HELD) {
    const size_t s = (size_t)row * ((p.f + kHeldGroup - 1) / kHeldGroup) + unit / 16;
    g = held8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.g) + at), p.gs[s]);
    u = held8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.u) + at), p.us[s]);
  } else {
    g = load8_once(static_cast<const T*>(p.g) + at);
    u = load8_once(static_cast<const T*>(p.u) + at);
  }
  const F8 dh = load8_once(static_cast<const T*>(p.dh) + at);
  F8 dg, du, h;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid<T>(g.v[i]);
    const float silu = g.v[i] * s;
    h.v[i] = silu * u.v[i];
    du.v[i] = dh.v[i] * silu;
    dg.v[i] = dh.v[i] * u.v[i] * s * (1.0f + g.v[i] * (1.0f - s));
  }
  store8_once(static_cast<T*>(p.dg) + at, dg);
  store8_once(static_cast<T*>(p.du) + at, du);
  if (p.h) store8_once(static_cast<T*>(p.h) + at, h);
  if (any_far(g)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g.v[i] < kFar) {  // 1 - s is 1
        const double s = far_sigmoid<T>(g.v[i]), silu = g.v[i] * s;
        h.v[i] = (float)(silu * u.v[i]);
        du.v[i] = (float)(silu * dh.v[i]);
        dg.v[i] = (float)((double)dh.v[i] * u.v[i] * s * (1.0 + g.v[i]));
      }
    store8_once(static_cast<T*>(p.dg) + at, dg);
    store8_once(static_cast<T*>(p.du) + at, du);
    if (p.h) store8_once(static_cast<T*>(p.h) + at, h);
  }
}

}  // namespace

long long row_kernel_grid(long long rows, int d) {
  const long long whole_groups = row_grid(row_map((d + 127) / 128 * 16), rows), plain = row_grid(row_map(d / 8), rows);
  return whole_groups > plain ? whole_groups : plain;
}

hipError_t launch_pack(const void* x, bool bf16, int rows, int d, void* codes, float* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const RowMap m = row_map((d + 127) / 128 * 16);  // whole groups
  const unsigned grid = (unsigned)row_grid(m, rows);
  uint8_t* c = static_cast<uint8_t*>(codes);
  if (bf16)
    pack_kernel<<<grid, m.threads(), 0, stream>>>(m, static_cast<const __bf16*>(x), rows, d, c, scales);
  else
    pack_kernel<<<grid, m.threads(), 0, stream>>>(m, static_cast<const float*>(x), rows, d, c, scales);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_unpack_t(const void* codes, const float* scales, int T_, int k, int d, const int32_t* f2s,
                                  void* out, hipStream_t stream) {
  const RowMap m = row_map(d / 8);
  // Non-temporal stores pay where a store instruction writes whole lines and the rows do not fit the
  // last-level cache: to 65,536 bf16 rows of 7168 183 us against 199, of 7176 270 against 247, to
  // 16,384 of 7168 47 against 31. In fp32 an instruction writes half of each line: 874 us against 373.
  const bool past_cache = sizeof(T) == 2 && d % 64 == 0 && (long long)T_ * k * d * 2 > kCacheBytes;
  auto kern = m.shift < 6 ? &unpack_kernel<T, false, false>
                          : (past_cache ? &unpack_kernel<T, true, true> : &unpack_kernel<T, true, false>);
  kern<<<(unsigned)row_grid(m, T_), m.threads(), 0, stream>>>(m, static_cast<const uint8_t*>(codes), scales, T_, k, d,
                                                              f2s, static_cast<T*>(out));
  return hipGetLastError();
}

hipError_t launch_unpack(const void* codes, const float* scales, int T, int k, int d, const int32_t* f2s,
                         void* out, bool bf16, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  return (bf16 ? &launch_unpack_t<__bf16> : &launch_unpack_t<float>)(codes, scales, T, k, d, f2s, out, stream);
}

hipError_t launch_swiglu(const void* g, const void* u, bool bf16, const int32_t* offsets, int E, int rows,
                         int f, void* h, void* g_codes, float* g_scales, void* u_codes, float* u_scales,
                         hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  SwigluArgs p{};
  p.g = g; p.u = u; p.h = h;
  p.gc = static_cast<uint8_t*>(g_codes); p.uc = static_cast<uint8_t*>(u_codes);
  p.gso = g_scales; p.uso = u_scales;
  p.offsets = offsets; p.E = E; p.rows = rows; p.f = f;
  const RowMap m = row_map((f + 127) / 128 * 16);
  const unsigned grid = (unsigned)row_grid(m, rows);
  if (bf16)
    swiglu_kernel<__bf16><<<grid, m.threads(), 0, stream>>>(m, p);
  else
    swiglu_kernel<float><<<grid, m.threads(), 0, stream>>>(m, p);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const void* dh, bool bf16, const void* g, const void* u, bool held,
                                  const float* g_scales, const float* u_scales, const int32_t* offsets,
                                  int E, int rows, int f, void* dg, void* du, void* h, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  SwigluArgs p{};
  p.g = g; p.u = u; p.dh = dh; p.gs = g_scales; p.us = u_scales;
  p.h = h; p.dg = dg; p.du = du;
  p.offsets = offsets; p.E = E; p.rows = rows; p.f = f;
  const RowMap m = row_map(f / 8);
  const unsigned grid = (unsigned)row_grid(m, rows);
  auto kern = bf16 ? (held ? &swiglu_backward_kernel<__bf16, true> : &swiglu_backward_kernel<__bf16, false>)
                   : (held ? &swiglu_backward_kernel<float, true> : &swiglu_backward_kernel<float, false>);
  kern<<<grid, m.threads(), 0, stream>>>(m, p);
  return hipGetLastError();
}

}  // namespace moe
