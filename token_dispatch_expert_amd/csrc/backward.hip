// Backward passes of combine, permute and route: a layer's gradient from the tokens to the
// expert-sorted rows and back, and to the router's logits.
//
//   combine  y[t]  = sum_j gate[t,j] ys[p(t,j)]    dys[p] = gate dy[t],  dgate[t,j] = <dy[t], ys[p]>
//   permute  xs[p(t,j)] = x[t]                     dx[t]  = sum_j dxs[p(t,j)]
//   route    gate = softmax of the k chosen logits dlogit[t, id_j] = g_j (dg_j - sum_i g_i dg_i)
// p(t, j) = flat_to_sorted[t*k + j]; an entry that names no row (an assignment dropped for its
// expert's capacity) has no gradient. Sums are fp32 in a fixed order, without atomics.
//
// Combine and permute are bound by HBM. 8,192 tokens, 8 experts each, d = 7168, bf16 gradients: combine
// 540 - 568 us (2.9 GB: y_sorted once, dy once per token, dy_sorted written; 5.2 - 5.4 TB/s, where a copy of
// 2 GiB reaches 4.8), permute 168 - 176 us (1.06 GB, 6.0 - 6.3 TB/s). Route, 256 experts, 7.1 us for 8.4 MB:
// an almost empty launch of it takes 2.6 - 2.9 us, then a wave's 4 stores of 256 bytes follow a loop over
// the k slots each.
#include "rows.h"

namespace moe {

namespace {

// The row of the sorted order that assignment i goes to, or -1.
__device__ __forceinline__ int sorted_row(const int32_t* f2s, long long i, int R) {
  const int p = f2s[i];
  return (unsigned)p < (unsigned)R ? p : -1;
}

// One assignment (t, j) per group of WAVES waves: 4 / WAVES assignments per workgroup. A
// token's k assignments go to consecutive workgroups of one XCD (workgroup b runs on XCD
// b % 8), so that dy[t] is read from HBM once and then from that XCD's L2. One workgroup for all of a
// token's assignments, with dy[t] in registers, took 571 us against 541.
// STREAM: dys is stored non-temporally (a branch in the kernel would be merged into plain stores).
template <typename TI, typename TO, int WAVES, bool STREAM>
__global__ __launch_bounds__(256) void combine_backward_kernel(const TI* __restrict__ dy,
                                                              const float* __restrict__ ys,
                                                              const int32_t* __restrict__ f2s,
                                                              const float* __restrict__ gates, int T,
                                                              int k, int d, TO* __restrict__ dys,
                                                              float* __restrict__ dgates) {
  constexpr int PER = 4 / WAVES;  // assignments per workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned x = blockIdx.x & 7, i = blockIdx.x >> 3;
  const long long slot = (long long)i * PER + wave / WAVES;  // this XCD's assignments in order
  const long long t = slot / k * 8 + x;
  const int j = (int)(slot % k);
  const bool live = t < T;
  const long long a = t * k + j;
  const int p = live ? sorted_row(f2s, a, T * k) : -1;
  float dot = 0.f;
  if (p >= 0) {
    const float g = gates[a];
    const TI* src = dy + (size_t)t * d;
    const float* y = ys ? ys + (size_t)p * d : nullptr;
    TO* dst = dys + (size_t)p * d;
    for (int c = ((wave % WAVES) * 64 + lane) * 8; c < d; c += WAVES * 512) {
      const F8 v = load8(src + c);
      F8 o;
#pragma unroll
      for (int q = 0; q < 8; ++q) o.v[q] = g * v.v[q];
      if constexpr (STREAM) store8_once(dst + c, o);
      else store8(dst + c, o);
      if (y) {
        const F8 w = load8_once(y + c);
#pragma unroll
        for (int q = 0; q < 8; ++q) dot = fmaf(v.v[q], w.v[q], dot);
      }
    }
  }
  if (!dgates) return;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) dot += __shfl_xor(dot, s);
  if constexpr (WAVES > 1) {
    __shared__ float part[4];
    if (lane == 0) part[wave] = dot;
    __syncthreads();
    dot = part[0] + part[1] + part[2] + part[3];
  }
  if (live && lane == 0 && wave % WAVES == 0) dgates[a] = p >= 0 ? dot : 0.f;
}

constexpr int kSumBatch = 8;  // rows whose loads are in flight together

template <typename TI, typename TO, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void permute_backward_kernel(RowMap m, const TI* __restrict__ dxs,
                                                                      const int32_t* __restrict__ f2s,
                                                                      int T, int k, int d,
                                                                      TO* __restrict__ dx) {
  unsigned t;
  int unit;
  row_unit<WIDE>(m, t, unit);
  if (t >= (unsigned)T || unit * 8 >= d) return;
  F8 acc{};
  for (int j0 = 0; j0 < k; j0 += kSumBatch) {
    F8 v[kSumBatch];
#pragma unroll
    for (int u = 0; u < kSumBatch; ++u) {
      const int p = j0 + u < k ? sorted_row(f2s, (long long)t * k + j0 + u, T * k) : -1;
      v[u] = p >= 0 ? load8_once(dxs + (size_t)p * d + unit * 8) : F8{};
    }
#pragma unroll
    for (int u = 0; u < kSumBatch; ++u)
#pragma unroll
      for (int q = 0; q < 8; ++q) acc.v[q] += v[u].v[q];
  }
  store8_once(dx + (size_t)t * d + unit * 8, acc);
}

// One wave per token; lane j holds slot j, the lanes then write the row 64 experts at a time.
// A slot whose id is no expert adds nothing; slots with the same id add up in slot order.
__global__ __launch_bounds__(256) void route_backward_kernel(const float* __restrict__ dgates,
                                                            const int32_t* __restrict__ ids,
                                                            const float* __restrict__ gates, int T,
                                                            int E, int k, float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const unsigned t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= (unsigned)T) return;
  const bool on = lane < k;
  const size_t a = (size_t)t * k + lane;
  const float g = on ? gates[a] : 0.f, dg = on ? dgates[a] : 0.f;
  const int id = on ? ids[a] : -1;
  float mean = g * dg;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) mean += __shfl_xor(mean, s);
  const float v = g * (dg - mean);
  for (int e = lane; e < ((E + 63) & ~63); e += 64) {
    float o = 0.f;
    for (int j = 0; j < k; ++j) {
      const int idj = __builtin_amdgcn_readlane(id, j);
      const float vj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
      o += idj == e ? vj : 0.f;
    }
    if (e < E) dlogits[(size_t)t * E + e] = o;
  }
}

// Workgroups of combine_backward_kernel: a row of more than 1024 elements takes a whole workgroup, else a
// wave. Four waves to a row against one, 8,192 tokens: d = 1024 100 and 80 us, 1544 146 and 127 (a
// workgroup takes 2048 elements at a time, so that waves idle up to there), 2048 176 and 173, 4096 325 and
// 334; 64 tokens: 1544 4.4 and 4.3, 4096 4.3 and 5.7.
constexpr int kWideRow = 1024;

template <typename TI, typename TO>
hipError_t launch_combine_backward_t(const void* dy, const float* ys, const int32_t* f2s, const float* gates,
                                     int T, int k, int d, void* dys, float* dgates, hipStream_t stream) {
  const unsigned grid = (unsigned)combine_backward_grid(T, k, d);
  const TI* s = static_cast<const TI*>(dy);
  TO* o = static_cast<TO*>(dys);
  // Rows that do not fit the last-level cache are stored non-temporally: 940 MB of them 568 us against
  // 601; 235 MB, which the next product finds there, 145 against 138.
  const bool past_cache = (long long)T * k * d * (long long)sizeof(TO) > kCacheBytes;
  auto kern = d > kWideRow ? (past_cache ? &combine_backward_kernel<TI, TO, 4, true> : &combine_backward_kernel<TI, TO, 4, false>)
                           : (past_cache ? &combine_backward_kernel<TI, TO, 1, true> : &combine_backward_kernel<TI, TO, 1, false>);
  kern<<<grid, 256, 0, stream>>>(s, ys, f2s, gates, T, k, d, o, dgates);
  return hipGetLastError();
}

}  // namespace

long long combine_backward_grid(int T, int k, int d) {
  const long long per_xcd = (T + 7LL) / 8 * k;  // assignments
  return 8 * (d > kWideRow ? per_xcd : (per_xcd + 3) / 4);
}

hipError_t launch_combine_backward(const void* dy, bool dy_bf16, const float* ys, const int32_t* f2s,
                                   const float* gates, int T, int k, int d, void* dys, bool out_bf16,
                                   float* dgates, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  auto f = dy_bf16 ? (out_bf16 ? &launch_combine_backward_t<__bf16, __bf16> : &launch_combine_backward_t<__bf16, float>)
                   : (out_bf16 ? &launch_combine_backward_t<float, __bf16> : &launch_combine_backward_t<float, float>);
  return f(dy, ys, f2s, gates, T, k, d, dys, dgates, stream);
}

template <typename TI, typename TO>
static hipError_t launch_permute_backward_t(const void* dxs, const int32_t* f2s, int T, int k, int d, void* dx,
                                            hipStream_t stream) {
  const RowMap m = row_map(d / 8);
  auto kern = m.shift >= 6 ? &permute_backward_kernel<TI, TO, true> : &permute_backward_kernel<TI, TO, false>;
  kern<<<(unsigned)row_grid(m, T), m.threads(), 0, stream>>>(m, static_cast<const TI*>(dxs), f2s, T, k, d,
                                                             static_cast<TO*>(dx));
  return hipGetLastError();
}

hipError_t launch_permute_backward(const void* dxs, bool bf16, const int32_t* f2s, int T, int k, int d,
                                   void* dx, bool out_bf16, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  auto f = bf16 ? (out_bf16 ? &launch_permute_backward_t<__bf16, __bf16> : &launch_permute_backward_t<__bf16, float>)
                : (out_bf16 ? &launch_permute_backward_t<float, __bf16> : &launch_permute_backward_t<float, float>);
  return f(dxs, f2s, T, k, d, dx, stream);
}

hipError_t launch_route_backward(const float* dgates, const int32_t* ids, const float* gates, int T, int E,
                                 int k, float* dlogits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  route_backward_kernel<<<(unsigned)((T + 3LL) / 4), 256, 0, stream>>>(dgates, ids, gates, T, E, k, dlogits);
  return hipGetLastError();
}

}  // namespace moe
