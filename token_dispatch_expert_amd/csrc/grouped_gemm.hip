// Matrix products grouped by expert over expert-sorted rows: the forward product, its input
// gradient and its weight gradient.
//
// Expert e owns rows r in [offsets[e], offsets[e+1]) and the matrix W_e [N, K] (row-major):
//   forward  y[r]  = W_e x[r]                          contraction over K
//   dgrad    dx[r] = W_e^T dy[r] (+ W2_e^T dy2[r])     contraction over N
//   wgrad    dW_e  = sum_r dy[r] x[r]^T                contraction over the expert's rows
// Products of the operands' values are summed in fp32; the result is rounded once, to the
// output's format.
//
// As C = A B with the contraction axis either contiguous in memory ("along") or the row axis of
// the stored matrix ("across"):
//   forward  A = x along K,   B = W along K
//   dgrad    A = dy along N,  B = W across N
//   wgrad    A = dy across r, B = x across r
#include "grouped.h"

namespace moe {

namespace {

// ---------------------------------------------------------------------------------------
// Tiles staged through registers, fp32 matrix instructions
// ---------------------------------------------------------------------------------------
// A workgroup of 4 waves (2 x 2) computes a TM x TM tile of C; the contraction goes in steps of
// 32. Both operands lie in LDS as fp32 in their memory order: along operands [m][32 + 4],
// across operands [32][m + 4]; the padding of 4 floats puts the 16 rows (or 4 row groups) of a
// fragment read on distinct banks. v_mfma_f32_16x16x4_f32 takes one contraction element per
// lane (row or column lane % 16, element lane / 16); lane group g takes elements 4g .. 4g + 3
// of a 16-long slice in turn, the same for both operands, so an along fragment is one 16-byte
// read. The operands go in as (B, A), which gives each lane 4 consecutive columns of one row of
// C: one 16-byte (fp32) or 8-byte (bf16) store.
constexpr int kStep = 32;
constexpr int kPad = 4;

template <typename T> struct Chunk;  // 4 elements as stored
template <> struct Chunk<float> { float4 v; };
template <> struct Chunk<__bf16> { uint2 v; };

__device__ __forceinline__ float4 widen(const Chunk<float>& c) { return c.v; }
__device__ __forceinline__ float4 widen(const Chunk<__bf16>& c) {
  return make_float4(__uint_as_float(c.v.x << 16), __uint_as_float(c.v.x & 0xffff0000u),
                     __uint_as_float(c.v.y << 16), __uint_as_float(c.v.y & 0xffff0000u));
}

struct ProductArgs {
  const void *a, *b, *a2, *b2;  // a2, b2: second pair of operands (dgrad), or null
  void* out;
  const int32_t* offsets;
  int rows, E, N, K;
  int out_bf16, accumulate;
};

// One row's 4 consecutive columns of C.
__device__ __forceinline__ void store4(const ProductArgs& p, size_t at, f32x4 v) {
  if (p.out_bf16) {
    bf16x4* o = reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p.out) + at);
    if (p.accumulate) {
      const bf16x4 old = *o;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += (float)old[j];
    }
    *o = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
  } else {
    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at);
    if (p.accumulate) v += *o;
    *o = v;
  }
}

// One operand of one step: TM rows (along) or columns (across) of C's side, 32 of the
// contraction. base: the operand's first element of the tile; lim: rows or columns of the tile
// that exist; ld: its row stride; k0, kdim: the step's first contraction element and their
// number. What lies outside reads as zero.
template <typename T, bool ACROSS, int TM>
struct Stage {
  static constexpr int NCH = TM * kStep / 4 / 256;  // chunks per thread
  Chunk<T> c[NCH];
  __device__ __forceinline__ static void at(int i, int& outer, int& inner) {
    const int q = threadIdx.x + i * 256;
    constexpr int per = (ACROSS ? TM : kStep) / 4;  // chunks per LDS row
    outer = q / per;
    inner = q % per * 4;
  }
  __device__ __forceinline__ void load(const T* base, int lim, int ld, int k0, int kdim) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      int o, n;
      at(i, o, n);
      const bool ok = ACROSS ? (k0 + o < kdim && n < lim) : (o < lim && k0 + n < kdim);
      const size_t e = ACROSS ? (size_t)(k0 + o) * ld + n : (size_t)o * ld + k0 + n;
      c[i] = ok ? *reinterpret_cast<const Chunk<T>*>(base + e) : Chunk<T>{};
    }
  }
  __device__ __forceinline__ void put(float* lds) const {
    constexpr int row = (ACROSS ? TM : kStep) + kPad;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      int o, n;
      at(i, o, n);
      *reinterpret_cast<float4*>(lds + o * row + n) = widen(c[i]);
    }
  }
};

template <bool ACROSS, int TM>
__device__ __forceinline__ f32x4 fragment(const float* lds, int m, int k) {
  if constexpr (ACROSS) {
    const float* s = lds + k * (TM + kPad) + m;
    return f32x4{s[0], s[TM + kPad], s[2 * (TM + kPad)], s[3 * (TM + kPad)]};
  } else {
    const float4 v = *reinterpret_cast<const float4*>(lds + m * (kStep + kPad) + k);
    return f32x4{v.x, v.y, v.z, v.w};
  }
}

template <bool ACROSS, int TM>
constexpr int stage_floats() { return ACROSS ? kStep * (TM + kPad) : TM * (kStep + kPad); }

template <typename T, GroupedProduct P, int TM>
__global__ __launch_bounds__(256) void product_kernel(ProductArgs p) {
  constexpr bool AX = P == kWgrad, BX = P != kForward;
  constexpr int FR = TM / 32;  // 16-wide fragments per wave and side
  __shared__ __align__(16) float la[stage_floats<AX, TM>()];
  __shared__ __align__(16) float lb[stage_floats<BX, TM>()];
  const long long item = xcd_item(blockIdx.x);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int cols = P == kForward ? p.N : p.K;
  const int CT = (cols + TM - 1) / TM;
  int e, ra, rb, mt, nt;
  if constexpr (P == kWgrad) {
    const int MT = (p.N + TM - 1) / TM;
    if (item >= (long long)p.E * MT * CT) return;
    const int local = (int)(item % ((long long)MT * CT));
    e = expert_of_rank(p.offsets, p.E, p.rows, (int)(item / ((long long)MT * CT)));
    group_rows(p.offsets, e, p.rows, ra, rb);
    mt = local / CT;
    nt = local % CT;
    if (ra == rb && p.accumulate) return;
  } else {
    if (!find_row_tile(p.offsets, p.E, p.rows, TM, CT, item, e, ra, rb, mt, nt)) return;
  }
  // C's rows and columns of the tile
  const int m0 = mt * TM, c0 = nt * TM;
  const int mlim = min(TM, (P == kWgrad ? p.N : rb - ra) - m0), clim = min(TM, cols - c0);
  const int kdim = P == kForward ? p.K : (P == kDgrad ? p.N : rb - ra);
  const int lda = P == kForward ? p.K : p.N;
  const size_t wbase = (size_t)e * p.N * p.K;
  const size_t a_at = P == kWgrad ? (size_t)ra * p.N + m0 : (size_t)(ra + m0) * lda;
  const size_t b_at = P == kForward ? wbase + (size_t)c0 * p.K
                      : P == kDgrad ? wbase + c0 : (size_t)ra * p.K + c0;

  f32x4 acc[FR][FR];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps1 = (kdim + kStep - 1) / kStep;
  const int steps = (P == kDgrad && p.a2) ? 2 * steps1 : steps1;
  Stage<T, AX, TM> sa;
  Stage<T, BX, TM> sb;
  auto load = [&](int st) __attribute__((always_inline)) {
    const bool second = st >= steps1;
    const int k0 = (second ? st - steps1 : st) * kStep;
    sa.load(static_cast<const T*>(second ? p.a2 : p.a) + a_at, mlim, lda, k0, kdim);
    sb.load(static_cast<const T*>(second ? p.b2 : p.b) + b_at, clim, p.K, k0, kdim);
  };
  if (steps > 0) load(0);
  for (int st = 0; st < steps; ++st) {
    __syncthreads();  // the previous step's reads are done
    sa.put(la);
    sb.put(lb);
    __syncthreads();
    if (st + 1 < steps) load(st + 1);  // in flight under the products
#pragma unroll
    for (int s = 0; s < kStep / 16; ++s) {
      const int k = s * 16 + (lane >> 4) * 4;
      f32x4 fa[FR], fb[FR];
#pragma unroll
      for (int i = 0; i < FR; ++i) fa[i] = fragment<AX, TM>(la, (wm * FR + i) * 16 + (lane & 15), k);
#pragma unroll
      for (int i = 0; i < FR; ++i) fb[i] = fragment<BX, TM>(lb, (wn * FR + i) * 16 + (lane & 15), k);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < FR; ++i)
#pragma unroll
          for (int j = 0; j < FR; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j][q], fa[i][q], acc[i][j], 0, 0, 0);
    }
  }
  const size_t crow0 = P == kWgrad ? (size_t)e * p.N + m0 : (size_t)ra + m0;
#pragma unroll
  for (int i = 0; i < FR; ++i) {
    const int r = (wm * FR + i) * 16 + (lane & 15);
    if (r >= mlim) continue;
#pragma unroll
    for (int j = 0; j < FR; ++j) {
      const int c = (wn * FR + j) * 16 + (lane >> 4) * 4;
      if (c < clim) store4(p, (crow0 + r) * cols + c0 + c, acc[i][j]);
    }
  }
}

// Tiles that a launch covers: for wgrad every expert's, for the row products the most that the
// rows can fill (an expert's last row tile may be partial).
long long tile_items(GroupedProduct kind, const GroupedGemmArgs& a, int TM) {
  const long long nt = (a.N + TM - 1) / TM, kt = (a.K + TM - 1) / TM;
  if (kind == kWgrad) return a.E * nt * kt;
  const long long mt = a.rows / TM + (a.E < a.rows ? a.E : a.rows);
  return mt * (kind == kForward ? nt : kt);
}

template <typename T, GroupedProduct P, int TM>
hipError_t launch_tiles(const GroupedGemmArgs& a, const ProductArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(P, a, TM));
  product_kernel<T, P, TM><<<(unsigned)grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <GroupedProduct P>
hipError_t launch_product(const GroupedGemmArgs& a, hipStream_t stream) {
  const ProductArgs p{a.a, a.b, a.a2, a.b2, a.out, a.offsets, a.rows, a.E, a.N, a.K,
                      a.out_bf16 ? 1 : 0, a.accumulate ? 1 : 0};
  return a.bf16 ? launch_tiles<__bf16, P, 64>(a, p, stream) : launch_tiles<float, P, 64>(a, p, stream);
}

}  // namespace

bool grouped_gemm_fits(const GroupedGemmArgs& a, GroupedProduct kind) {
  return xcd_grid(tile_items(kind, a, 64)) <= 0x7fffffffLL;
}

hipError_t launch_grouped_gemm(const GroupedGemmArgs& a, GroupedProduct kind, hipStream_t stream) {
  switch (kind) {
    case kForward: return launch_product<kForward>(a, stream);
    case kDgrad: return launch_product<kDgrad>(a, stream);
    case kWgrad: return launch_product<kWgrad>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
