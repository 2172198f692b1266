// Matrix products grouped by expert with MXFP4 weights (the format is in mxfp4.h): y[r] = W_e x[r] with rows
// x in bf16 or in MXFP4, and the gate and up products with SwiGLU in the epilogue.
//
// Rows in MXFP4 go with the weights' codes into v_mfma_scale_f32_16x16x128_f8f6f4, which takes 16
// elements x 128 of each operand and a scale byte per lane: lane r + 16 g holds row r and one group of 32 elements,
// with its scale. Weights that meet bf16 rows are converted in registers, exactly, and go into
// v_mfma_f32_16x16x32_bf16. Both sum in fp32.
//
// The order in which a product takes its contraction elements is free as long as both operands agree, and it
// is chosen such that each lane's part of a step lies together: with Q = DK / 4 elements of a step for
// each of the four lane groups, group g takes elements Q g .. Q g + Q - 1, slice after slice. A lane's codes of a
// step are then Q / 2 consecutive bytes, and its scales Q / 32 consecutive ones.
#include "mxfp4.h"
#include "mxfp4_internal.h"
#include "product_tiles.h"
#include "swiglu.h"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct MxProductArgs {
  ProductArgs p;                          // a: x, b: W (gate), b2: up
  const uint8_t *a_scales, *b_scales, *b2_scales;
  uint8_t* out_scales;                    // h in MXFP4
};

// Chunk c of 16 bytes of a row of CPR chunks sits at c ^ x(row), so that the 16 rows that a fragment read
// meets (one chunk of each) fall on distinct banks.
template <int CPR>
__device__ __forceinline__ int swizzle(int row) {
  static_assert(CPR == 2 || CPR == 4 || CPR == 8 || CPR == 16 || CPR == 32, "row width");
  if constexpr (CPR == 2) return row >> 3 & 1;
  else if constexpr (CPR == 4) return row >> 2 & 3;
  else if constexpr (CPR == 8) return row >> 1 & 7;
  else return row & 15;
}

// One operand of a tile: T rows of ROWB bytes per step, loaded by NW waves with buffer loads of 1 KB into LDS. PAIR:
// units of U rows of two matrices in turn (gate, up, gate, ..).
template <int T, int ROWB, int NW, bool PAIR>
struct Tile {
  static constexpr int CPR = ROWB / 16, kChunks = T * CPR, kLoads = kChunks / 64 / NW, kRowsPerLoad = 64 / CPR;
  static constexpr int U = kRowsPerLoad > 16 ? kRowsPerLoad : 16;
  static_assert(kLoads >= 1 && kLoads * 64 * NW == kChunks, "loads split evenly over the waves");
  static_assert(kRowsPerLoad * NW % 16 == 0, "the permutation repeats from one load to the next");
  static_assert(!PAIR || T % (2 * U) == 0, "whole pairs of units");
  static constexpr int kOutside = 0x40000000;  // past any extent (at most 256 rows of 2^21 bytes)

  const char *base, *base2;
  int extent, ld, lane_at, at_in_row;

  // first, count: the tile's first row in the matrix (PAIR: in each of the two) and how many exist
  __device__ __forceinline__ void set(const void* origin, const void* origin2, size_t first, int count, int row_bytes,
                                      int wave, int lane) {
    ld = row_bytes;
    base = static_cast<const char*>(origin) + first * row_bytes;
    base2 = static_cast<const char*>(origin2) + first * row_bytes;
    extent = count * row_bytes;
    const int row = lane / CPR, pos = lane % CPR;
    at_in_row = (pos ^ swizzle<CPR>(wave * kRowsPerLoad + row)) * 16;
    lane_at = row * row_bytes + at_in_row;
  }
  // bytes byte0 .. byte0 + ROWB - 1 of each row into `slot`; past the end of a row (`left` bytes from byte0 on) and
  // in rows that do not exist zeros
  template <int AUX>
  __device__ __forceinline__ void issue(u32x4* slot, int byte0, int left, int wave) const {
    const int at = at_in_row < left ? lane_at : kOutside;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int l = wave + i * NW, r0 = l * kRowsPerLoad;
      const int row0 = PAIR ? (r0 / (2 * U)) * U + r0 % U : r0;
      const char* b = PAIR && (r0 / U & 1) ? base2 : base;
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)b, (short)0, extent, kBufferWord3);
      buffer_load_lds16<AUX>(r, slot + l * 64, at + row0 * ld, byte0);
    }
  }
  // 16 bytes: chunk c of row m of the slot
  __device__ __forceinline__ static u32x4 read(const u32x4* slot, int m, int c) {
    return slot[m * CPR + (c ^ swizzle<CPR>(m))];
  }
};

// 4 bytes a lane from a buffer into LDS at lds + 4 * lane
__device__ __forceinline__ void buffer_load_lds4(__amdgpu_buffer_rsrc_t rsrc, void* lds, int voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)lds, 4, voffset, 0, 0, 0);
}
// The 8 scale bytes of n rows for a block of 256 elements, into an area of kScaleArea(n) bytes: `load` is
// the number of the 256-byte load.
constexpr int scale_loads(int n) { return (n * 8 + 255) / 256; }
__device__ __forceinline__ void issue_scales(const uint8_t* from, int count, char* area, int load, int lane) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)from, (short)0, count * 8, kBufferWord3);
  buffer_load_lds4(r, area + load * 256, load * 256 + lane * 4);
}

// h = silu(g) u; far results as in swiglu.h
__device__ __forceinline__ float silu_times(float g, float u) {
  float h = g * sigmoid<__bf16>(g) * u;
  if (g < kFar) h = (float)(g * far_sigmoid<__bf16>(g) * u);
  return h;
}

// 16 rows of h from r0 and NH * 16 columns from c0 of the tile, as groups of 32 in MXFP4. v as in store_fragments.
// The codes are rounded from the fp32 value, once.
template <int NH>
__device__ __forceinline__ void store_mxfp4(const MxProductArgs& a, const TileAt& t, const f32x4 (&v)[NH], int r0, int c0,
                                            int lane) {
  static_assert(NH % 2 == 0, "whole groups");
  const int g = lane >> 4, r = r0 + (lane & 15);
#pragma unroll
  for (int j = 0; j < NH; j += 2) {
    const int c = c0 + j * 16;
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      top = max(top, max(__float_as_uint(v[j][i]) & 0x7fffffffu, __float_as_uint(v[j + 1][i]) & 0x7fffffffu));
    top = max(top, (unsigned)__shfl_xor((int)top, 16));
    top = max(top, (unsigned)__shfl_xor((int)top, 32));
    const int scale = mx_scale(top);
    const float inv = mx_inverse(scale);
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = v[j][i] * inv;
      q[4 + i] = v[j + 1][i] * inv;
    }
    // columns 4g .. 4g + 3 in the low half, 16 more in the high one; the row's 16 bytes are the low
    // halves of its four lanes, then the high ones
    const unsigned mine = scale == kMxNan ? 0u : mx_codes8(q);
    const unsigned next = (unsigned)__shfl_xor((int)mine, 16);
    const u32x2 two = (g & 1) ? u32x2{next & 0xffffu | mine << 16, next >> 16 | mine & 0xffff0000u}
                              : u32x2{mine & 0xffffu | next << 16, mine >> 16 | next & 0xffff0000u};
    const u32x2 far{(unsigned)__shfl_xor((int)two[0], 32), (unsigned)__shfl_xor((int)two[1], 32)};
    if (g == 0 && r < t.mlim && c < t.clim) {
      const size_t row = (size_t)t.ra + t.m0 + r;
      const int col = t.c0 + c;
      *reinterpret_cast<u32x4*>(static_cast<char*>(a.p.out) + (row * a.p.N + col) / 2) = u32x4{two[0], far[0], two[1], far[1]};
      a.out_scales[mx_scale_at(0, 0, col / kMxBlock, a.p.rows, row) + (col / kMxGroup & 7)] = (uint8_t)scale;
    }
  }
}

// A workgroup of WGM x WGN waves computes a tile of C, each wave WM x WN of it; steps of DK contraction elements go
// through a ring of RING slots in LDS, the scales of a block of 256 elements through a ring of their own. X4: rows in
// MXFP4. PAIR: the tile's columns are those of two matrices, U of the one and U of the other in turn, so that a wave
// holds gate and up of the same columns of h.
template <bool X4, bool PAIR, int WM, int WN, int WGM, int WGN, int DK, int RING, bool ONCE, bool DEAL>
__global__ __launch_bounds__(64 * WGM * WGN) void mx_kernel(MxProductArgs a) {
  constexpr int TM = WM * WGM, TN = WN * WGN, NW = WGM * WGN;
  constexpr int MF = WM / 16, NF = WN / 16;
  constexpr int NS = DK / (X4 ? 128 : 32);  // slices of a step: one matrix instruction per pair of fragments
  constexpr int Q = DK / 4;                 // elements of a step per lane group
  using OA = Tile<TM, X4 ? DK / 2 : DK * 2, NW, false>;
  using OB = Tile<TN, DK / 2, NW, PAIR>;
  constexpr int STAGE = OA::kChunks + OB::kChunks, LOADS = OA::kLoads + OB::kLoads;
  constexpr int SPB = kMxBlock / DK;        // steps per block of scales
  constexpr int SR = (RING + SPB - 2) / SPB + 1;  // blocks that RING steps in a row may meet
  constexpr int LA = X4 ? scale_loads(TM) : 0, LB = scale_loads(PAIR ? TN / 2 : TN), LT = LA + LB * (PAIR ? 2 : 1);
  static_assert(DK <= kMxBlock && (!X4 || DK == kMxBlock), "steps within a block");
  static_assert(!PAIR || WN % (2 * OB::U) == 0, "a wave holds whole pairs");
  static_assert((RING * STAGE * 16 + SR * LT * 256) <= 160 * 1024, "LDS");
  __shared__ __align__(16) u32x4 ring[RING * STAGE];
  __shared__ __align__(16) char scale_ring[SR * LT * 256];
  const ProductArgs& p = a.p;
  TileAt t;
  if (!tile_at<kForward, DEAL>(p, TM, PAIR ? TN / 2 : TN, t)) return;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WGN * WM, wn = wave % WGN * WN;
  const int K = p.K, blocks = mx_blocks(K), steps = (K + DK - 1) / DK;

  OA oa;
  OB ob;
  const size_t row0 = (size_t)t.ra + t.m0;
  const int a_bytes = X4 ? K / 2 : K * 2;
  oa.set(p.a, p.a, row0, t.mlim, a_bytes, wave, lane);
  const size_t we = (size_t)t.e * p.N * (K / 2);
  ob.set(static_cast<const char*>(p.b) + we, PAIR ? static_cast<const char*>(p.b2) + we : nullptr, t.c0, t.clim, K / 2,
         wave, lane);
  // The expert's weights are read by this row tile alone, in whole lines.
  const bool once = ONCE && DK == kMxBlock && t.rb - t.ra <= TM && K % kMxBlock == 0;

  auto issue = [&](int st) __attribute__((always_inline)) {
    // A block's scales go before the first step that uses them: whoever waits for that step's operands has them too.
    if (SPB == 1 || st % SPB == 0) {
      const int b = st / SPB;
      char* area = scale_ring + b % SR * (LT * 256);
      const size_t wb = mx_scale_at(t.e, blocks, b, p.N, t.c0);
#pragma unroll
      for (int i = 0; i < (LT + NW - 1) / NW; ++i) {
        const int l = wave + i * NW;
        if (X4 && l < LA) issue_scales(a.a_scales + mx_scale_at(0, 0, b, p.rows, row0), t.mlim, area, l, lane);
        else if (l < LA + LB) issue_scales(a.b_scales + wb, t.clim, area + LA * 256, l - LA, lane);
        else if (PAIR && l < LT) issue_scales(a.b2_scales + wb, t.clim, area + (LA + LB) * 256, l - LA - LB, lane);
      }
    }
    u32x4* slot = ring + st % RING * STAGE;
    const int k0 = st * DK;
    oa.template issue<0>(slot, X4 ? k0 / 2 : k0 * 2, a_bytes - (X4 ? k0 / 2 : k0 * 2), wave);
    if (once) ob.template issue<kNonTemporal>(slot + OA::kChunks, k0 / 2, (K - k0) / 2, wave);
    else ob.template issue<0>(slot + OA::kChunks, k0 / 2, (K - k0) / 2, wave);
  };
  // Scales of this lane's groups of step st: byte i for its i-th group. Groups past K hold zeros under whatever their scale
  // bytes are; their scale is taken to be 2^-127, so that zeros they stay.
  const int groups = K / kMxGroup;
  auto scales_of = [&](const char* rows, int m, int st) __attribute__((always_inline)) {
    const int first = st * (DK / kMxGroup) + (DK >= 128 ? lg * (Q / 32) : lg / 2);  // group of the whole row
    const char* at = rows + (m + lr) * 8 + (first & 7);
    if constexpr (DK == 256) {
      const unsigned s = *reinterpret_cast<const unsigned short*>(at);
      return first + 1 < groups ? s : (first < groups ? s & 0xffu : 0u);
    } else {
      const unsigned s = *reinterpret_cast<const unsigned char*>(at);
      return first < groups ? s : 0u;
    }
  };
  auto a_scales = [&](int st, int i) __attribute__((always_inline)) {
    return scales_of(scale_ring + st / SPB % SR * (LT * 256), wm + i * 16, st);
  };
  auto b_scales = [&](int st, int j) __attribute__((always_inline)) {
    const char* area = scale_ring + st / SPB % SR * (LT * 256) + LA * 256;
    const int n = wn + j * 16;
    if constexpr (PAIR) {
      constexpr int U = OB::U;
      return scales_of(area + (n / U & 1) * (LB * 256), n / (2 * U) * U + n % U, st);
    } else {
      return scales_of(area, n, st);
    }
  };

  auto run = [&](auto present) __attribute__((always_inline)) {
    constexpr int F = decltype(present)::value;
    f32x4 acc[F ? F : 1][NF];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 fa[F ? F : 1];
    unsigned sa[F ? F : 1], sb[NF], sn[NF];  // sn: the next step's
    u32x4 fb[2][NF];  // X4: codes; else bf16 values
    auto read_a = [&](const u32x4* slot, int i, int h) __attribute__((always_inline)) {
      return OA::read(slot, wm + i * 16 + lr, lg * NS + h);
    };
    // B's fragment of slice h: the codes of 32 elements (X4), or 8 elements converted
    auto read_b = [&](const u32x4* slot, int j, int h, unsigned scale) __attribute__((always_inline)) {
      const int n = wn + j * 16 + lr;
      if constexpr (X4) {
        return OB::read(slot + OA::kChunks, n, lg * NS + h);
      } else {
        const int byte = lg * (Q / 2) + h * 4, c = byte / 16;
        const unsigned* at = reinterpret_cast<const unsigned*>(slot + OA::kChunks + n * OB::CPR + (c ^ swizzle<OB::CPR>(n)));
        const unsigned s = DK == 256 ? (h < NS / 2 ? scale & 0xffu : scale >> 8) : scale;
        return __builtin_bit_cast(u32x4, mx_bf16x8(at[byte / 4 % 4], mx_scale_f32(s)));
      }
    };
    if (steps > 0) {
#pragma unroll
      for (int r = 0; r < RING; ++r)
        if (r < steps) issue(r);
      wait_steps<LOADS, RING - 1>(steps - 1);
      bare_barrier();
#pragma unroll
      for (int j = 0; j < (F ? NF : 0); ++j) {
        sb[j] = b_scales(0, j);
        fb[0][j] = read_b(ring, j, 0, sb[j]);
      }
#pragma unroll
      for (int i = 0; i < F; ++i) {
        if (X4) sa[i] = a_scales(0, i);
        fa[i] = read_a(ring, i, 0);
      }
    }
    for (int st = 0; st < steps; ++st) {
      const u32x4* slot = ring + st % RING * STAGE;
      const u32x4* next = ring + (st + 1) % RING * STAGE;
      static_for<NS>([&](auto hc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value, cur = h & 1;
        static_assert(NS % 2 == 0, "fragments alternate");
        constexpr bool last = h == NS - 1;
        if (last) {
          wait_lgkmcnt0();  // this wave's reads of step st are back
          if (st + 1 < steps) {
            // step st + 1 has landed for this wave, and after the barrier for all; all are done with step st's slot
            wait_steps<LOADS, RING - 2>(steps - 2 - st);
            bare_barrier();
            if (st + RING < steps) issue(st + RING);
          }
        }
        // Past the last step these reads bring nothing that is used (any slot, in bounds).
        const u32x4* rs = last ? next : slot;
        constexpr int rh = (h + 1) % NS;
#pragma unroll
        for (int j = 0; j < (F ? NF : 0); ++j) {
          if (last) sn[j] = b_scales(st + 1, j);
          fb[cur ^ 1][j] = read_b(rs, j, rh, last ? sn[j] : sb[j]);
        }
#pragma unroll
        for (int i = 0; i < F; ++i) {
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            if constexpr (X4) {
              const u32x4 x = fb[cur][j], y = fa[i];
              const i32x8 w{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
              const i32x8 v{(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, v, acc[i][j], 4, 4, h, (int)sb[j], h,
                                                                          (int)sa[i]);
            } else {
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[cur][j]),
                                                                  __builtin_bit_cast(bf16x8, fa[i]), acc[i][j], 0, 0, 0);
            }
          }
          fa[i] = read_a(rs, i, rh);
          if (X4 && last) sa[i] = a_scales(st + 1, i);
        }
        __atomic_signal_fence(__ATOMIC_SEQ_CST);  // the reads stay in this slice
      });
#pragma unroll
      for (int j = 0; j < NF; ++j) sb[j] = sn[j];
    }
    OutTile o;
    if constexpr (PAIR) {
      constexpr int UF = OB::U / 16, NH = NF / 2;
      o.set(p, row0, t.mlim, t.c0, t.clim, p.N);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        f32x4 h[NH];
#pragma unroll
        for (int q = 0; q < NH; ++q)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            constexpr int two = 2 * UF;
            h[q][x] = silu_times(acc[i][q / UF * two + q % UF][x], acc[i][q / UF * two + q % UF + UF][x]);
          }
        if constexpr (NH % 2 == 0) {
          if (a.out_scales) {
            store_mxfp4<NH>(a, t, h, wm + i * 16, wn / 2, lane);
            continue;
          }
        }
        store_fragments<NH>(o, p, h, wm + i * 16, wn / 2, lane);
      }
    } else {
      o.set(p, row0, t.mlim, t.c0, t.clim, p.N);
#pragma unroll
      for (int i = 0; i < F; ++i) store_fragments<NF>(o, p, acc[i], wm + i * 16, wn, lane);
    }
  };
  if constexpr (DEAL) {
    const int mine = __builtin_amdgcn_readfirstlane(min(MF, max(0, (t.mlim - wm + 15) / 16)));
    static_for<MF + 1>([&](auto c) __attribute__((always_inline)) {
      if (mine == decltype(c)::value) run(c);
    });
  } else {
    run(std::integral_constant<int, MF>{});
  }
}

template <bool X4, bool PAIR, int WM, int WN, int WGM, int WGN, int DK, int RING, bool ONCE, bool DEAL>
hipError_t launch_mx(const MxGemmArgs& a, const MxProductArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(kForward, a.g, WM * WGM, PAIR ? WN * WGN / 2 : WN * WGN));
  mx_kernel<X4, PAIR, WM, WN, WGM, WGN, DK, RING, ONCE, DEAL><<<(unsigned)grid, 64 * WGM * WGN, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool X4, bool PAIR>
hipError_t launch_mx_product(const MxGemmArgs& a, hipStream_t stream) {
  const GroupedGemmArgs& g = a.g;
  const MxProductArgs p{{g.a, g.b, g.a2, g.b2, g.out, g.offsets, g.rows, g.E, g.N, g.K, g.out_bf16 ? 1 : 0, 0,
                         stream_rows(g, kForward)},
                        a.a_scales, a.b_scales, a.b2_scales, a.out_scales};
  const long long mean = g.rows / g.E;
  if constexpr (X4) {
    if (mean >= 128) return launch_mx<true, PAIR, 128, 64, 2, 4, 256, 2, false, true>(a, p, stream);
    return launch_mx<true, PAIR, 32, 64, 2, 2, 256, 3, true, false>(a, p, stream);
  } else {
    if (mean >= 128) return launch_mx<false, PAIR, 128, 64, 2, 4, 64, 3, false, true>(a, p, stream);
    return launch_mx<false, PAIR, 32, 64, 1, 4, 128, 3, true, false>(a, p, stream);
  }
}

}  // namespace

bool mx_gemm_fits(const MxGemmArgs& a) {
  return xcd_grid(tile_items(kForward, a.g, 16, 32)) <= kMaxWorkgroups / 2;
}

bool mx_ffn_fits(int rows, int E, int d, int d_ff) {
  MxGemmArgs up{}, down{};
  up.g.rows = down.g.rows = rows;
  up.g.E = down.g.E = E;
  up.g.N = down.g.K = d_ff;
  up.g.K = down.g.N = d;
  return mx_gemm_fits(up) && mx_gemm_fits(down);
}

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
  const bool pair = a.g.b2 != nullptr;
  if (a.x4) return (pair ? &launch_mx_product<true, true> : &launch_mx_product<true, false>)(a, stream);
  return (pair ? &launch_mx_product<false, true> : &launch_mx_product<false, false>)(a, stream);
}

}  // namespace moe
