// Matrix products grouped by expert with MXFP4 weights (the format is in mxfp4.h): y[r] = W_e x[r] with rows
// x in bf16 or in MXFP4, and the gate and up products with SwiGLU in the epilogue.
//
// Rows in MXFP4 go with the weights' codes into v_mfma_scale_f32_16x16x128_f8f6f4, which takes 16
// elements x 128 of each operand and a scale byte per lane: lane r + 16 g holds row r and one group of 32 elements,
// with its scale. Weights that meet bf16 rows are converted in registers, exactly, and go into
// v_mfma_f32_16x16x32_bf16. Both sum in fp32.
//
// The order in which a product takes its contraction elements is free as long as both operands agree; each
// kernel takes the one that gives it whole pieces of memory and few reads of LDS.
#include "mxfp4.h"
#include "mxfp4_internal.h"
#include "mxfp4_shapes.h"
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

// Chunk c of 16 bytes of a row of CPR chunks sits at c ^ x(row), so that the lanes that read LDS together fall on distinct banks.
// They are, of a fragment read, 8 rows of lane group 0 and the 8 others of group 1 (or of groups 2 and 3). Where the groups
// read chunks 2^ROT apart, their bits are turned left by ROT from what groups that read neighbouring chunks need. (Without
// that, 17% of the cycles of the product of 4-bit rows were bank conflicts.)
template <int CPR, int ROT>
__device__ __forceinline__ constexpr int swizzle(int row) {
  static_assert(CPR == 8 || CPR == 32, "row width");
  constexpr int bits = CPR == 8 ? 3 : 4, all = (1 << bits) - 1;
  const int x = (CPR == 8 ? row >> 1 : row) & all;
  return (x << ROT | x >> (bits - ROT)) & all;
}

// One operand of a tile: T rows of ROWB bytes per step, loaded by NW waves with buffer loads of 1 KB into LDS. PAIR:
// units of U rows of two matrices in turn (gate, up, gate, ..). Lane groups read chunks 2^ROT apart.
template <int T, int ROWB, int NW, int ROT, bool PAIR>
struct Tile {
  static constexpr int CPR = ROWB / 16, kChunks = T * CPR, kAll = kChunks / 64, kRowsPerLoad = 64 / CPR;
  static constexpr int kLoads = (kAll + NW - 1) / NW, kLeast = kAll / NW;  // of a wave, at most and at least
  static constexpr int U = kRowsPerLoad > 16 ? kRowsPerLoad : 16;
  static_assert(kAll * 64 == kChunks, "whole loads");
  // The permutation repeats after this many of a wave's loads.
  static constexpr int kTurn = CPR < 16 || kRowsPerLoad * NW >= 16 ? 1 : 16 / (kRowsPerLoad * NW);
  static_assert(CPR >= 16 || kRowsPerLoad * NW % 16 == 0, "the permutation repeats from one load to the next");
  static_assert(!PAIR || T % (2 * U) == 0, "whole pairs of units");
  static_assert(!PAIR || NW * kRowsPerLoad % (2 * U) == 0, "a wave's loads are all of one matrix");
  static constexpr int kOutside = 0x40000000;  // past any extent (at most 256 rows of 2^21 bytes)

  // PAIR: in the matrix that this wave loads. (Chosen per load between two members, both went to LDS, 32 bytes a thread, and every load
  // read its descriptor from there and ran in a loop over its lanes' values: 65,536 4-bit rows by 32 x 2048 x 7168 gate and up in
  // 1,042 - 1,054 us, now 960 - 978; bf16 rows 2,743 - 2,768, now 2,670 - 2,693.)
  const char* base;
  int extent, ld, row_at, at_in_row;

  // first, count: the tile's first row in the matrix (PAIR: in each of the two) and how many exist
  __device__ __forceinline__ void set(const void* origin, const void* origin2, size_t first, int count, int row_bytes,
                                      int wave, int lane) {
    ld = row_bytes;
    const void* mine = PAIR && (wave * kRowsPerLoad / U & 1) ? origin2 : origin;
    base = static_cast<const char*>(mine) + first * row_bytes;
    extent = count * row_bytes;
    const int row = lane / CPR, pos = lane % CPR;
    at_in_row = (pos ^ swizzle<CPR, ROT>(wave * kRowsPerLoad + row)) * 16;
    row_at = row * row_bytes;
  }
  // bytes byte0 .. byte0 + ROWB - 1 of each row into `slot`; past the end of a row (`left` bytes from byte0 on) and
  // in rows that do not exist zeros
  // (of PARTS parts of the loads the one given).
  template <int AUX, int PARTS = 1>
  __device__ __forceinline__ void issue(u32x4* slot, int byte0, int left, int wave, int part = 0) const {
    int at[kTurn];
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      const int in_row = at_in_row ^ (kTurn > 1 ? swizzle<CPR, ROT>(i * kRowsPerLoad * NW) * 16 : 0);
      at[i] = in_row < left ? row_at + in_row : kOutside;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (PARTS > 1 && i * PARTS / kLoads != part) continue;
      const int l = wave + i * NW, r0 = l * kRowsPerLoad;
      if (kLeast < kLoads && l >= kAll) continue;
      const int row0 = PAIR ? (r0 / (2 * U)) * U + r0 % U : r0;
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, extent, kBufferWord3);
      buffer_load_lds16<AUX>(r, slot + l * 64, at[i % kTurn] + row0 * ld, byte0);
    }
  }
  // 16 bytes: chunk c of row m of the slot
  __device__ __forceinline__ static u32x4 read(const u32x4* slot, int m, int c) {
    return slot[m * CPR + (c ^ swizzle<CPR, ROT>(m))];
  }
};

// 4 bytes a lane from a buffer into LDS at lds + 4 * lane
__device__ __forceinline__ void buffer_load_lds4(__amdgpu_buffer_rsrc_t rsrc, void* lds, int voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)lds, 4, voffset, 0, 0, 0);
}
// The 8 scale bytes of each of n rows for a block of 256 elements, in scale_loads(n) loads of 256 bytes: `load` is
// the number of this one.
constexpr int scale_loads(int n) { return (n * 8 + 255) / 256; }
__device__ __forceinline__ void issue_scales(const uint8_t* from, int count, char* area, int load, int lane) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)from, (short)0, count * 8, kBufferWord3);
  buffer_load_lds4(r, area + load * 256, load * 256 + lane * 4);
}

// The same for weights in loads of 1 KB: a tile has a multiple of 8 of their rows, so that no lane's 16 bytes cross the last one's
// end. (4-bit rows: 65,536 by 32 x 2048 x 7168 in 540 - 545 us against 551 - 564 when it was taken. Rows could be read like this but for an odd last one; that gained nothing.)
constexpr int wide_scale_loads(int n) { return (n * 8 + 1023) / 1024; }
__device__ __forceinline__ void issue_scales_wide(const uint8_t* from, int count, char* area, int load, int lane) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)from, (short)0, count * 8, kBufferWord3);
  buffer_load_lds16(r, area + load * 1024, load * 1024 + lane * 16, 0);
}

// h = silu(g) u, in place of the gates. Where the sigmoid is no normal fp32 number (g < kFar, see swiglu.h) it is taken as the
// fourth power of q = e^(g/4), a factor at a time: u q q is far from both ends of the format unless the result is 0, and the
// factors' errors ((|g| + 13) 2^-24 in all) are far inside h's rounding.
template <int N>
__device__ __forceinline__ void silu_times(float (&g)[N], const float (&u)[N]) {
  float low = g[0];
#pragma unroll
  for (int i = 1; i < N; ++i) low = fminf(low, g[i]);  // (NaN is passed over: it needs no care)
  float h[N];
#pragma unroll
  for (int i = 0; i < N; ++i) h[i] = g[i] * sigmoid<__bf16>(g[i]) * u[i];
  if (low < kFar) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float q = __builtin_amdgcn_exp2f(g[i] * (0.25f * 1.44269504088896f));
      if (g[i] < kFar) h[i] = u[i] * q * q * g[i] * q * q;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) g[i] = h[i];
}
template <int NH>
__device__ __forceinline__ void silu_times(f32x4 (&g)[NH], const f32x4 (&u)[NH]) {
  float x[4 * NH], y[4 * NH];
#pragma unroll
  for (int i = 0; i < 4 * NH; ++i) {
    x[i] = g[i / 4][i % 4];
    y[i] = u[i / 4][i % 4];
  }
  silu_times(x, y);
#pragma unroll
  for (int i = 0; i < 4 * NH; ++i) g[i / 4][i % 4] = x[i];
}

// 16 rows of h in bf16 from r0 and 32 columns from c0 of the tile, 64 bytes of a row together (store_fragments would write 32).
__device__ __forceinline__ void store_32_columns(const OutTile& o, bool stream, const f32x4 (&v)[2], int r0, int c0, int lane) {
  u32x4 q;  // 8 columns of fragment 0 (even lane groups) or 1 (odd ones)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto s = __builtin_amdgcn_permlane16_swap(pack_bf16(v[0][2 * h], v[0][2 * h + 1]),
                                                    pack_bf16(v[1][2 * h], v[1][2 * h + 1]), false, false);
    q[h] = s[0];
    q[2 + h] = s[1];
  }
  const int g = lane >> 4;
  o.put(q, o.at(r0 + (lane & 15), c0 + (g & 1) * 16 + (g >> 1) * 8, 2), stream);
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

// 16 rows of h from r0 and NH * 16 columns from c0 of the tile, in the output's format.
template <int NH>
__device__ __forceinline__ void store_h(const MxProductArgs& a, const TileAt& t, const OutTile& o, const f32x4 (&h)[NH], int r0,
                                        int c0, int lane) {
  if constexpr (NH % 2 == 0) {
    if (a.out_scales) return store_mxfp4<NH>(a, t, h, r0, c0, lane);
  }
  if constexpr (NH == 2) store_32_columns(o, a.p.stream, h, r0, c0, lane);
  else store_fragments<NH>(o, a.p, h, r0, c0, lane);
}

// A workgroup of WGM x WGN waves computes a tile of C, each wave WM x WN of it. Rows go through two slots of DK
// contraction elements in LDS, codes and their scales through two slots of blocks of 256 elements, so that a load takes whole
// lines of a row: X4 (rows in MXFP4) has steps of a block and both operands loaded
// together; bf16 rows have four steps to a block, and the next block is loaded in four parts. PAIR: the
// tile's columns are those of two matrices, 16 of the one and 16 of the other in turn, so that a wave holds gate and up of
// the same columns of h.
// Many rows per expert. bf16 rows are bound by the matrix instructions and the card's power: 65,536 rows over 32 experts of 2048 x 7168
// in 1.41 - 1.50 ms over several cards, 1.28 - 1.36 PFLOP/s, matrix instructions 64% of the cycles, no LDS conflicts; codes take a
// quarter of the bytes and LDS of bf16 weights. 4-bit rows: 517 - 531 us, 3.6 - 3.7 PFLOP/s, matrix instructions 46%
// of the cycles: a step of 256 elements is over in 2,048 cycles of them, less than its loads take to arrive from the L2, and LDS holds
// no third slot of 256 x 256 tiles. (Three slots of smaller tiles 656 - 724 us, four waves of 128 x 128 633; loads issued between the
// products 977 and more; waves of a SIMD in turn 570, and 1,585 for bf16 rows.) Gate and up: 0.97 - 1.01 ms with 4-bit rows, also with h
// in codes, 2.68 - 2.92 with bf16 ones.
template <bool X4, bool PAIR, int WM, int WN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN) void mx_kernel(MxProductArgs a) {
  constexpr int TM = WM * WGM, TN = WN * WGN, NW = WGM * WGN;
  constexpr int MF = WM / 16, NF = WN / 16;
  constexpr int DK = X4 ? kMxBlock : 64;
  constexpr int NS = 2;                     // slices of a step: one matrix instruction per pair of fragments
  using OA = Tile<TM, 128, NW, 1, false>;
  using OB = Tile<TN, 128, NW, 1, PAIR>;
  constexpr int SPB = kMxBlock / DK;        // steps per block
  constexpr int SLOTS = 2;
  constexpr int LOADS = OA::kLeast + (X4 ? OB::kLeast : 0);
  // loads of scales, and bytes of their areas
  constexpr int LA = X4 ? scale_loads(TM) : 0, LB = wide_scale_loads(PAIR ? TN / 2 : TN), LT = LA + LB * (PAIR ? 2 : 1);
  constexpr int kRowArea = LA * 256, kWeightArea = LB * 1024, kArea = kRowArea + kWeightArea * (PAIR ? 2 : 1);
  static_assert(!PAIR || WN % (2 * OB::U) == 0, "a wave holds whole pairs");
  static_assert(SLOTS * (OA::kChunks * 16 + OB::kChunks * 16 + kArea) <= 160 * 1024, "LDS");
  // (One object: with several, the compiler takes reads of each to depend on the loads into it that are in flight and waits for
  // all of them first. What is read has landed, the kernel's own waits see to that.)
  __shared__ __align__(16) u32x4 ring[SLOTS * (OA::kChunks + OB::kChunks + kArea / 16)];
  u32x4* const code_ring = ring + SLOTS * OA::kChunks;
  char* const scale_ring = reinterpret_cast<char*>(code_ring + SLOTS * OB::kChunks);
  const ProductArgs& p = a.p;
  TileAt t;
  if (!tile_at<kForward, true>(p, TM, PAIR ? TN / 2 : TN, t)) return;
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

  auto issue_block = [&](int b, int part) __attribute__((always_inline)) {
    if (part == 0) {
      char* area = scale_ring + b % SLOTS * kArea;
      const size_t wb = mx_scale_at(t.e, blocks, b, p.N, t.c0);
#pragma unroll
      for (int i = 0; i < (LT + NW - 1) / NW; ++i) {
        const int l = wave + i * NW;
        if (X4 && l < LA) issue_scales(a.a_scales + mx_scale_at(0, 0, b, p.rows, row0), t.mlim, area, l, lane);
        else if (l < LA + LB) issue_scales_wide(a.b_scales + wb, t.clim, area + kRowArea, l - LA, lane);
        else if (PAIR && l < LT) issue_scales_wide(a.b2_scales + wb, t.clim, area + kRowArea + kWeightArea, l - LA - LB, lane);
      }
    }
    ob.template issue<0, SPB>(code_ring + b % SLOTS * OB::kChunks, b * 128, K / 2 - b * 128, wave, part);
  };
  // Rows of step st, and the codes whose turn it is: X4 those of the step; else, once all are done with block q - 1 (the
  // barrier in step 4q - 1, when the rows of step 4q + 1 are issued), one part of block q + 1 with each of steps
  // 4q + 1 .. 4q + 4. Codes go before the rows: whoever waits for step 4q + 4's rows has block q + 1 too.
  auto issue = [&](int st) __attribute__((always_inline)) {
    if constexpr (X4) {
      issue_block(st, 0);
    } else {
      const int at = st - 1;
      if (at >= 0 && at / SPB + 1 < blocks) issue_block(at / SPB + 1, at % SPB);
    }
    oa.template issue<0>(ring + st % SLOTS * OA::kChunks, st * 128, a_bytes - st * 128, wave);
  };
  // Scales of this lane's groups of step st: X4 two, in two bytes; else one. Groups past K hold zeros under whatever their
  // scale bytes are; their scale is taken to be 2^-127, so that zeros they stay.
  const int groups = K / kMxGroup;
  auto scales_of = [&](const char* rows, int m, int st) __attribute__((always_inline)) {
    const int first = st * (DK / kMxGroup) + (X4 ? lg * 2 : lg / 2);  // group of the whole row
    const char* at = rows + (m + lr) * 8 + (first & 7);
    if constexpr (X4) {
      const unsigned s = *reinterpret_cast<const unsigned short*>(at);
      return first + 1 < groups ? s : (first < groups ? s & 0xffu : 0u);
    } else {
      const unsigned s = *reinterpret_cast<const unsigned char*>(at);
      return first < groups ? s : 0u;
    }
  };
  auto a_scales = [&](int st, int i) __attribute__((always_inline)) {
    return scales_of(scale_ring + st / SPB % SLOTS * kArea, wm + i * 16, st);
  };
  auto b_scales = [&](int st, int j) __attribute__((always_inline)) {
    const char* area = scale_ring + st / SPB % SLOTS * kArea + kRowArea;
    const int n = wn + j * 16;
    if constexpr (PAIR) return scales_of(area + (n / 16 & 1) * kWeightArea, n / 32 * 16, st);
    else return scales_of(area, n, st);
  };

  auto run = [&](auto present) __attribute__((always_inline)) {
    constexpr int F = decltype(present)::value;
    f32x4 acc[F ? F : 1][NF];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 fa[F ? F : 1], fb[2][NF];   // fb: codes (X4) or bf16 values
    unsigned sa[F ? F : 1], sb[NF], sn[NF];  // scales; sn: the next step's
    u32x2 codes[NF];                  // of a step's two slices (bf16 rows)
    auto read_a = [&](const u32x4* slot, int i, int h) __attribute__((always_inline)) {
      return OA::read(slot, wm + i * 16 + lr, lg * NS + h);
    };
    // The codes of step st, 16 bytes for slice h (X4) or 8 for both slices.
    auto read_codes = [&](int st, int j, int h) __attribute__((always_inline)) {
      const u32x4* slot = code_ring + st / SPB % SLOTS * OB::kChunks;
      const int n = wn + j * 16 + lr;
      if constexpr (X4) {
        return OB::read(slot, n, lg * NS + h);
      } else {
        const int c = (st % SPB * 2 + (lg >> 1)) ^ swizzle<8, 1>(n);
        return reinterpret_cast<const u32x2*>(slot)[(n * 8 + c) * 2 + (lg & 1)];
      }
    };
    auto convert = [&](int j, int h, unsigned scale) __attribute__((always_inline)) {
      return __builtin_bit_cast(u32x4, mx_bf16x8(codes[j][h], mx_scale_f32(scale)));
    };
    for (int i = 0; i < (X4 ? 0 : SPB); ++i) issue_block(0, i);
#pragma unroll
    for (int r = 0; r < SLOTS; ++r)
      if (r < steps) issue(r);
    wait_steps<LOADS, 1>(steps - 1);
    bare_barrier();
    auto product = [&](int i, int j, u32x4 x, auto hc) __attribute__((always_inline)) {
      constexpr int h = decltype(hc)::value;
      if constexpr (X4) {
        const u32x4 y = fa[i];
        const i32x8 w{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
        const i32x8 v{(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, v, acc[i][j], 4, 4, h, (int)sb[j], h, (int)sa[i]);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, fa[i]),
                                                            acc[i][j], 0, 0, 0);
      }
    };
#pragma unroll
    for (int j = 0; j < (F ? NF : 0); ++j) {
      sb[j] = b_scales(0, j);
      if constexpr (X4) fb[0][j] = read_codes(0, j, 0);
      else {
        codes[j] = read_codes(0, j, 0);
        fb[0][j] = convert(j, 0, sb[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if (X4) sa[i] = a_scales(0, i);
      fa[i] = read_a(ring, i, 0);
    }
    for (int st = 0; st < steps; ++st) {
      const u32x4* slot = ring + st % SLOTS * OA::kChunks;
      const u32x4* next = ring + (st + 1) % SLOTS * OA::kChunks;
      static_for<NS>([&](auto hc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value, cur = h & 1;
        constexpr bool last = h == NS - 1;
        if (last) {
          wait_lgkmcnt0();  // this wave's reads of step st are back
          if (st + 1 < steps) {
            // step st + 1 has landed for this wave, and after the barrier for all; all are done with step st's slot
            wait_vmcnt<0>();
            bare_barrier();
            if (st + SLOTS < steps) issue(st + SLOTS);
          }
        }
        // Past the last step these reads bring nothing that is used (any slot, in bounds).
        const u32x4* rs = last ? next : slot;
        constexpr int rh = (h + 1) % NS;
#pragma unroll
        for (int j = 0; j < (F ? NF : 0); ++j) {
          if (last) sn[j] = b_scales(st + 1, j);
          if constexpr (X4) fb[cur ^ 1][j] = read_codes(st + last, j, rh);
          else if (last) codes[j] = read_codes(st + 1, j, 0);
        }
#pragma unroll
        for (int i = 0; i < F; ++i) {
          if (!X4 && i == F / 2) {  // the codes have had time to arrive
#pragma unroll
            for (int j = 0; j < NF; ++j) fb[cur ^ 1][j] = convert(j, rh, last ? sn[j] : sb[j]);
          }
#pragma unroll
          for (int j = 0; j < NF; ++j) product(i, j, fb[cur][j], hc);
          fa[i] = read_a(rs, i, rh);
          if (X4 && last) sa[i] = a_scales(st + 1, i);
        }
        // order of the slice for bf16 rows: the reads of codes and scales, then each row fragment's products and its next read
        // (65,536 rows over 32 experts of 2048 x 7168: 1,452 us against 1,479; with 4-bit rows 547 against 537)
        if constexpr (!X4 && F > 0) {
          if (last) __builtin_amdgcn_sched_group_barrier(0x100, 2 * NF, 0);
#pragma unroll
          for (int i = 0; i < F; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, NF, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
        }
        __atomic_signal_fence(__ATOMIC_SEQ_CST);  // the reads stay in this slice
      });
#pragma unroll
      for (int j = 0; j < NF; ++j) sb[j] = sn[j];
    }
    OutTile o;
    o.set(p, row0, t.mlim, t.c0, t.clim, p.N);
    if constexpr (PAIR) {
      constexpr int NH = NF / 2;
#pragma unroll
      for (int i = 0; i < F; ++i) {
        f32x4 h[NH], u[NH];
#pragma unroll
        for (int q = 0; q < NH; ++q) {
          h[q] = acc[i][2 * q];
          u[q] = acc[i][2 * q + 1];
        }
        silu_times(h, u);
        store_h<NH>(a, t, o, h, wm + i * 16, wn / 2, lane);
      }
    } else {
#pragma unroll
      for (int i = 0; i < F; ++i) store_fragments<NF>(o, p, acc[i], wm + i * 16, wn, lane);
    }
  };
  const int mine = __builtin_amdgcn_readfirstlane(min(MF, max(0, (t.mlim - wm + 15) / 16)));
  static_for<MF + 1>([&](auto c) __attribute__((always_inline)) {
    if (mine == decltype(c)::value) run(c);
  });
}

// Few rows per expert: the weights' codes go straight to registers, DEPTH - 1 blocks of 256 contraction elements ahead, the
// rows, which all waves share, through a ring of DEPTH slots in LDS. A wave takes MF * 16 rows and NF * 16 columns (PAIR: NF / 2
// fragments of gate and as many of up), the NW waves of a workgroup neighbouring columns. Of each half of a block (128
// elements) a lane holds one group of 32 of each of its weight rows, so that a load takes 64 bytes of 16 rows.
// The weights' stream bounds it: 1,024 rows over 128 experts of 1536 x 4096 (428 MB of weights) in 88 us, 5.0 TB/s with rows
// and results; of 4096 x 1536 with 4-bit rows 88; gate and up of the former 172. (Tiles of mx_kernel 117; a lane with 512 elements
// of a row 157; loads that pass the L2 by 101 - 103: both halves of a line are loaded by themselves.)
// In some shapes the scales' descriptors end up in vector registers and each of their loads in a loop over the lanes' values. With the
// extents in scalar registers those loops go, but the compiler then sinks a block's loads behind the products: 32 rows for each
// of 8 experts of 2048 x 4096 took 19.0 us against 16.1, gate and up of 256 tokens over 128 experts 178 against 168.
template <bool X4, bool PAIR, int MF, int NF, int NW, int DEPTH>
__global__ __launch_bounds__(64 * NW) void mx_rows_kernel(MxProductArgs a) {
  constexpr int TM = 16 * MF, WN = 16 * NF, TN = WN * NW, TH = PAIR ? TN / 2 : TN, WH = PAIR ? WN / 2 : WN;
  constexpr int NH = PAIR ? NF / 2 : NF, kRowBytes = X4 ? 128 : 512;
  using OA = Tile<TM, kRowBytes, NW, X4 ? 0 : 2, false>;
  constexpr int LA = X4 ? scale_loads(TM) : 0;
  constexpr int kOutside = 0x40000000;
  // loads of a block by every wave: rows, codes and scales (those that only some waves make just lengthen their waits)
  constexpr int LOADS = OA::kLeast + 3 * NF;
  __shared__ __align__(16) u32x4 ring[DEPTH * (OA::kChunks + LA * 16)];  // (one object: see mx_kernel)
  char* const scale_ring = reinterpret_cast<char*>(ring + DEPTH * OA::kChunks);
  const ProductArgs& p = a.p;
  TileAt t;
  if (!tile_at<kForward, false>(p, TM, TH, t)) return;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = p.K, blocks = mx_blocks(K), ld = K / 2, a_ld = X4 ? ld : K * 2, groups = K / kMxGroup;
  const size_t row0 = (size_t)t.ra + t.m0, we = (size_t)t.e * p.N * ld + (size_t)t.c0 * ld;
  OA oa;
  oa.set(p.a, p.a, row0, t.mlim, a_ld, wave, lane);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(static_cast<const char*>(p.b) + we), (short)0, t.clim * ld, kBufferWord3);
  const __amdgpu_buffer_rsrc_t rb2 = __builtin_amdgcn_make_buffer_rsrc(
      PAIR ? (void*)(static_cast<const char*>(p.b2) + we) : nullptr, (short)0, PAIR ? t.clim * ld : 0, kBufferWord3);

  struct Block {
    u32x4 b[NF][2];
    u32x2 s[NF];
  };
  // block b (past the last: zeros) into slot i of the ring and into q
  auto load = [&](Block& q, int b, int i) __attribute__((always_inline)) {
    const bool in = b < blocks;
    const int at = b * 128 + lg * 16;  // of the lane's codes in a row
    oa.template issue<0>(ring + i * OA::kChunks, b * kRowBytes, a_ld - b * kRowBytes, wave);
    const size_t ws = mx_scale_at(t.e, blocks, in ? b : 0, p.N, t.c0);
    const __amdgpu_buffer_rsrc_t s =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.b_scales + ws), (short)0, in ? t.clim * 8 : 0, kBufferWord3);
    const __amdgpu_buffer_rsrc_t s2 = __builtin_amdgcn_make_buffer_rsrc(
        PAIR ? (void*)(a.b2_scales + ws) : nullptr, (short)0, PAIR && in ? t.clim * 8 : 0, kBufferWord3);
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const bool up = PAIR && j >= NH;
      const int n = wave * WH + (up ? j - NH : j) * 16 + lr;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q.b[j][h] = __builtin_amdgcn_raw_buffer_load_b128(up ? rb2 : rb, at + h * 64 < ld ? n * ld + at + h * 64 : kOutside, 0, 0);
      q.s[j] = __builtin_amdgcn_raw_buffer_load_b64(up ? s2 : s, n * 8, 0, 0);
    }
    if (X4 && wave < LA)
      issue_scales(a.a_scales + mx_scale_at(0, 0, in ? b : 0, p.rows, row0), in ? t.mlim : 0, scale_ring + i * LA * 256, wave,
                   lane);
  };
  auto run = [&](auto present) __attribute__((always_inline)) {
    constexpr int F = decltype(present)::value;
    f32x4 acc[F][NF];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Block& q, int b, int slot) __attribute__((always_inline)) {
      const u32x4* rows = ring + slot * OA::kChunks;
      static_for<2>([&](auto hc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value;
        // A group past K holds zeros; its scale is taken to be 2^-127 whatever the byte, so that zeros they stay.
        const unsigned mask = b * 8 + h * 4 + lg < groups ? 0xffu : 0u;
        unsigned s[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j) s[j] = q.s[j][h] >> lg * 8 & mask;
        if constexpr (X4) {
#pragma unroll
          for (int i = 0; i < F; ++i) {
            const u32x4 y = OA::read(rows, i * 16 + lr, h * 4 + lg);
            const unsigned sa =
                *reinterpret_cast<const unsigned char*>(scale_ring + slot * LA * 256 + (i * 16 + lr) * 8 + h * 4 + lg) & mask;
            const i32x8 v{(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NF; ++j) {
              const u32x4 x = q.b[j][h];
              const i32x8 w{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, v, acc[i][j], 4, 4, 0, (int)s[j], 0, (int)sa);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            bf16x8 w[NF];
#pragma unroll
            for (int j = 0; j < NF; ++j) w[j] = mx_bf16x8(q.b[j][h][k], mx_scale_f32(s[j]));
#pragma unroll
            for (int i = 0; i < F; ++i) {
              const bf16x8 v = __builtin_bit_cast(bf16x8, OA::read(rows, i * 16 + lr, h * 16 + lg * 4 + k));
#pragma unroll
              for (int j = 0; j < NF; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], v, acc[i][j], 0, 0, 0);
            }
          }
        }
      });
    };
    Block q[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) {
      load(q[i], i, i);
      if constexpr (DEPTH > 2) __atomic_signal_fence(__ATOMIC_SEQ_CST);  // block by block, as the waits count them
    }
    for (int b0 = 0; b0 < blocks; b0 += DEPTH) {
      static_for<DEPTH>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        const int b = b0 + i;
        if (b < blocks) {
          wait_vmcnt<(DEPTH - 2) * LOADS>();  // block b has landed for this wave, and after the barrier for all;
          wait_lgkmcnt0();
          bare_barrier();                     // all are done with block b - 1
          load(q[(i + DEPTH - 1) % DEPTH], b + DEPTH - 1, (i + DEPTH - 1) % DEPTH);
          multiply(q[i], b, i);
          __atomic_signal_fence(__ATOMIC_SEQ_CST);
        }
      });
    }
    OutTile o;
    o.set(p, row0, t.mlim, t.c0, t.clim, p.N);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if constexpr (PAIR) {
        f32x4 h[NH], u[NH];
#pragma unroll
        for (int j = 0; j < NH; ++j) {
          h[j] = acc[i][j];
          u[j] = acc[i][j + NH];
        }
        silu_times(h, u);
        store_h<NH>(a, t, o, h, i * 16, wave * WH, lane);
      } else {
        store_fragments<NF>(o, p, acc[i], i * 16, wave * WN, lane);
      }
    }
  };
  const int mine = __builtin_amdgcn_readfirstlane((t.mlim + 15) / 16);
  static_for<MF>([&](auto c) __attribute__((always_inline)) {
    if (mine == decltype(c)::value + 1) run(std::integral_constant<int, decltype(c)::value + 1>{});
  });
}

// Few rows and few tiles: no LDS on the operands' way. A workgroup takes 16 rows and NF * 16 columns (PAIR: NF / 2 fragments of
// gate and as many of up), and its NW waves share the contraction, wave w blocks w, w + NW, .. of 256 elements, in
// the order of mx_rows_kernel. A wave issues its next block's loads before a block's products (after them: a row for each of
// 4 experts of 2048 x 7168 in 9.8 us against 8.7). At the end the waves' sums are joined in order in LDS.
// Latency bounds it: one row of 8 of 128 experts of 1536 x 4096, gate and up, in 15.6 us with bf16 rows (54 MB, 11.3 at the rate of a copy; an
// empty launch takes 3; 45.7 in tiles of mx_kernel), 13.7 with 4-bit ones, a product of those 9.1.
template <bool X4, bool PAIR, int NF, int NW>
__global__ __launch_bounds__(64 * NW) void mx_stream_kernel(MxProductArgs a) {
  constexpr int TN = 16 * NF, TH = PAIR ? TN / 2 : TN, kThreads = 64 * NW, NH = PAIR ? NF / 2 : NF;
  constexpr int kPitch = TN + 4;
  constexpr int kOutside = 0x40000000;
  __shared__ __align__(16) float sums[NW][16][kPitch];
  const ProductArgs& p = a.p;
  TileAt t;
  if (!tile_at<kForward, false>(p, 16, TH, t)) return;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = p.K, blocks = mx_blocks(K), ld = K / 2, a_ld = X4 ? ld : K * 2, groups = K / kMxGroup;
  const size_t row0 = (size_t)t.ra + t.m0, we = (size_t)t.e * p.N * ld + (size_t)t.c0 * ld;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(static_cast<const char*>(p.a) + row0 * a_ld), (short)0, t.mlim * a_ld, kBufferWord3);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(static_cast<const char*>(p.b) + we), (short)0, t.clim * ld, kBufferWord3);
  const __amdgpu_buffer_rsrc_t rb2 = __builtin_amdgcn_make_buffer_rsrc(
      PAIR ? (void*)(static_cast<const char*>(p.b2) + we) : nullptr, (short)0, PAIR ? t.clim * ld : 0, kBufferWord3);

  struct Block {
    u32x4 a[X4 ? 2 : 8], b[NF][2];
    u32x2 sa, sb[NF];
  };
  auto load = [&](Block& q, int b) __attribute__((always_inline)) {
    const bool in = b < blocks;
    const int at = b * 128 + lg * 16;  // of the lane's codes in a row
    const size_t ws = mx_scale_at(t.e, blocks, in ? b : 0, p.N, t.c0);
    const __amdgpu_buffer_rsrc_t s =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.b_scales + ws), (short)0, in ? t.clim * 8 : 0, kBufferWord3);
    const __amdgpu_buffer_rsrc_t s2 = __builtin_amdgcn_make_buffer_rsrc(
        PAIR ? (void*)(a.b2_scales + ws) : nullptr, (short)0, PAIR && in ? t.clim * 8 : 0, kBufferWord3);
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const bool up = PAIR && j >= NH;
      const int n = (up ? j - NH : j) * 16 + lr;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q.b[j][h] = __builtin_amdgcn_raw_buffer_load_b128(up ? rb2 : rb, at + h * 64 < ld ? n * ld + at + h * 64 : kOutside, 0, 0);
      q.sb[j] = __builtin_amdgcn_raw_buffer_load_b64(up ? s2 : s, n * 8, 0, 0);
    }
    if constexpr (X4) {
      const __amdgpu_buffer_rsrc_t sa = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(a.a_scales + mx_scale_at(0, 0, in ? b : 0, p.rows, row0)), (short)0, in ? t.mlim * 8 : 0, kBufferWord3);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q.a[h] = __builtin_amdgcn_raw_buffer_load_b128(ra, at + h * 64 < ld ? lr * ld + at + h * 64 : kOutside, 0, 0);
      q.sa = __builtin_amdgcn_raw_buffer_load_b64(sa, lr * 8, 0, 0);
    } else {
#pragma unroll
      for (int h = 0; h < 8; ++h)
        q.a[h] = __builtin_amdgcn_raw_buffer_load_b128(
            ra, at + h / 4 * 64 < ld ? lr * a_ld + (at + h / 4 * 64) * 4 + h % 4 * 16 : kOutside, 0, 0);
    }
  };
  f32x4 acc[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // A group past K holds zeros; its scale is taken to be 2^-127 whatever the byte, so that zeros they stay.
  auto multiply = [&](const Block& q, int b) __attribute__((always_inline)) {
    static_for<2>([&](auto hc) __attribute__((always_inline)) {
      constexpr int h = decltype(hc)::value;
      const unsigned mask = b * 8 + h * 4 + lg < groups ? 0xffu : 0u;
      unsigned s[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) s[j] = q.sb[j][h] >> lg * 8 & mask;
      if constexpr (X4) {
        const u32x4 y = q.a[h];
        const i32x8 v{(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
        const unsigned sa = q.sa[h] >> lg * 8 & mask;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const u32x4 x = q.b[j][h];
          const i32x8 w{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
          acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, v, acc[j], 4, 4, 0, (int)s[j], 0, (int)sa);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < NF; ++j)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_bf16x8(q.b[j][h][k], mx_scale_f32(s[j])),
                                                             __builtin_bit_cast(bf16x8, q.a[h * 4 + k]), acc[j], 0, 0, 0);
      }
    });
  };
  Block q;
  load(q, wave);
  for (int b = wave; b < blocks; b += NW) {
    const Block now = q;
    load(q, b + NW);
    multiply(now, b);
  }
#pragma unroll
  for (int j = 0; j < NF; ++j) *reinterpret_cast<f32x4*>(&sums[wave][lr][j * 16 + lg * 4]) = acc[j];
  __syncthreads();
  auto sum = [&](int r, int c) __attribute__((always_inline)) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += sums[w][r][c];
    return v;
  };
  // a thread takes columns c of rows r, r + kThreads / TH, ..
  const int c = threadIdx.x % TH;
#pragma unroll
  for (int r = threadIdx.x / TH; r < 16; r += kThreads / TH) {
    float v = sum(r, c);
    if constexpr (PAIR) {
      float g[1] = {v};
      const float u[1] = {sum(r, c + TH)};
      silu_times(g, u);
      v = g[0];
    }
    const size_t row = row0 + r;
    const int col = t.c0 + c;
    const bool in = r < t.mlim && c < t.clim;
    if constexpr (PAIR && TH % 32 == 0) {
      if (a.out_scales) {  // 32 threads in a row hold a group
        unsigned top = __float_as_uint(v) & 0x7fffffffu;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) top = max(top, (unsigned)__shfl_xor((int)top, d));
        const int scale = mx_scale(top);
        const float q0 = v * mx_inverse(scale), q1 = __shfl_xor(q0, 1);
        const unsigned code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, q0, q1, 1.0f, 0);
        if (in && !(c & 1))
          static_cast<uint8_t*>(p.out)[(row * p.N + col) / 2] = scale == kMxNan ? 0 : (uint8_t)code;
        if (in && !(c & 31))
          a.out_scales[mx_scale_at(0, 0, col / kMxBlock, p.rows, row) + (col / kMxGroup & 7)] = (uint8_t)scale;
        continue;
      }
    }
    if (!in) continue;
    if (p.out_bf16) static_cast<__bf16*>(p.out)[row * p.N + col] = (__bf16)v;
    else static_cast<float*>(p.out)[row * p.N + col] = v;
  }
}

template <bool X4, bool PAIR, int MF, int NF, int NW, int DEPTH>
hipError_t launch_rows(const MxGemmArgs& a, const MxProductArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(kForward, a.g, 16 * MF, (PAIR ? 8 : 16) * NF * NW));
  mx_rows_kernel<X4, PAIR, MF, NF, NW, DEPTH><<<(unsigned)grid, 64 * NW, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool X4, bool PAIR, int NF, int NW>
hipError_t launch_stream(const MxGemmArgs& a, const MxProductArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(kForward, a.g, 16, PAIR ? 8 * NF : 16 * NF));
  mx_stream_kernel<X4, PAIR, NF, NW><<<(unsigned)grid, 64 * NW, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool X4, bool PAIR, int WM, int WN, int WGM, int WGN>
hipError_t launch_mx(const MxGemmArgs& a, const MxProductArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(kForward, a.g, WM * WGM, PAIR ? WN * WGN / 2 : WN * WGN));
  mx_kernel<X4, PAIR, WM, WN, WGM, WGN><<<(unsigned)grid, 64 * WGM * WGN, 0, stream>>>(p);
  return hipGetLastError();
}

// The shapes of mxfp4_shapes.h, in their order.
template <bool X4, bool PAIR>
hipError_t launch_shape(int i, const MxGemmArgs& a, const MxProductArgs& p, hipStream_t s);
template <>
hipError_t launch_shape<false, false>(int i, const MxGemmArgs& a, const MxProductArgs& p, hipStream_t s) {
  switch (i) {
    case 0: return launch_stream<false, false, 2, 4>(a, p, s);
    case 1: return launch_stream<false, false, 4, 4>(a, p, s);
    case 2: return launch_rows<false, false, 1, 1, 4, 4>(a, p, s);
    case 3: return launch_rows<false, false, 1, 2, 8, 3>(a, p, s);
    case 4: return launch_rows<false, false, 2, 1, 4, 4>(a, p, s);
    case 5: return launch_rows<false, false, 2, 1, 8, 3>(a, p, s);
    case 6: return launch_rows<false, false, 2, 4, 4, 3>(a, p, s);
    case 7: return launch_rows<false, false, 4, 2, 8, 2>(a, p, s);
    default: return launch_mx<false, false, 128, 64, 2, 4>(a, p, s);
  }
}
template <>
hipError_t launch_shape<false, true>(int i, const MxGemmArgs& a, const MxProductArgs& p, hipStream_t s) {
  switch (i) {
    case 0: return launch_stream<false, true, 2, 4>(a, p, s);
    case 1: return launch_stream<false, true, 4, 4>(a, p, s);
    case 2: return launch_rows<false, true, 1, 2, 4, 3>(a, p, s);
    case 3: return launch_rows<false, true, 1, 4, 4, 3>(a, p, s);
    case 4: return launch_rows<false, true, 2, 2, 4, 3>(a, p, s);
    case 5: return launch_rows<false, true, 2, 4, 4, 3>(a, p, s);
    case 6: return launch_rows<false, true, 4, 2, 8, 2>(a, p, s);
    default: return launch_mx<false, true, 128, 64, 2, 4>(a, p, s);
  }
}
template <>
hipError_t launch_shape<true, false>(int i, const MxGemmArgs& a, const MxProductArgs& p, hipStream_t s) {
  switch (i) {
    case 0: return launch_stream<true, false, 2, 4>(a, p, s);
    case 1: return launch_stream<true, false, 4, 4>(a, p, s);
    case 2: return launch_rows<true, false, 2, 1, 4, 4>(a, p, s);
    case 3: return launch_rows<true, false, 2, 2, 4, 3>(a, p, s);
    case 4: return launch_mx<true, false, 64, 64, 2, 2>(a, p, s);
    default: return launch_mx<true, false, 128, 64, 2, 4>(a, p, s);
  }
}
template <>
hipError_t launch_shape<true, true>(int i, const MxGemmArgs& a, const MxProductArgs& p, hipStream_t s) {
  switch (i) {
    case 0: return launch_stream<true, true, 2, 4>(a, p, s);
    case 1: return launch_stream<true, true, 4, 4>(a, p, s);
    case 2: return launch_rows<true, true, 2, 2, 2, 4>(a, p, s);
    case 3: return launch_rows<true, true, 2, 2, 4, 3>(a, p, s);
    case 4: return launch_rows<true, true, 2, 4, 4, 3>(a, p, s);
    case 5: return launch_mx<true, true, 64, 64, 2, 2>(a, p, s);
    default: return launch_mx<true, true, 128, 64, 2, 4>(a, p, s);
  }
}

template <bool X4, bool PAIR>
hipError_t launch_mx_product(const MxGemmArgs& a, hipStream_t stream) {
  const GroupedGemmArgs& g = a.g;
  const MxProductArgs p{{g.a, g.b, g.a2, g.b2, g.out, g.offsets, g.rows, g.E, g.N, g.K, g.out_bf16 ? 1 : 0, 0,
                         stream_rows(g, kForward)},
                        a.a_scales, a.b_scales, a.b2_scales, a.out_scales};
  DeviceInfo dev;
  const hipError_t e = device_info(&dev);
  if (e != hipSuccess) return e;
  return launch_shape<X4, PAIR>(pick_gemm<X4, PAIR>(a, dev.num_cus), a, p, stream);
}

}  // namespace

// (the largest tiles: the choice passes over those that do not fit)
bool mx_gemm_fits(const MxGemmArgs& a) {
  return shape_fits(kForward, a.g, a.g.b2 ? TileCost{256, 128, 1, 0, 0} : TileCost{256, 256, 1, 0, 0});
}

bool mx_ffn_fits(int rows, int E, int d, int d_ff) {
  MxGemmArgs up{}, down{};
  up.g.rows = down.g.rows = rows;
  up.g.E = down.g.E = E;
  up.g.N = down.g.K = d_ff;
  up.g.K = down.g.N = d;
  up.g.b2 = &up;  // (a pair)
  return mx_gemm_fits(up) && mx_gemm_fits(down);
}

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
  const bool pair = a.g.b2 != nullptr;
  if (a.x4) return (pair ? &launch_mx_product<true, true> : &launch_mx_product<true, false>)(a, stream);
  return (pair ? &launch_mx_product<false, true> : &launch_mx_product<false, false>)(a, stream);
}

}  // namespace moe
