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
#include <cmath>

#include "grouped.h"
#include "lds_tiles.h"

namespace moe {

namespace {

// ---------------------------------------------------------------------------------------
// fp32: tiles staged through registers
// ---------------------------------------------------------------------------------------
// A workgroup of 4 waves computes a tile of C, each wave FM x FN fragments of 16 x 16; the contraction
// goes in steps of 32. Both operands lie in LDS in their memory order: along operands [m][32 + 4],
// across operands [32][m + 4]; the padding of 4 floats puts the 16 rows (or 4 row groups) of a
// fragment read on distinct banks. v_mfma_f32_16x16x4_f32 takes one contraction element per
// lane (row or column lane % 16, element lane / 16); lane group g takes elements 4g .. 4g + 3
// of a 16-long slice in turn, the same for both operands, so an along fragment is one 16-byte
// read. The operands go in as (B, A), which gives each lane 4 consecutive columns of one row of C.
// Bound by the matrix instructions: 16,384 rows over 8 experts of 1024 x 2048 take 548 - 558 us
// forward (123 - 125 TFLOP/s; a large fp32 library product reaches 132), 1.09 - 1.11 ms for two input
// gradients, 554 us for the weight gradient. Tiles of 128 measured slower at every size, by 9 to 19%. With few tiles it
// is the chain of a step that bounds (LDS, barriers, dependent products); two to four steps' loads
// ahead gained nothing there.
constexpr int kStep = 32;
constexpr int kPad = 4;

struct ProductArgs {
  const void *a, *b, *a2, *b2;  // a2, b2: second pair of operands (dgrad), or null
  void* out;
  const int32_t* offsets;
  int rows, E, N, K;
  int out_bf16, accumulate;
  int stream;  // C's rows are stored non-temporally
};

// The value of the lane 8 further within the 16.
__device__ __forceinline__ u32x4 rotate8(u32x4 v) {
  u32x4 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) r[q] = (unsigned)__builtin_amdgcn_mov_dpp((int)v[q], 0x128, 0xf, 0xf, true);
  return r;
}
// 16 rows of which a lane holds 16 bytes of row lane % 16 in each of two 64-byte parts, a and b, to
// 8 whole 128-byte pieces twice: put(row, part, v) gets 16 bytes of that row's part 0 or 1.
template <typename F>
__device__ __forceinline__ void store_row_halves(u32x4 a, u32x4 b, int lane, F&& put) {
  const bool low = (lane & 8) == 0;
  const u32x4 moved = rotate8(low ? b : a);
  put(lane & 7, low ? 0 : 1, low ? a : moved);
  put((lane & 7) + 8, low ? 0 : 1, low ? moved : b);
}
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  const bf16x2 v{(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(unsigned, v);
}

// The part of a tile of C that a wave stores. Stores go through a buffer descriptor that ends
// with the tile's last row, and lanes past the last column aim behind it, so what lies outside
// is dropped without a branch.
struct OutTile {
  __amdgpu_buffer_rsrc_t to;
  int ld, clim;  // bytes of a row of C; columns that exist
  static constexpr int kOutside = (int)0x80000000u;

  // rows from row0 (mlim of them exist) and columns from c0 of out [.., cols]
  __device__ __forceinline__ void set(const ProductArgs& p, size_t row0, int mlim, int c0, int clim_, int cols) {
    const int size = p.out_bf16 ? 2 : 4;
    ld = cols * size;
    clim = clim_;
    to = __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(p.out) + (row0 * cols + c0) * size, (short)0,
                                           mlim * ld - c0 * size, kBufferWord3);
  }
  __device__ __forceinline__ int at(int r, int c, int size) const { return c < clim ? r * ld + c * size : kOutside; }
  __device__ __forceinline__ void put(u32x4 x, int at, bool stream) const {
    if (stream) __builtin_amdgcn_raw_buffer_store_b128(x, to, at, 0, kNonTemporal);
    else __builtin_amdgcn_raw_buffer_store_b128(x, to, at, 0, 0);
  }
};

// 16 rows of C from r0 and NF * 16 columns from c0 of the tile. `v` is as the products leave it: 4
// consecutive columns (from 4 (lane / 16)) of row lane % 16 in each 16-column fragment. Stored
// like that, an instruction would write 64 bytes (fp32) or 32 (bf16) of each of 16 rows; lanes
// first exchange parts so that it writes 128 bytes of each of 8 (2% of the large products' time),
// most often non-temporally (stream_rows), which leaves the L2 to the operands (fp32 weight gradients of 64
// experts of 2048 x 4096, 128 rows each: 515 against 422 us). Tiles whose waves have too few columns for
// the exchange (one fragment, or up to two with bf16 results: tiles for few rows) and results that are
// added to what is there store fragment by fragment, plainly. For the latter HBM bounds that: the fp32 weight
// gradient of 32 experts of 2048 x 7168 reads dw once more (1.9 GB by counter) and takes, for 65,536 rows, 2.17 ms
// against 1.83, for 1,024 rows 0.88 (3.85 GB, 4.4 TB/s) against 0.35.
template <int NF>
__device__ __forceinline__ void store_fragments(const OutTile& o, const ProductArgs& p, const f32x4 (&v)[NF], int r0,
                                                int c0, int lane) {
  if constexpr (NF % 2 == 0) {
    if (!p.accumulate && !p.out_bf16) {
#pragma unroll
      for (int j = 0; j < NF; j += 2)
        store_row_halves(__builtin_bit_cast(u32x4, v[j]), __builtin_bit_cast(u32x4, v[j + 1]), lane,
                         [&](int r, int part, u32x4 x) __attribute__((always_inline)) {
                           o.put(x, o.at(r0 + r, c0 + (j + part) * 16 + (lane >> 4) * 4, 4), p.stream);
                         });
      return;
    }
  }
  if constexpr (NF % 4 == 0) {
    if (!p.accumulate) {
      u32x4 q[NF / 2];  // 8 columns of fragment j (even lane groups) or j + 1 (odd ones)
#pragma unroll
      for (int j = 0; j < NF; j += 2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto s = __builtin_amdgcn_permlane16_swap(pack_bf16(v[j][2 * h], v[j][2 * h + 1]),
                                                          pack_bf16(v[j + 1][2 * h], v[j + 1][2 * h + 1]), false, false);
          q[j / 2][h] = s[0];
          q[j / 2][2 + h] = s[1];
        }
#pragma unroll
      for (int j = 0; j < NF / 2; j += 2)
        store_row_halves(q[j], q[j + 1], lane, [&](int r, int part, u32x4 x) __attribute__((always_inline)) {
          const int g = lane >> 4;
          o.put(x, o.at(r0 + r, c0 + (j + part) * 32 + (g & 1) * 16 + (g >> 1) * 8, 2), p.stream);
        });
      return;
    }
  }
  const int r = r0 + (lane & 15);
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const int c = c0 + j * 16 + (lane >> 4) * 4;
    f32x4 x = v[j];
    if (p.out_bf16) {
      const int at = o.at(r, c, 2);
      if (p.accumulate) {
        const u32x2 old = __builtin_amdgcn_raw_buffer_load_b64(o.to, at, 0, 0);
        x[0] += __uint_as_float(old[0] << 16);
        x[1] += __uint_as_float(old[0] & 0xffff0000u);
        x[2] += __uint_as_float(old[1] << 16);
        x[3] += __uint_as_float(old[1] & 0xffff0000u);
      }
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}, o.to, at, 0, 0);
    } else {
      const int at = o.at(r, c, 4);
      if (p.accumulate) x += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(o.to, at, 0, 0));
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), o.to, at, 0, 0);
    }
  }
}
// Where a tile lies: expert, its rows [ra, rb), C's rows from m0 (of mlim in the tile) and
// columns from c0 (of clim), and the contraction's length.
struct TileAt {
  int e, ra, rb, m0, mlim, c0, clim, kdim;
};
// DEAL: C's rows are dealt to their row tiles in 16-row fragments as evenly as the number of
// tiles allows (300 rows: tiles of 160 and 140, not 256 and 44), so that row tiles side by side,
// which read the same B, take about the same time.
template <GroupedProduct P, bool DEAL>
__device__ __forceinline__ bool tile_at(const ProductArgs& p, int TM, int TN, TileAt& t) {
  const int cols = P == kForward ? p.N : p.K;
  const int CT = (cols + TN - 1) / TN;
  int mt, nt;
  if constexpr (P == kWgrad) {
    const int per = (p.N + TM - 1) / TM * CT;
    const int item = xcd_item(blockIdx.x, (unsigned)p.E * (unsigned)per);
    if (item < 0) return false;
    // Experts in their order: starting with those of the most rows cost 3 to 12%, whichever way the
    // rows were dealt (64 experts, Zipf 1.2: 444 against 396 us). Side by side, tiles of different
    // lengths do not all store at the same time.
    t.e = item / per;
    group_rows(p.offsets, t.e, p.rows, t.ra, t.rb);
    tile_pair(item % per, (p.N + TM - 1) / TM, CT, mt, nt);
    if (t.ra == t.rb && p.accumulate) return false;
  } else {
    if (!find_row_tile(p.offsets, p.E, p.rows, TM, CT, t.e, t.ra, t.rb, mt, nt)) return false;
  }
  const int n = P == kWgrad ? p.N : t.rb - t.ra;  // C's rows
  t.m0 = mt * TM;
  t.mlim = min(TM, n - t.m0);
  if constexpr (DEAL) {
    const int tiles = (n + TM - 1) / TM, frags = (n + 15) / 16;
    const int q = frags / tiles, more = frags - q * tiles;  // the first `more` tiles take q + 1
    t.m0 = 16 * (mt * q + min(mt, more));
    t.mlim = min(16 * (q + (mt < more ? 1 : 0)), n - t.m0);
  }
  t.c0 = nt * TN;
  t.clim = min(TN, cols - t.c0);
  t.kdim = P == kForward ? p.K : (P == kDgrad ? p.N : t.rb - t.ra);
  // the same in every lane: kept in scalar registers, as buffer descriptors need it
  for (int* v : {&t.e, &t.ra, &t.rb, &t.m0, &t.mlim, &t.c0, &t.clim, &t.kdim}) *v = __builtin_amdgcn_readfirstlane(*v);
  return true;
}

// One operand: TM rows (along) or columns (across) of C's side, KD of the contraction per step, loaded
// by NT threads in 16-byte chunks. Loads go through a buffer descriptor that ends with the last row that
// exists, so that what lies outside reads as zero and a step needs hardly any address arithmetic. (An
// across operand's columns past the matrix read what is there: they meet only columns or rows of C that
// do not exist either.)
template <bool ACROSS, int TM, int KD, int NT>
struct Stage {
  static constexpr int kAll = TM * KD / 4;              // chunks
  static constexpr int NCH = (kAll + NT - 1) / NT;      // per thread
  static constexpr int kRowChunks = (ACROSS ? TM : KD) / 4;
  static constexpr int kRow = (ACROSS ? TM : KD) + kPad;  // floats of an LDS row
  static constexpr int kOutside = 0x40000000;           // past any extent (at most 128 * 2^22 bytes)
  static_assert(NT % kRowChunks == 0, "a thread's chunks lie in one column");
  u32x4 c[NCH];
  const char* base;
  int ld, extent, lane_at, inner;

  // base_: the operand's first element of the tile; count: its rows that exist (along) or the columns
  // before it in a row (across); ld_elems: row stride
  __device__ __forceinline__ void set(const float* base_, int count, int ld_elems) {
    base = reinterpret_cast<const char*>(base_);
    ld = ld_elems * 4;
    inner = (int)threadIdx.x % kRowChunks * 4;
    lane_at = (int)threadIdx.x / kRowChunks * ld + inner * 4;
    if (kAll < NT && (int)threadIdx.x >= kAll) lane_at = kOutside;
    extent = ACROSS ? -count * 4 : count * ld;
  }
  // contraction elements from k0 (kdim in all); moved: bytes to the operand of the second pair
  __device__ __forceinline__ void load(int k0, int kdim, ptrdiff_t moved) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + moved + (ACROSS ? (ptrdiff_t)k0 * ld : 0)), (short)0,
        ACROSS ? min(KD, kdim - k0) * ld + extent : extent, kBufferWord3);
    const int at = ACROSS || inner < kdim - k0 ? lane_at : kOutside;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      c[i] = __builtin_amdgcn_raw_buffer_load_b128(r, at + i * (NT / kRowChunks) * ld, ACROSS ? 0 : k0 * 4, 0);
  }
  __device__ __forceinline__ void put(float* lds) const {
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (kAll % NT == 0 || (int)threadIdx.x + i * NT < kAll)
        *reinterpret_cast<u32x4*>(lds + ((int)threadIdx.x / kRowChunks + i * (NT / kRowChunks)) * kRow + inner) = c[i];
  }
};

template <bool ACROSS, int TM, int KD>
__device__ __forceinline__ f32x4 fragment(const float* lds, int m, int k) {
  if constexpr (ACROSS) {
    const float* s = lds + k * (TM + kPad) + m;
    return f32x4{s[0], s[TM + kPad], s[2 * (TM + kPad)], s[3 * (TM + kPad)]};
  } else {
    const float4 v = *reinterpret_cast<const float4*>(lds + m * (KD + kPad) + k);
    return f32x4{v.x, v.y, v.z, v.w};
  }
}

template <bool ACROSS, int TM, int KD>
constexpr int stage_floats() { return ACROSS ? KD * (TM + kPad) : TM * (KD + kPad); }

// KS: groups of 4 waves, each of which takes 32 of a step's KS * 32 contraction elements; their sums
// are joined at the end, in order.
template <GroupedProduct P, int FM, int FN, int WGM, int KS>
__global__ __launch_bounds__(256 * KS) void f32_kernel(ProductArgs p) {
  constexpr bool AX = P == kWgrad, BX = P != kForward;
  constexpr int WGN = 4 / WGM, TM = 16 * FM * WGM, TN = 16 * FN * WGN;
  constexpr int KD = kStep * KS, NT = 256 * KS;
  constexpr int kA = stage_floats<AX, TM, KD>(), kB = stage_floats<BX, TN, KD>();
  __shared__ __align__(16) float lds[kA + kB];
  float *const la = lds, *const lb = lds + kA;
  TileAt t;
  if (!tile_at<P, false>(p, TM, TN, t)) return;
  const int e = t.e, ra = t.ra, m0 = t.m0, c0 = t.c0, mlim = t.mlim, clim = t.clim, kdim = t.kdim;
  const int cols = P == kForward ? p.N : p.K;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wm = wave % WGM, wn = wave / WGM;
  const int lda = P == kForward ? p.K : p.N;
  const size_t wbase = (size_t)e * p.N * p.K;
  const size_t a_at = P == kWgrad ? (size_t)ra * p.N + m0 : (size_t)(ra + m0) * lda;
  const size_t b_at = P == kForward ? wbase + (size_t)c0 * p.K
                      : P == kDgrad ? wbase + c0 : (size_t)ra * p.K + c0;

  // Sums in two levels: `acc` over kRun steps, `sum` over those. One chain of K / 4 additions was
  // twice as far from the 64-bit result at K = 4096.
  constexpr int kRun = 8;
  f32x4 acc[FM][FN], sum[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = sum[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps1 = (kdim + KD - 1) / KD;
  const int steps = (P == kDgrad && p.a2) ? 2 * steps1 : steps1;
  Stage<AX, TM, KD, NT> sa;
  Stage<BX, TN, KD, NT> sb;
  sa.set(static_cast<const float*>(p.a) + a_at, AX ? m0 : mlim, lda);
  sb.set(static_cast<const float*>(p.b) + b_at, BX ? c0 : clim, p.K);
  const bool pair = P == kDgrad && p.a2;
  const ptrdiff_t moved_a = pair ? static_cast<const char*>(p.a2) - static_cast<const char*>(p.a) : 0;
  const ptrdiff_t moved_b = pair ? static_cast<const char*>(p.b2) - static_cast<const char*>(p.b) : 0;
  auto load = [&](int st) __attribute__((always_inline)) {
    const bool second = st >= steps1;
    const int k0 = (second ? st - steps1 : st) * KD;
    sa.load(k0, kdim, second ? moved_a : 0);
    sb.load(k0, kdim, second ? moved_b : 0);
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
      const int k = group * kStep + s * 16 + (lane >> 4) * 4;
      f32x4 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = fragment<AX, TM, KD>(la, (wm * FM + i) * 16 + (lane & 15), k);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = fragment<BX, TN, KD>(lb, (wn * FN + j) * 16 + (lane & 15), k);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j][q], fa[i][q], acc[i][j], 0, 0, 0);
    }
    if (st % kRun == kRun - 1 || st == steps - 1) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          sum[i][j] += acc[i][j];
          acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
  }
  if constexpr (KS > 1) {
    static_assert((KS - 1) * FM * FN * 1024 <= kA + kB, "the groups' sums fit where the operands were");
    __syncthreads();
    float* const mine = lds + ((group - 1) * FM * FN * 4 + wave) * 256 + lane * 4;
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) *reinterpret_cast<f32x4*>(mine + (i * FN + j) * 1024) = sum[i][j];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < KS - 1; ++g)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          sum[i][j] += *reinterpret_cast<const f32x4*>(lds + ((g * FM * FN + i * FN + j) * 4 + wave) * 256 + lane * 4);
  }
  OutTile o;
  o.set(p, P == kWgrad ? (size_t)e * p.N + m0 : (size_t)ra + m0, mlim, c0, clim, cols);
#pragma unroll
  for (int i = 0; i < FM; ++i) store_fragments<FN>(o, p, sum[i], (wm * FM + i) * 16, wn * FN * 16, lane);
}

// ---------------------------------------------------------------------------------------
// bf16: tiles loaded straight into LDS
// ---------------------------------------------------------------------------------------
typedef short s16x4 __attribute__((ext_vector_type(4)));

// One transposing LDS read. The pointer is declared not to alias anything so that the compiler
// does not take the read to depend on the loads into LDS that are in flight (it would wait for
// all of them first, in every step); what is read has landed, the kernel's own waits see to that.
__device__ __forceinline__ s16x4 read_transposed(const char* __restrict__ at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
}

// One operand of a tile: T rows or columns of C's side, DK of the contraction per step, loaded
// by NW waves with buffer loads of 1 KB into LDS (16 bytes a lane). The LDS image is the
// operand's memory order, [T][DK] (along) or [DK][T] (across), in 16-byte chunks that are
// permuted within a row so that the lanes of a fragment read fall on distinct banks:
//   along   dswz of lds_tiles.h; a fragment is one 16-byte read, 8 contraction elements of row
//           lane % 16, chunk lane / 16
//   across  32-byte units, unit u of row k at u ^ x(k), x(k) = (k & 3) + 4 ((k >> 3) & 1); a fragment
//           is two transposing reads, each 4 contraction rows of 16 columns per 16 lanes (lane i
//           gives the address of row i / 4, columns 4 (i % 4) .. + 3, and gets column i of the 4
//           rows). The units of the 8 rows that a read of 32 lanes touches differ.
// Lane group g = lane / 16 takes contraction elements 8g .. 8g + 7 of a 32-long slice in both
// forms, so along and across operands meet.
template <bool ACROSS, int T, int DK, int NW>
struct Operand {
  static constexpr int kChunks = T * DK / 8;          // 16-byte chunks per step
  static constexpr int kRowChunks = (ACROSS ? T : DK) / 8;
  static constexpr int kLoads = kChunks / 64 / NW;    // load instructions per wave and step
  static constexpr int kRowsPerLoad = 64 / kRowChunks;
  static_assert(kLoads >= 1 && kLoads * 64 * NW == kChunks, "loads split evenly over the waves");
  static_assert(!ACROSS || T >= 128, "across: at least 8 units in a row");
  static_assert(kRowsPerLoad * NW % 16 == 0, "the permutation repeats from one load to the next");
  // Past any extent (at most 2^20 * 2 * 256 bytes): the lanes that load nothing but zeros.
  static constexpr int kOutside = 0x40000000;

  const char* base;  // along: the tile's first row; across: its first column in row 0
  unsigned extent;   // along: bytes of the tile's rows
  int ld;            // row stride in bytes
  int col;           // across: bytes before the tile's first column in a row
  int lane_at, stride, k_of_lane;

  __device__ __forceinline__ static int unit(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

  // origin: the operand's element (0, 0) for this expert; first: the tile's first row (along)
  // or column (across); count: how many rows of the tile exist (along); ld_elems: row stride.
  __device__ __forceinline__ void set(const __bf16* origin, int first, int count, int ld_elems, int wave, int lane) {
    ld = ld_elems * 2;
    const int row = wave * kRowsPerLoad + lane / kRowChunks, pos = lane % kRowChunks;
    stride = NW * kRowsPerLoad * ld;
    if constexpr (ACROSS) {
      base = reinterpret_cast<const char*>(origin) + (size_t)first * 2;
      col = first * 2;
      lane_at = row * ld + (pos ^ (unit(row) << 1)) * 16;
    } else {
      base = reinterpret_cast<const char*>(origin) + (size_t)first * ld;
      extent = (unsigned)count * (unsigned)ld;
      const int chunk = dswz<kRowChunks>(row, pos) - row * kRowChunks;
      lane_at = row * ld + chunk * 16;
      k_of_lane = chunk * 8;
    }
  }

  // Contraction elements k0 .. k0 + DK - 1 of the tile into `slot`; those at or past kdim, and
  // rows or columns that do not exist, become zeros. `moved`: bytes from this operand to the one
  // of the second pair.
  template <int AUX>
  __device__ __forceinline__ void issue(u32x4* slot, int k0, int kdim, ptrdiff_t moved, int wave) const {
    if constexpr (ACROSS) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + moved + (size_t)k0 * ld), (short)0, min(DK, kdim - k0) * ld - col, kBufferWord3);
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        buffer_load_lds16<AUX>(r, slot + (wave + i * NW) * 64, lane_at + i * stride, 0);
    } else {
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc((void*)(base + moved), (short)0, (int)extent, kBufferWord3);
      const bool in = k_of_lane < kdim - k0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        buffer_load_lds16<AUX>(r, slot + (wave + i * NW) * 64, in ? lane_at + i * stride : kOutside, k0 * 2);
    }
  }

  // Fragment of 16 rows or columns from m0, contraction slice h (32 elements).
  __device__ __forceinline__ static bf16x8 read(const u32x4* slot, int m0, int h, int lane) {
    bf16x8 f;
    if constexpr (ACROSS) {
      const int i = lane & 15, g = lane >> 4;
      const int k = h * 32 + g * 8 + (i >> 2);
      const char* at = reinterpret_cast<const char*>(slot) + k * (T * 2) + ((m0 >> 4) ^ unit(k)) * 32 + (i & 3) * 8;
      const s16x4 v[2] = {read_transposed(at), read_transposed(at + 4 * T * 2)};  // unit(k + 4) = unit(k)
      __builtin_memcpy(&f, v, 16);
    } else {
      const u32x4 v = slot[dswz<kRowChunks>(m0 + (lane & 15), h * 4 + (lane >> 4))];
      __builtin_memcpy(&f, &v, 16);
    }
    return f;
  }
};

// Workgroup barrier without a fence: a fence would make the compiler wait for every outstanding
// load into LDS. The signal fences keep the compiler from moving LDS accesses across it.
__device__ __forceinline__ void bare_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Until at most min(n, MOST) steps of LOADS loads each are in flight; n is the same in every lane.
template <int LOADS, int MOST>
__device__ __forceinline__ void wait_steps(int n) {
  if (n >= MOST) wait_vmcnt<MOST * LOADS>();
  else static_for<MOST>([&](auto i) { if (n == decltype(i)::value) wait_vmcnt<decltype(i)::value * LOADS>(); });
}

// A workgroup of WGM x WGN waves computes a tile of C, each wave WM x WN of it with
// v_mfma_f32_16x16x32_bf16; steps of DK go through a ring of RING slots in LDS. While a
// slice's products run, the fragments of the next slice are read (B into the other of two
// register sets, each A fragment after its last product); the barrier that frees a step's slot
// stands before the products of the step's last slice, whose fragments are in registers by then.
// DEAL: each wave runs a loop compiled for the number of its 16-row fragments that hold rows, so
// a partial tile costs what its rows need; waves w and w + 4 share a SIMD and own different
// halves of the tile, so every SIMD has work.
//
// Measured, 65,536 rows dealt by Zipf 1.2 to 32 experts of 2048 x 7168 (bf16): forward 1.56 - 1.62 ms
// (1.19 - 1.23 PFLOP/s), two input gradients 3.09 - 3.26 ms (1.18 - 1.25), fp32 weight gradients 1.83 -
// 1.91 ms (1.01 - 1.05); a library product of these sizes without the experts reaches 1.34, 1.13 and
// 1.02. The sums over the contraction are one chain per value: 4.0e-7 from the 64-bit result on the decode
// product below, where a library product in fp32 is 3.7e-7 from it; a second set of accumulators does not
// fit beside the large tile's. The clock falls to 1.9 - 2.05 GHz under the power limit; of the cycles the matrix instructions take 59%
// (forward, input gradients) and 47% (weight gradients, whose 1.9 GB of fp32 stores take another
// 20%). LDS is busy 18 - 23% without bank conflicts; taking out, one by one, LDS reads, loads that
// hit in the L2 and those that miss it gives back about 9% of the time each. Few rows are bound by the
// stream of the weights: 1,024 rows over 128 experts of 1536 x 4096 take 252 us (1.6 GB, 6.4 TB/s),
// 8 rows on 8 of them 18 us (101 MB, 5.6 TB/s).
//
// The tile: 256 x 256 with 8 waves of 128 x 64 has the most products per byte that the registers
// of 8 waves hold, and its two slots of 64 fill 128 KB of LDS. Slower were 4 or 5 slots of 32 (1.83 ms
// forward), a slot more for one operand (1.72), two workgroups per CU with half the tile (2.41),
// 4 waves of 128 x 128 (accumulators move between register files), and workgroups that stay and load
// the next tile's first steps under the last products (1.66).
template <GroupedProduct P, int WM, int WN, int WGM, int WGN, int DK, int RING, bool ONCE, bool DEAL>
__global__ __launch_bounds__(64 * WGM * WGN) void tile_kernel(ProductArgs p) {
  constexpr bool AX = P == kWgrad, BX = P != kForward;
  constexpr int TM = WM * WGM, TN = WN * WGN, NW = WGM * WGN;
  constexpr int MF = WM / 16, NF = WN / 16, NS = DK / 32;
  using OA = Operand<AX, TM, DK, NW>;
  using OB = Operand<BX, TN, DK, NW>;
  constexpr int STAGE = OA::kChunks + OB::kChunks, LOADS = OA::kLoads + OB::kLoads;
  __shared__ __align__(16) u32x4 ring[RING * STAGE];
  TileAt t;
  if (!tile_at<P, DEAL>(p, TM, TN, t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WGN * WM, wn = wave % WGN * WN;

  OA oa;
  OB ob;
  const size_t weights = (size_t)t.e * p.N * p.K;
  const __bf16 *a = static_cast<const __bf16*>(p.a), *b = static_cast<const __bf16*>(p.b);
  if constexpr (P == kForward) {
    oa.set(a + (size_t)t.ra * p.K, t.m0, t.mlim, p.K, wave, lane);
    ob.set(b + weights, t.c0, t.clim, p.K, wave, lane);
  } else if constexpr (P == kDgrad) {
    oa.set(a + (size_t)t.ra * p.N, t.m0, t.mlim, p.N, wave, lane);
    ob.set(b + weights, t.c0, t.clim, p.K, wave, lane);
  } else {
    oa.set(a + (size_t)t.ra * p.N, t.m0, t.mlim, p.N, wave, lane);
    ob.set(b + (size_t)t.ra * p.K, t.c0, t.clim, p.K, wave, lane);
  }
  const bool pair = P == kDgrad && p.a2;
  const ptrdiff_t moved_a = pair ? static_cast<const char*>(p.a2) - static_cast<const char*>(p.a) : 0;
  const ptrdiff_t moved_b = pair ? static_cast<const char*>(p.b2) - static_cast<const char*>(p.b) : 0;
  const int steps1 = (t.kdim + DK - 1) / DK, steps = pair ? 2 * steps1 : steps1;
  // The expert's weights are read by this row tile alone, in whole lines (1,024 rows on 128 experts of
  // 1536 x K, two input gradients: Zipf 1.2: K = 4096 439 us against 484 with plain loads, K = 4104 517 against 470).
  const bool once = ONCE && t.rb - t.ra <= TM && p.K % 64 == 0;

  auto issue = [&](int st) __attribute__((always_inline)) {
    u32x4* slot = ring + st % RING * STAGE;
    const bool second = st >= steps1;
    const int k0 = (second ? st - steps1 : st) * DK;
    oa.template issue<0>(slot, k0, t.kdim, second ? moved_a : 0, wave);
    if (once)
      ob.template issue<kNonTemporal>(slot + OA::kChunks, k0, t.kdim, second ? moved_b : 0, wave);
    else
      ob.template issue<0>(slot + OA::kChunks, k0, t.kdim, second ? moved_b : 0, wave);
  };

  const int cols = P == kForward ? p.N : p.K;
  const size_t row0 = P == kWgrad ? (size_t)t.e * p.N + t.m0 : (size_t)t.ra + t.m0;
  // F: this wave's fragments with rows
  auto run = [&](auto present) __attribute__((always_inline)) {
    constexpr int F = decltype(present)::value;
    f32x4 acc[F ? F : 1][NF];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    bf16x8 fa[F ? F : 1], fb[2][NF];
    if (steps > 0) {
#pragma unroll
      for (int r = 0; r < RING; ++r)
        if (r < steps) issue(r);
      wait_steps<LOADS, RING - 1>(steps - 1);
      bare_barrier();
#pragma unroll
      for (int j = 0; j < (F ? NF : 0); ++j) fb[0][j] = OB::read(ring + OA::kChunks, wn + j * 16, 0, lane);
#pragma unroll
      for (int i = 0; i < F; ++i) fa[i] = OA::read(ring, wm + i * 16, 0, lane);
    }
    for (int st = 0; st < steps; ++st) {
      const u32x4* slot = ring + st % RING * STAGE;
      const u32x4* next = ring + (st + 1) % RING * STAGE;
      static_for<NS>([&](auto hc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value, cur = h & 1;
        if (h == NS - 1) {
          wait_lgkmcnt0();  // this wave's reads of step st are back
          if (st + 1 < steps) {
            // step st + 1 has landed for this wave, and after the barrier for all; all are done
            // with step st's slot
            wait_steps<LOADS, RING - 2>(steps - 2 - st);
            bare_barrier();
            if (st + RING < steps) issue(st + RING);
          }
        }
        // Past the last step these reads bring nothing that is used (any slot, in bounds).
        const u32x4* rs = h + 1 < NS ? slot : next;
        constexpr int rh = (h + 1) % NS;
#pragma unroll
        for (int j = 0; j < (F ? NF : 0); ++j) fb[cur ^ 1][j] = OB::read(rs + OA::kChunks, wn + j * 16, rh, lane);
#pragma unroll
        for (int i = 0; i < F; ++i) {
#pragma unroll
          for (int j = 0; j < NF; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[cur][j], fa[i], acc[i][j], 0, 0, 0);
          fa[i] = OA::read(rs, wm + i * 16, rh, lane);
        }
        // order of the slice: the B reads, then each A fragment's products and its next read
        if constexpr (F > 0) __builtin_amdgcn_sched_group_barrier(0x100, NF * (BX ? 2 : 1), 0);
#pragma unroll
        for (int i = 0; i < F; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, NF, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, AX ? 2 : 1, 0);
        }
        __atomic_signal_fence(__ATOMIC_SEQ_CST);  // the reads stay in this slice
      });
    }
    OutTile o;
    o.set(p, row0, t.mlim, t.c0, t.clim, cols);
#pragma unroll
    for (int i = 0; i < F; ++i) store_fragments<NF>(o, p, acc[i], wm + i * 16, wn, lane);
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

// Tiles of TM x TN that a launch covers: for wgrad every expert's, for the row products the
// most that the rows can fill (an expert's last row tile may be partial).
long long tile_items(GroupedProduct kind, const GroupedGemmArgs& a, int TM, int TN) {
  const long long cols = ((kind == kForward ? a.N : a.K) + TN - 1LL) / TN;
  if (kind == kWgrad) return a.E * ((a.N + TM - 1LL) / TM) * cols;
  return (a.rows / TM + (a.E < a.rows ? a.E : a.rows)) * cols;
}

template <GroupedProduct P, int WM, int WN, int WGM, int WGN, int DK, int RING, bool ONCE, bool DEAL>
hipError_t launch_tiles(const GroupedGemmArgs& a, const ProductArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(P, a, WM * WGM, WN * WGN));
  tile_kernel<P, WM, WN, WGM, WGN, DK, RING, ONCE, DEAL><<<(unsigned)grid, 64 * WGM * WGN, 0, stream>>>(p);
  return hipGetLastError();
}

template <GroupedProduct P, int FM, int FN, int WGM, int KS>
hipError_t launch_f32(const GroupedGemmArgs& a, const ProductArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(P, a, 16 * FM * WGM, 16 * FN * (4 / WGM)));
  f32_kernel<P, FM, FN, WGM, KS><<<(unsigned)grid, 256 * KS, 0, stream>>>(p);
  return hipGetLastError();
}

// How many of them to expect; with several experts, each one's last row tile is taken to be half full.
double expected_tiles(GroupedProduct kind, const GroupedGemmArgs& a, int TM, int TN) {
  const double active = a.E < a.rows ? a.E : a.rows;
  const double rows = kind == kWgrad ? a.E * std::ceil(a.N / (double)TM)
                      : a.E == 1     ? std::ceil(a.rows / (double)TM)
                                     : std::fmax(a.rows / (double)TM + 0.5 * active, active);
  return rows * std::ceil((kind == kForward ? a.N : a.K) / (double)TN);
}

// Time, per contraction step of 64 (us), of TM x TN tiles over the CUs, `fit` to each at a time: `full`
// where the CUs are filled, `alone` for a last round with at most one tile to a CU. The times are from
// products of 512 to 8192 rows over 1 to 16 experts (forward, 1024 rows of 2048 x 7168 for one expert:
// 138 us in tiles of 256, 83 of 128, 59 of 64 x 128; 4096 rows of 4096 x 1024 for 8 experts: 33, 44 and 56).
struct TileCost {
  int TM, TN, fit;
  double alone, full;
};
constexpr TileCost kBig{256, 256, 1, 1.3, 1.3}, kMid{128, 128, 2, 0.7, 1.05}, kSmall{64, 128, 2, 0.48, 0.75};

double step_time(GroupedProduct kind, const GroupedGemmArgs& a, const TileCost& c, int cus) {
  const double tiles = expected_tiles(kind, a, c.TM, c.TN);
  const double slots = (double)cus * c.fit, whole = std::floor(tiles / slots), left = tiles - whole * slots;
  return whole * c.full + (left == 0 ? 0 : left <= cus ? c.alone : c.full);
}

// Whether C's rows are stored non-temporally. Rows of whole 128-byte lines always are. Others share lines
// between tiles and between a row's pieces; those lines are put together in the L2 if they may stay
// there, which pays unless the products are long enough that the L2 is worth more to the operands
// (16,384 rows over 8 experts of 3288 x K, bf16, plain and non-temporal: K = 264 55 and 67 us, 1032 127
// and 137, 4104 508 and 493; weight gradients of 42 experts of 2488 x 3288, bf16: 64 rows per expert 213 and
// 278 us, 256 357 and 309; fp32: 256 rows 480 and 592, 512 641 and 620).
int stream_rows(const GroupedGemmArgs& a, GroupedProduct kind) {
  const long long cols = kind == kForward ? a.N : a.K;
  if (cols * (a.out_bf16 ? 2 : 4) % 128 == 0) return 1;
  if (kind == kWgrad) return a.rows / a.E >= (a.out_bf16 ? 192 : 512);
  return (kind == kForward ? a.K : a.N) >= 4096;
}

template <GroupedProduct P>
hipError_t launch_product(const GroupedGemmArgs& a, int cus, hipStream_t stream) {
  const ProductArgs p{a.a, a.b, a.a2, a.b2, a.out, a.offsets, a.rows, a.E, a.N, a.K,
                      a.out_bf16 ? 1 : 0, a.accumulate ? 1 : 0, stream_rows(a, P)};
  if (!a.bf16) {
    // Few rows leave most of a 64-row tile's products empty: at 64 experts of 1024 x 2048, even rows,
    // tiles of 16 x 64 against 64 x 64 took (forward) 123 and 148 us at 1 row per expert, 125 and
    // 162 at 32, 205 and 170 at 64. The contraction is split over the waves where there are few tiles
    // (one expert of 1024 x 1024, 512 rows, forward: 28 us in tiles of 64 x 64, 24 split in two, 20 in tiles of
    // 16 x 64 split in four; 4 experts, 1,024 rows, input gradient 31, 26 and 36) or one row tile per
    // expert (the 64 experts at 1 row 97 us against 123); at 32 rows each it costs (133 against 125).
    if constexpr (P == kWgrad) {
      // few tiles of many rows: one expert of 1024 x 1024, 4,096 rows 87 us against 113
      if (a.rows / a.E >= 128 && expected_tiles(P, a, 64, 64) <= cus) return launch_f32<P, 2, 2, 2, 2>(a, p, stream);
      return launch_f32<P, 2, 2, 2, 1>(a, p, stream);
    } else {
      if (a.rows / a.E < 16 || tile_items(P, a, 16, 64) <= 5LL * cus / 2)
        return launch_f32<P, 1, 1, 1, 4>(a, p, stream);
      if (a.rows / a.E < 48) return launch_f32<P, 1, 1, 1, 1>(a, p, stream);
      if (tile_items(P, a, 64, 64) <= 2LL * cus) return launch_f32<P, 2, 2, 2, 2>(a, p, stream);
      return launch_f32<P, 2, 2, 2, 1>(a, p, stream);
    }
  }
  // Which tiles, from the sizes alone (the host does not know the offsets). Measured at 64 experts of
  // 2048 x 4096, rows spread evenly (us):
  //   rows per expert             8     16     32     64     96    128    256    512
  //   forward  32 x 64 tiles    164    172    188    257    325    413    740   1368
  //            64 x 128         181    184    190    198    249    265    439    822
  //            128 x 128        220    222    225    227    230    234    351    634
  //            256 x 256        241    242    245    250    255    259    281    479
  //   dgrad 2  32 x 128         322    341    357    497    580    720   1295   2444
  //            64 x 128         328    334    347    364    529    553    922   1747
  //            128 x 128        328    335    340    359    383    396    704   1309
  //            256 x 256        375    377    381    389    394    413    527    971
  //   wgrad    128 x 128, fp32  341    352    360    368    415    422    584   1001
  //            256 x 256, fp32  429    439    439    443    471    476    560    758
  //            128 x 128, bf16  228    244    249    261    312    319    460    850
  //            256 x 256, bf16  220    228    229    238    279    286    389    618
  // (Where two are within 7% the rule may take either.) With rows dealt by Zipf 1.2 or 0.6 the borders are the
  // same or a little lower, but forward tiles of 128 stay ahead at 128 rows (Zipf 0.6: 259 us against
  // 326; at 192, evenly dealt, 325 against 271). With 1 row per expert a bf16 weight gradient takes 175 us
  // in tiles of 128, 189 in tiles of 256 (Zipf 1.2; evenly dealt 226 and 220). Large tiles are wasted on
  // a width that fills less than one of them, and where there are fewer of them than CUs (step_time).
  const long long mean = a.rows / a.E;
  const double big = step_time(P, a, kBig, cus), mid = step_time(P, a, kMid, cus);
  if constexpr (P == kWgrad) {
    if (mean >= (a.out_bf16 ? 16 : 160) && a.N > 128 && a.K > 128 && big <= mid)
      return launch_tiles<P, 128, 64, 2, 4, 64, 2, false, true>(a, p, stream);
    // With a CU to each tile, eight waves and steps of 128: one expert of 1024 x 1024, 8,192 rows 63 us
    // against 96.
    if (expected_tiles(P, a, 128, 128) <= cus)
      return launch_tiles<P, 64, 32, 2, 4, 128, 2, false, false>(a, p, stream);
    return launch_tiles<P, 64, 64, 2, 2, 64, 2, false, false>(a, p, stream);
  } else {
    // With a CU to each tile, the smallest tiles of which that is so, with as many steps in flight as the
    // LDS holds, eight waves and steps of 128 (in steps of 64 their waits and barriers take most of the
    // time). One expert of 1024 x 2048, forward: 256 rows 10.0 us in tiles of 32 x 64 against 17.5 in the
    // three-slot tiles of 64 x 128; 1,024 rows 14.4 in these tiles of 64 x 128 against 18.5; 4,096 rows 23.0
    // in these of 128 against 28.0 in the ones for full CUs. Input gradients of two: 1,536 rows 20.8 in these of
    // 128 against 28.4; 512 rows over 8 such experts 19.0 in these of 64 x 128 against 22.7. One token for 8 of 128
    // experts of 1536 x 4096 takes 18.5 in rings of six and of three.
    const auto few = [&](int TM, int TN) { return expected_tiles(P, a, TM, TN) <= cus; };
    if constexpr (P == kForward) {
      if (few(32, 64)) return launch_tiles<P, 32, 16, 1, 4, 128, 6, true, false>(a, p, stream);
    } else {
      if (few(32, 128)) return launch_tiles<P, 32, 16, 1, 8, 128, 3, true, false>(a, p, stream);
    }
    if (few(64, 128)) return launch_tiles<P, 32, 32, 2, 4, 128, 3, true, false>(a, p, stream);
    if (few(128, 128)) return launch_tiles<P, 64, 32, 2, 4, 128, 2, true, false>(a, p, stream);
    if (mean >= 96) {
      const double small = step_time(P, a, kSmall, cus);
      if (mean >= (P == kForward ? 192 : 96) && (P == kForward ? a.N : a.K) > 128 && big <= mid && big <= small)
        return launch_tiles<P, 128, 64, 2, 4, 64, 2, false, true>(a, p, stream);
      if (mid <= small) return launch_tiles<P, 64, 64, 2, 2, 64, 2, true, false>(a, p, stream);
    }
    if (mean >= 12) return launch_tiles<P, 32, 64, 2, 2, 64, 3, true, false>(a, p, stream);
    if constexpr (P == kForward) return launch_tiles<P, 32, 16, 1, 4, 128, 3, true, false>(a, p, stream);
    return launch_tiles<P, 32, 32, 1, 4, 64, 3, true, false>(a, p, stream);
  }
}

}  // namespace

bool grouped_gemm_fits(const GroupedGemmArgs& a, GroupedProduct kind) {
  // the smallest tiles that launch_product may take (but where it takes them for being few)
  const long long mean = a.rows / a.E;
  int TM = 64, TN = 64, threads = 256;
  if (kind == kWgrad) TM = TN = a.bf16 ? 128 : 64;
  else if (a.bf16) TM = mean >= 12 ? 64 : 32, TN = mean >= 12 ? 128 : 64;
  else if (mean < 48) TM = 16, threads = mean < 16 ? 1024 : 256;
  return xcd_grid(tile_items(kind, a, TM, TN)) <= kMaxWorkgroups * 256 / threads;
}

hipError_t launch_grouped_gemm(const GroupedGemmArgs& a, GroupedProduct kind, hipStream_t stream) {
  DeviceInfo dev;
  const hipError_t e = device_info(&dev);
  if (e != hipSuccess) return e;
  switch (kind) {
    case kForward: return launch_product<kForward>(a, dev.num_cus, stream);
    case kDgrad: return launch_product<kDgrad>(a, dev.num_cus, stream);
    case kWgrad: return launch_product<kWgrad>(a, dev.num_cus, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
