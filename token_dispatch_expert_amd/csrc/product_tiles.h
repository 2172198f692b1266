// Device and host helpers of the grouped products' tiles, shared by the kernels for bf16, fp32 and 4-bit
// weights: where a tile lies, its operands in LDS, its stores, and the model that picks tiles.
#pragma once

#include <cmath>

#include "grouped.h"
#include "lds_tiles.h"

namespace moe {

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

// Tiles of TM x TN that a launch covers: for wgrad every expert's, for the row products the
// most that the rows can fill (an expert's last row tile may be partial).
inline long long tile_items(GroupedProduct kind, const GroupedGemmArgs& a, int TM, int TN) {
  const long long cols = ((kind == kForward ? a.N : a.K) + TN - 1LL) / TN;
  if (kind == kWgrad) return a.E * ((a.N + TM - 1LL) / TM) * cols;
  return (a.rows / TM + (a.E < a.rows ? a.E : a.rows)) * cols;
}

// How many of them to expect; with several experts, each one's last row tile is taken to be half full.
inline double expected_tiles(GroupedProduct kind, const GroupedGemmArgs& a, int TM, int TN) {
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

inline double step_time(GroupedProduct kind, const GroupedGemmArgs& a, const TileCost& c, int cus) {
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
inline int stream_rows(const GroupedGemmArgs& a, GroupedProduct kind) {
  const long long cols = kind == kForward ? a.N : a.K;
  if (cols * (a.out_bf16 ? 2 : 4) % 128 == 0) return 1;
  if (kind == kWgrad) return a.rows / a.E >= (a.out_bf16 ? 192 : 512);
  return (kind == kForward ? a.K : a.N) >= 4096;
}

}  // namespace moe
