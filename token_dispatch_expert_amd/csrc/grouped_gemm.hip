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
#include "product_tiles.h"

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
