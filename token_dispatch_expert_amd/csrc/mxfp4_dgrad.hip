// The input gradient of the products with MXFP4 weights: dx[r] = W_e^T dy[r] (+ W2_e^T dy2[r]).
//
// The contraction runs over W's rows, while codes and scales lie along them, so the matrix instructions cannot take the
// codes as they are stored. A step's weights are converted to bf16 on their way into LDS instead, exactly, where they lie
// as bf16 weights would, and the transposing LDS reads of the bf16 input gradient bring them to the matrix
// instructions: the codes move a quarter of the bytes from HBM, and the products run at the bf16 rate. With few rows
// per expert, where a conversion serves few products, the codes do not pass LDS (mx_dgrad_stream_kernel).
#include "mxfp4.h"
#include "mxfp4_internal.h"
#include "mxfp4_shapes.h"
#include "product_tiles.h"

namespace moe {

namespace {

struct MxDgradArgs {
  ProductArgs p;  // a: dy, b: W's codes; a2, b2: the second pair, or null
  const uint8_t *scales, *scales2;
};

// Steps of DK rows of W: each thread loads CPT chunks of 16 bytes (32 columns of a row) with their scale bytes, a step before
// it converts and writes them into the image that Operand<true, ..> reads.
template <int TN, int DK, int NT>
struct Codes {
  static constexpr int kRowChunks = TN / 32, CPT = DK * kRowChunks / NT, kRowsPerPass = NT / kRowChunks;
  static_assert(CPT >= 1 && CPT * NT == DK * kRowChunks && kMxBlock % TN == 0, "chunks split evenly over the threads");
  using Image = Operand<true, TN, DK, NT / 64>;
  const char* base;       // the tile's first column in W's row 0
  const uint8_t* scales;  // of W's row 0, in the block that holds the tile's columns
  int ld, col, row, part; // bytes of a row; bytes before the tile's first column; this thread's first row and chunk
  u32x4 c[CPT];
  unsigned s[CPT];

  __device__ __forceinline__ void set(const MxDgradArgs& a, int e, int c0) {
    const ProductArgs& p = a.p;
    ld = p.K / 2;
    col = c0 / 2;
    base = static_cast<const char*>(p.b) + (size_t)e * p.N * ld + col;
    row = threadIdx.x / kRowChunks;
    part = threadIdx.x % kRowChunks;
    scales = a.scales + mx_scale_at(e, mx_blocks(p.K), c0 / kMxBlock, p.N, 0) + (c0 & (kMxBlock - 1)) / kMxGroup;
  }
  // rows k0 .. k0 + DK - 1 of W (of N); rows past the last are zeros. What a tile's columns past K read is
  // in bounds and meets only columns of dx that do not exist.
  __device__ __forceinline__ void load(int k0, int N, ptrdiff_t moved, ptrdiff_t scales_moved) {
    const int left = N - k0;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)(base + moved + (size_t)k0 * ld), (short)0,
                                                                       min(DK, left) * ld - col, kBufferWord3);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(scales + scales_moved + (size_t)k0 * 8), (short)0, min(DK, left) * 8, kBufferWord3);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int n = row + i * kRowsPerPass;
      c[i] = __builtin_amdgcn_raw_buffer_load_b128(r, n * ld + part * 16, 0, 0);
      s[i] = (unsigned char)__builtin_amdgcn_raw_buffer_load_b8(rs, n * 8 + part, 0, 0);
    }
  }
  __device__ __forceinline__ void put(u32x4* slot) const {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int n = row + i * kRowsPerPass;
      const float scale = mx_scale_f32(s[i]);
      char* const to = reinterpret_cast<char*>(slot) + n * (TN * 2);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<bf16x8*>(to + ((part * 2 + (q >> 1)) ^ Image::unit(n)) * 32 + (q & 1) * 16) =
            mx_bf16x8(c[i][q], scale);
    }
  }
};

// As tile_kernel of the bf16 products (grouped_gemm.hip), with W through registers. The matrix instructions and the card's power
// bound it: two gradients of 65,536 rows over 32 experts of 2048 x 7168 in 2.93 - 3.21 ms over several cards, 1.20 - 1.31 PFLOP/s, matrix
// instructions 56% of the cycles; with bf16 weights 3.09 - 3.26. 22% of the cycles are bank conflicts of the converted weights' writes;
// an order of them without two thirds of those took as long (3,054 - 3,082 against 3,047 - 3,058 us).
template <int WM, int WN, int WGM, int WGN, int DK, bool DEAL>
__global__ __launch_bounds__(64 * WGM * WGN) void mx_dgrad_kernel(MxDgradArgs a) {
  constexpr int TM = WM * WGM, TN = WN * WGN, NW = WGM * WGN;
  constexpr int MF = WM / 16, NF = WN / 16, NS = DK / 32;
  using OA = Operand<false, TM, DK, NW>;
  using OB = Operand<true, TN, DK, NW>;
  constexpr int STAGE = OA::kChunks + OB::kChunks, SLOTS = 2;
  static_assert(SLOTS * STAGE * 16 <= 160 * 1024, "LDS");
  __shared__ __align__(16) u32x4 ring[SLOTS * STAGE];
  const ProductArgs& p = a.p;
  TileAt t;
  if (!tile_at<kDgrad, DEAL>(p, TM, TN, t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WGN * WM, wn = wave % WGN * WN;

  OA oa;
  Codes<TN, DK, 64 * NW> codes;
  oa.set(static_cast<const __bf16*>(p.a) + (size_t)t.ra * p.N, t.m0, t.mlim, p.N, wave, lane);
  codes.set(a, t.e, t.c0);
  const bool pair = p.a2 != nullptr;
  const ptrdiff_t moved_a = pair ? static_cast<const char*>(p.a2) - static_cast<const char*>(p.a) : 0;
  const ptrdiff_t moved_b = pair ? static_cast<const char*>(p.b2) - static_cast<const char*>(p.b) : 0;
  const ptrdiff_t moved_s = pair ? a.scales2 - a.scales : 0;
  const int steps1 = (t.kdim + DK - 1) / DK, steps = pair ? 2 * steps1 : steps1;

  auto issue = [&](int st) __attribute__((always_inline)) {
    const bool second = st >= steps1;
    oa.template issue<0>(ring + st % SLOTS * STAGE, (second ? st - steps1 : st) * DK, t.kdim, second ? moved_a : 0, wave);
  };
  auto load = [&](int st) __attribute__((always_inline)) {
    const bool second = st >= steps1;
    codes.load((second ? st - steps1 : st) * DK, t.kdim, second ? moved_b : 0, second ? moved_s : 0);
  };
  auto run = [&](auto present) __attribute__((always_inline)) {
    constexpr int F = decltype(present)::value;
    f32x4 acc[F ? F : 1][NF];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    bf16x8 fa[F ? F : 1], fb[2][NF];
#pragma unroll
    for (int r = 0; r < SLOTS; ++r)
      if (r < steps) {
        load(r);
        issue(r);
        codes.put(ring + r * STAGE + OA::kChunks);
      }
    if (SLOTS < steps) load(SLOTS);
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    bare_barrier();
#pragma unroll
    for (int j = 0; j < (F ? NF : 0); ++j) fb[0][j] = OB::read(ring + OA::kChunks, wn + j * 16, 0, lane);
#pragma unroll
    for (int i = 0; i < F; ++i) fa[i] = OA::read(ring, wm + i * 16, 0, lane);
    for (int st = 0; st < steps; ++st) {
      u32x4* slot = ring + st % SLOTS * STAGE;
      const u32x4* next = ring + (st + 1) % SLOTS * STAGE;
      static_for<NS>([&](auto hc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value, cur = h & 1;
        if (h == NS - 1) {
          wait_lgkmcnt0();  // this wave's reads of step st are back, its weights of later steps written
          if (st + 1 < steps) {
            // step st + 1 has landed for this wave, and after the barrier for all; all are done with step st's slot
            wait_vmcnt<0>();
            bare_barrier();
            if (st + SLOTS < steps) {
              codes.put(slot + OA::kChunks);
              if (st + SLOTS + 1 < steps) load(st + SLOTS + 1);
              issue(st + SLOTS);
            }
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
        __atomic_signal_fence(__ATOMIC_SEQ_CST);  // the reads stay in this slice
      });
    }
    OutTile o;
    o.set(p, (size_t)t.ra + t.m0, t.mlim, t.c0, t.clim, p.K);
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

template <int WM, int WN, int WGM, int WGN, int DK, bool DEAL>
hipError_t launch_tiles(const GroupedGemmArgs& g, const MxDgradArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(kDgrad, g, WM * WGM, WN * WGN));
  mx_dgrad_kernel<WM, WN, WGM, WGN, DK, DEAL><<<(unsigned)grid, 64 * WGM * WGN, 0, stream>>>(p);
  return hipGetLastError();
}

// Few rows per expert: the codes go straight to registers, and waves share the contraction, wave w steps w, w + NW, .. of 32 rows of W
// (of the two pairs one after the other). Lane r + 16 g holds, of W's rows 8 g .. 8 g + 7, the same NC dwords of 8 columns
// each, so that it has 8 contraction elements of each of its columns: converted in pairs of columns, two rows' halves
// joined by v_perm are what the matrix instructions take, without LDS. Instruction j takes column 8 NC r + j for lane r; a row's
// load is 64 NC bytes. At the end the waves' sums are joined in order in LDS.
// Two gradients of 64 experts of 2048 x 4096 (570 MB of weights) with a row each take 104 us, 5.5 TB/s, the weights' stream (223 in the best
// tiles through LDS). There loads a step further ahead gain nothing (122 against 127 us for 128 columns, 110 against 107 for
// 256): every CU is full and other waves fill the time. 104 rows over 8 experts of 1544 x 800 take 12.2 us against 21.8, bound by
// latency: 70 workgroups on 256 CUs, whose 8 waves share 98 steps, 12 or 13 loads of a wave one after the other.
template <int MF, int NC, int NW>
__global__ __launch_bounds__(64 * NW) void mx_dgrad_stream_kernel(MxDgradArgs a) {
  typedef unsigned Dwords __attribute__((ext_vector_type(NC)));
  constexpr int TM = 16 * MF, TN = 128 * NC, kLaneColumns = 8 * NC, kPitch = TN + 4;
  constexpr int kOutside = 0x40000000;  // past any extent (at most TM rows of 2^21 bytes)
  __shared__ __align__(16) float sums[NW][16][kPitch];
  const ProductArgs& p = a.p;
  TileAt t;
  if (!tile_at<kDgrad, false>(p, TM, TN, t)) return;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = t.kdim, ld = p.K / 2, col = t.c0 / 2, dy_ld = N * 2;
  const size_t row0 = (size_t)t.ra + t.m0;
  const bool pair = p.a2 != nullptr;
  const int steps1 = (N + 31) / 32, steps = pair ? 2 * steps1 : steps1;
  const size_t we = (size_t)t.e * N * ld + col, se = mx_scale_at(t.e, mx_blocks(p.K), t.c0 / kMxBlock, N, 0);
  const int group = (t.c0 & (kMxBlock - 1)) / kMxGroup + lr * kLaneColumns / kMxGroup;  // of the lane's columns in the block

  struct Step {
    Dwords c[8];
    unsigned s[8];
    u32x4 d[MF];
  };
  // step st (past the last: zeros); what columns past K read is in bounds and meets only columns of dx that do not exist
  auto load = [&](Step& q, int st) __attribute__((always_inline)) {
    const bool in = st < steps, second = in && st >= steps1;
    const int k0 = in ? (second ? st - steps1 : st) * 32 : 0, left = in ? min(32, N - k0) : 0;
    const __amdgpu_buffer_rsrc_t rd = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(static_cast<const char*>(second ? p.a2 : p.a) + row0 * dy_ld), (short)0, t.mlim * dy_ld, kBufferWord3);
    const __amdgpu_buffer_rsrc_t rc =
        __builtin_amdgcn_make_buffer_rsrc((void*)(static_cast<const char*>(second ? p.b2 : p.b) + we + (size_t)k0 * ld),
                                          (short)0, in ? left * ld - col : 0, kBufferWord3);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((second ? a.scales2 : a.scales) + se + (size_t)k0 * 8), (short)0, left * 8, kBufferWord3);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = (lg * 8 + i) * ld + lr * (4 * NC);
      if constexpr (NC == 1) q.c[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rc, at, 0, 0);
      else q.c[i] = __builtin_amdgcn_raw_buffer_load_b64(rc, at, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) q.s[i] = (unsigned char)__builtin_amdgcn_raw_buffer_load_b8(rs, (lg * 8 + i) * 8 + group, 0, 0);
#pragma unroll
    for (int f = 0; f < MF; ++f)  // (N is a multiple of 8: a lane's 8 elements all exist, or none)
      q.d[f] = __builtin_amdgcn_raw_buffer_load_b128(
          rd, lg * 8 < left ? (f * 16 + lr) * dy_ld + (k0 + lg * 8) * 2 : kOutside, 0, 0);
  };
  f32x4 acc[MF][kLaneColumns];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int j = 0; j < kLaneColumns; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Step& q) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      u32x4 v[8];  // of each row the 8 columns
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(u32x4, mx_bf16x8(q.c[i][c], mx_scale_f32(q.s[i])));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = __builtin_amdgcn_perm(v[2 * i + 1][j / 2], v[2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int f = 0; f < MF; ++f)
          acc[f][c * 8 + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, q.d[f]), acc[f][c * 8 + j], 0, 0, 0);
      }
    }
  };
  Step q;
  load(q, wave);
  for (int st = wave; st < steps; st += NW) {
    multiply(q);
    load(q, st + NW);
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    if (f) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kLaneColumns; j += 4)
        *reinterpret_cast<f32x4*>(&sums[wave][lr][(lg * 4 + i) * kLaneColumns + j]) =
            f32x4{acc[f][j][i], acc[f][j + 1][i], acc[f][j + 2][i], acc[f][j + 3][i]};
    __syncthreads();
    // a thread takes 4 columns of a row at a time
#pragma unroll
    for (int i = threadIdx.x; i < 16 * TN / 4; i += 64 * NW) {
      const int r = i / (TN / 4), c = i % (TN / 4) * 4;
      if (f * 16 + r >= t.mlim || c >= t.clim) continue;
      f32x4 v = *reinterpret_cast<const f32x4*>(&sums[0][r][c]);
#pragma unroll
      for (int w = 1; w < NW; ++w) v += *reinterpret_cast<const f32x4*>(&sums[w][r][c]);
      const size_t at = (row0 + f * 16 + r) * p.K + t.c0 + c;
      if (p.out_bf16) *reinterpret_cast<u32x2*>(static_cast<__bf16*>(p.out) + at) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      else *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at) = v;
    }
  }
}

template <int MF, int NC, int NW>
hipError_t launch_stream(const GroupedGemmArgs& g, const MxDgradArgs& p, hipStream_t stream) {
  const long long grid = xcd_grid(tile_items(kDgrad, g, 16 * MF, 128 * NC));
  mx_dgrad_stream_kernel<MF, NC, NW><<<(unsigned)grid, 64 * NW, 0, stream>>>(p);
  return hipGetLastError();
}

// The shapes of mxfp4_shapes.h, in their order.
hipError_t launch_shape(int i, const GroupedGemmArgs& g, const MxDgradArgs& p, hipStream_t s) {
  switch (i) {
    case 0: return launch_stream<1, 1, 8>(g, p, s);
    case 1: return launch_stream<1, 2, 4>(g, p, s);
    case 2: return launch_stream<1, 2, 8>(g, p, s);
    case 3: return launch_stream<2, 1, 8>(g, p, s);
    case 4: return launch_stream<2, 2, 8>(g, p, s);
    case 5: return launch_tiles<64, 32, 2, 4, 128, false>(g, p, s);
    case 6: return launch_tiles<64, 64, 2, 2, 64, false>(g, p, s);
    default: return launch_tiles<128, 64, 2, 4, 64, true>(g, p, s);
  }
}

}  // namespace

// (the largest tiles: the choice passes over those that do not fit)
bool mx_dgrad_fits(const MxGemmArgs& a) { return shape_fits(kDgrad, a.g, kDgradShapes[kDgradShapeCount - 1].cost); }

hipError_t launch_mx_dgrad(const MxGemmArgs& a, hipStream_t stream) {
  const GroupedGemmArgs& g = a.g;
  const MxDgradArgs p{{g.a, g.b, g.a2, g.b2, g.out, g.offsets, g.rows, g.E, g.N, g.K, g.out_bf16 ? 1 : 0, 0,
                       stream_rows(g, kDgrad)},
                      a.b_scales, a.b2_scales};
  DeviceInfo dev;
  const hipError_t e = device_info(&dev);
  if (e != hipSuccess) return e;
  return launch_shape(pick_dgrad(g, dev.num_cus), g, p, stream);
}

}  // namespace moe
