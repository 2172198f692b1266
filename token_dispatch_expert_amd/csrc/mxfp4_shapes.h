// Which kernel of the MXFP4 products a call takes. Host code alone.
#pragma once

#include "mxfp4_internal.h"
#include "product_tiles.h"

namespace moe {

// What a launch may take, and the time of 256 contraction elements (us): `alone` for at most one tile of TM x TN (of gate and up: TN
// columns of h) to a CU, `full` for `fit` tiles to each CU, when there are many. `start`: what a tile takes before and after
// them.
struct Shape {
  TileCost cost;
  double start;
  bool groups;  // a wave holds groups of 32 columns of h, as h in MXFP4 needs
};

// (at most 512 threads a workgroup)
inline bool shape_fits(GroupedProduct kind, const GroupedGemmArgs& g, const TileCost& c) {
  return xcd_grid(tile_items(kind, g, c.TM, c.TN)) <= kMaxWorkgroups / 2;
}

// The shape to take, from the sizes alone (the host does not know the offsets): the one that a model of the rounds over the CUs finds
// fastest, but no faster than the weights' stream. weights: of an expert; blocks: of 256 contraction elements; groups: only
// shapes that have them; whole: tiles count in whole rounds over the CUs up to two, a tenth more of them than expected where experts'
// rows may fill more than one (two input gradients of 8 experts of 2048 x 4096 in tiles of 32 x 256: 27 us for half a tile to a CU,
// 50 for 1.25, 73 for 2.25).
template <int COUNT>
inline int pick_shape(GroupedProduct kind, const GroupedGemmArgs& g, const Shape (&shapes)[COUNT], double weights, double blocks,
                      bool groups, bool whole, int cus) {
  const double active = g.E < g.rows ? g.E : g.rows;
  const double stream = active * weights * (17. / 32) / 5.5e6;  // us
  int best = 0;
  double least = -1;
  for (int i = 0; i < COUNT; ++i) {
    const Shape& s = shapes[i];
    if ((groups && !s.groups) || !shape_fits(kind, g, s.cost)) continue;
    const TileCost& c = s.cost;
    // Large tiles go over the CUs in rounds. Of the small ones several are on a CU at a time, and a new one starts as one ends; with a
    // row or two each, `fit` of them to a CU take hardly longer than one.
    const double tiles = expected_tiles(kind, g, c.TM, c.TN);
    double work;
    if (whole) {
      const double more = g.E > 1 && g.rows * 4. > c.TM * active ? 1.1 : 1, rounds = tiles * more / cus / c.fit;
      work = s.start + std::fmax(c.alone, c.full * (rounds <= 2 ? std::ceil(rounds) : rounds)) * blocks;
    } else if (c.TM >= 128) {
      work = step_time(kind, g, TileCost{c.TM, c.TN, c.fit, c.alone * blocks + s.start, c.full * blocks + s.start}, cus);
    } else if (c.fit > 1 && g.rows < 4 * active && tiles > cus && tiles <= (double)c.fit * cus) {
      work = s.start + 1.2 * c.alone * blocks;
    } else {
      work = s.start + std::fmax(c.alone, c.full * tiles / cus) * blocks;
    }
    const double time = std::fmax(work, stream) + 0.1 * work;  // of those that the stream bounds the one with the least work
    if (least < 0 || time < least) {
      least = time;
      best = i;
    }
  }
  return best;
}

// From products of 1 to 32,768 rows over 1 to 128 experts, of K = 4096, 2048 and 800. X4: rows in MXFP4; PAIR: gate and up. The
// launches (mxfp4_gemm.hip) are in the same order.
template <bool X4, bool PAIR>
struct GemmShapes;
template <>
struct GemmShapes<false, false> {
  static constexpr Shape all[] = {
      {{16, 32, 2, 0.36, 0.37}, 3.3, false},   // stream: 2 fragments, 4 waves
      {{16, 64, 2, 0.49, 0.50}, 3.4, false},   // stream: 4, 4
      {{16, 64, 1, 0.40, 0.34}, 3.6, false},   // rows: 1 x 1 fragments, 4 waves, 4 blocks
      {{16, 256, 1, 1.09, 1.12}, 3.8, false},  // rows: 1 x 2, 8, 3
      {{32, 64, 1, 0.47, 0.50}, 4, false},   // rows: 2 x 1, 4, 4
      {{32, 128, 1, 0.69, 0.76}, 4, false},  // rows: 2 x 1, 8, 3
      {{32, 256, 1, 1.27, 1.30}, 4.5, false},  // rows: 2 x 4, 4, 3
      {{64, 256, 1, 2.10, 2.00}, 4.5, false},  // rows: 4 x 2, 8, 2
      {{256, 256, 1, 5.20, 6.70}, 6, false}};
};
template <>
struct GemmShapes<false, true> {
  static constexpr Shape all[] = {
      {{16, 16, 2, 0.36, 0.37}, 3.3, false},
      {{16, 32, 2, 0.49, 0.50}, 3.4, true},
      {{16, 64, 1, 0.57, 0.59}, 3.8, false},
      {{16, 128, 1, 1.11, 1.14}, 4.5, true},
      {{32, 64, 1, 0.85, 0.70}, 4, false},
      {{32, 128, 1, 1.30, 1.31}, 5, true},
      {{64, 128, 1, 2.10, 1.91}, 5, false},
      {{256, 128, 1, 5.70, 6.80}, 12, true}};
};
template <>
struct GemmShapes<true, false> {
  static constexpr Shape all[] = {
      {{16, 32, 2, 0.17, 0.20}, 3.3, false},
      {{16, 64, 2, 0.31, 0.34}, 3.4, false},
      {{32, 64, 1, 0.36, 0.31}, 3.6, false},
      {{32, 128, 1, 0.54, 0.57}, 3.8, false},
      {{128, 128, 2, 0.77, 1.54}, 4, false},
      {{256, 256, 1, 1.70, 2.65}, 6, false}};
};
template <>
struct GemmShapes<true, true> {
  static constexpr Shape all[] = {
      {{16, 16, 2, 0.18, 0.21}, 3.3, false},
      {{16, 32, 2, 0.31, 0.33}, 3.4, true},
      {{32, 32, 1, 0.34, 0.31}, 3.6, false},
      {{32, 64, 1, 0.54, 0.56}, 3.8, false},
      {{32, 128, 1, 1.08, 1.09}, 5, true},
      {{128, 64, 2, 0.97, 1.70}, 10, true},
      {{256, 128, 1, 2.15, 2.90}, 11, true}};
};
template <bool X4, bool PAIR>
inline int pick_gemm(const MxGemmArgs& a, int cus) {
  const GroupedGemmArgs& g = a.g;
  return pick_shape(kForward, g, GemmShapes<X4, PAIR>::all, (PAIR ? 2. : 1.) * g.N * g.K, (g.K + 255) / 256, a.out_scales != nullptr,
                    false, cus);
}

// From products of 1 to 32,768 rows over 1 to 64 experts of 2048 x 4096 and 4096 x 1536, one and two input gradients.
// The launches (mxfp4_dgrad.hip) are in the same order.
constexpr Shape kDgradShapes[] = {
    {{16, 128, 1, 0.75, 0.84}, 6, false},  // stream: 16 rows, 1 dword of 8 columns, 8 waves
    {{16, 256, 1, 1.75, 1.42}, 6, false},  // 2, 4
    {{16, 256, 1, 1.20, 1.56}, 6, false},  // 2, 8
    {{32, 128, 1, 0.86, 1.10}, 6, false},  // 32 rows, 1, 8
    {{32, 256, 1, 1.35, 1.75}, 6, false},  // 2, 8
    {{128, 128, 1, 1.90, 2.65}, 5, false}, {{128, 128, 2, 2.90, 5.00}, 5, false}, {{256, 256, 1, 5.40, 5.90}, 5, false}};
constexpr int kDgradShapeCount = sizeof(kDgradShapes) / sizeof(Shape);
inline int pick_dgrad(const GroupedGemmArgs& g, int cus) {
  const double pairs = g.b2 ? 2 : 1;
  return pick_shape(kDgrad, g, kDgradShapes, pairs * g.N * g.K, pairs * g.N / 256, false, true, cus);
}

}  // namespace moe
