// Which kernel of the MXFP4 products a call takes.
#pragma once

#include "moe_internal.h"
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

}  // namespace moe
