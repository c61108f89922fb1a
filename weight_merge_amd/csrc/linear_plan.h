// Which kernel, tile and split a linear or gated product or its backward pass takes, and its
// workspace: rules on sizes and types alone, host code without the HIP headers.
#pragma once

#include <stdint.h>

#include "adafuse.h"

namespace ada {
namespace {

// ---- few rows ------------------------------------------------------------------------
// Sizes that take the few-rows kernel, timed against the tiles at 2400 pairs of columns and depths
// (1024 to 32768 columns, 1 to 64 KB of depth), 2 to 48 rows, both types, gated and not; the rule
// is within 4% of the faster of the two in the mean of every kind, within 15% at nine of ten.
//   to 16 rows: it is ahead throughout, or level (8 x 4096 x 4096: 7.9 against 13.4 us, 16 x 28672
//     x 2048: 25.2 and 25.1)
//   17 to 32 rows: x's second block leaves room for one workgroup on a CU.  In fp32, whose matrix
//     instructions bind the tiles, it is still ahead (32 x 11008 x 4096: 48.5 against 78.9).  In
//     bf16 while the workgroups are one round (24 x 4096 x 4096: 9.7 against 13.7), or two with
//     rows short enough for two waves each (32 x 8192 x 1024: 6.8 against 9.1; gated 30 x 8192 x
//     4096: 24.7 against 36.9); not where there are more (32 x 16384 x 4096: 35.9 against 26.8;
//     gated 32 x 11008 x 1024: 15.1 against 13.6) or two of longer rows (32 x 5120 x 5560: 32
//     against 22)
//   33 to 48 rows: short rows in one round or two (48 x 4096 x 4096: 12.0 against 14.4; 48 x 8192 x
//     1024: 7.6 against 9.4; but 48 x 8192 x 8192: 40 against 33), longer ones for a gated pair
//     whose round nearly fills the CUs (48 x 4096 x 8192: 30 against 34, but 48 x 2048 x 7168: 23
//     against 20), fp32 pairs always (48 x 11008 x 4096: 101 against 130)
inline bool few_rows_sizes(int64_t rows, int64_t cols, int64_t depth, bool gated, int esz) {
  if (rows <= 16 || rows > 48) return rows <= 16;
  if (esz == 4 && (gated || rows <= 32)) return true;
  const int64_t bytes = depth * esz;
  if (rows <= 32) return cols <= 4096 || (cols <= 8192 && (gated ? bytes < 16384 : bytes <= 8192));
  return (cols <= 8192 && bytes <= 8192) || (gated && cols > 2048 && cols <= 4096 && bytes <= 16384);
}

// Into how many parts the contraction is split over workgroups: where the columns leave most CUs
// idle and k is long (14 x 216 x 13456: 12.0 against 19.7 us; fp32 12 x 1016 x 28552: 33 against
// 79 us), at least 32 windows a part.
inline int few_rows_splits(int64_t cols, int64_t depth, int esz) {
  const int64_t blocks = (cols + 15) / 16, windows = (depth * esz + 255) / 256;
  int64_t splits = 256 / blocks;
  if (splits > windows / 32) splits = windows / 32;
  return static_cast<int>(splits < 2 ? 1 : splits > 16 ? 16 : splits);
}

// Two waves a workgroup, and several workgroups on a CU, where there are more of them than CUs
// and k is short; else as many waves as have room for their rings (16 x 4096 x 4096: 9.4 against
// 10.9 us).  To 16 rows, and for gated pairs, two waves are ahead below 16 KB of depth (8 x 11008 x
// 1024: 6.6 against 10.2 us, 8 x 14176 x 6144: 33 against 37, gated 16 x 28672 x 2048: 40 against
// 49) and behind from there on (8 x 8192 x 8192: 29 against 26, gated 16 x 8192 x 8192: 49 against
// 45); with x's second block beside one W to 8 KB (32 x 8192 x 1024: 6.8 against 8.6, fp32 24 x
// 8192 x 8192: 73 against 56).
inline bool few_rows_two_waves(int64_t cols, int64_t depth, bool gated, int blocks_of_rows, int esz) {
  return cols > 256 * 16 && (blocks_of_rows > 1 && !gated ? depth * esz <= 8192 : depth * esz < 16384);
}

// ---- tiles ---------------------------------------------------------------------------
// The tiles, and what a step and a workgroup's start and end cost on a CU of its own, in us
// (bf16 step, fp32 step, rest), beside 4 us for a launch: fitted to 19 shapes from 24 x 4096 x
// 11008 to 4096 x 4096 x 4096 timed with every tile and split.  At 30 other shapes, drawn from 92
// to 3508 rows of either type, gated and not, the choice is within 4% of the fastest tile and
// split 23 times, within 11% 29 times, and 18% behind once (fp32, 670 x 2024 x 1816).
constexpr int kTiles = 6;
constexpr int kTileRows[kTiles] = {256, 256, 128, 128, 64, 64};
constexpr int kTileCols[kTiles] = {256, 128, 256, 128, 128, 64};
constexpr float kStep16[kTiles] = {1.45f, 0.85f, 0.85f, 0.50f, 0.37f, 0.27f};
constexpr float kStep32[kTiles] = {7.5f, 3.9f, 3.9f, 2.05f, 1.1f, 0.65f};
constexpr float kRest[kTiles] = {17.f, 9.f, 9.f, 6.f, 4.f, 2.5f};

// Which tile, and into how many parts a contraction is split: the least sum of rounds (256
// workgroups at a time, one per CU) times the steps and the rest of each, and for a split the
// join: a launch, and its parts written and read at about 4 TB/s.
struct Plan {
  int tile;
  int splits;
  float us;
};

struct Product {
  int64_t rows, cols, depth;  // cols: of all products together
  int esz;
  int64_t steps() const { return (depth * esz + 127) / 128; }
  int64_t tiles(int t) const {
    return ((rows + kTileRows[t] - 1) / kTileRows[t]) * ((cols + kTileCols[t] - 1) / kTileCols[t]);
  }
  float one(int t, int splits) const {  // a workgroup's time
    return static_cast<float>((steps() + splits - 1) / splits) * (esz == 2 ? kStep16[t] : kStep32[t]) + kRest[t];
  }
  float join(int splits) const { return splits > 1 ? static_cast<float>(splits * cols * rows) * 2e-6f : 0.f; }
  bool may_split(int t, int splits) const {
    return splits == 1 || (steps() / splits >= 3 && tiles(t) * splits <= 1024);
  }
};
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
constexpr float kLaunch = 4.f;

// When the last of n workgroups of `longer` us and then m of `shorter` ends, each on the CU that
// is free first.
inline float makespan(int64_t n, float longer, int64_t m, float shorter) {
  constexpr int64_t kCus = 256;
  if (m == 0) return static_cast<float>((n + kCus - 1) / kCus) * longer;
  const int64_t late = n % kCus, early = kCus - late;  // CUs that take one more of the long ones
  const float load[2] = {static_cast<float>(n / kCus) * longer, static_cast<float>(n / kCus + 1) * longer};
  auto room = [&](float end) {
    auto in = [&](float from) { return end > from ? static_cast<int64_t>((end - from) / shorter + 1e-3f) : 0; };
    return early * in(load[0]) + late * in(load[1]);
  };
  const float least = (static_cast<float>(n) * longer + static_cast<float>(m) * shorter) / kCus;
  float best = -1.f;
  for (float from : load) {
    float end = from + shorter * static_cast<float>(least > from ? static_cast<int64_t>((least - from) / shorter) : 1);
    while (room(end) < m) end += shorter;
    if (best < 0.f || end < best) best = end;
  }
  return late > 0 && best < load[1] ? load[1] : best;
}

inline Plan plan_product(const Product& p) {
  Plan best{0, 1, -1.f};
  for (int t = 0; t < kTiles; ++t)
    for (int splits : kSplits) {
      if (!p.may_split(t, splits)) break;
      const float us = makespan(p.tiles(t) * splits, p.one(t, splits), 0, 0.f) + p.join(splits) +
                       (splits > 1 ? 2 : 1) * kLaunch;
      if (best.us < 0.f || us < best.us) best = {t, splits, us};
    }
  return best;
}

// Two products: one after the other with a tile each, or side by side in one grid with one
// tile, which fills the CUs that the other's last round leaves idle.
struct PairPlan {
  bool together;
  Plan plan[2];
};

inline PairPlan plan_pair(const Product& p, const Product& q) {
  PairPlan best{false, {plan_product(p), plan_product(q)}};
  float least = best.plan[0].us + best.plan[1].us;
  for (int t = 0; t < kTiles; ++t)
    for (int sp : kSplits) {
      if (!p.may_split(t, sp)) break;
      for (int sq : kSplits) {
        if (!q.may_split(t, sq)) break;
        const int64_t np = p.tiles(t) * sp, nq = q.tiles(t) * sq;
        const float op = p.one(t, sp), oq = q.one(t, sq);
        float us = op >= oq ? makespan(np, op, nq, oq) : makespan(nq, oq, np, op);
        us += p.join(sp) + q.join(sq) + (sp > 1 || sq > 1 ? 2 : 1) * kLaunch;
        if (us < least) {
          least = us;
          best = {true, {{t, sp, op}, {t, sq, oq}}};
        }
      }
    }
  return best;
}

inline int64_t part_bytes(const Product& p, int splits) { return splits > 1 ? splits * p.rows * p.cols * 4 : 0; }

// A forward product's plan.  Few rows have a kernel of their own; the tile is for those with
// rows too far apart for it.
inline Plan plan_forward(int64_t rows, int64_t cols, int64_t depth, int gated, int esz) {
  Plan p = plan_product({rows, gated ? 2 * cols : cols, depth, esz});
  if (rows == 1 || few_rows_sizes(rows, cols, depth, gated, esz))
    p = {kTiles - 1, rows == 1 ? 1 : few_rows_splits(cols, depth, esz), 0.f};
  return p;
}

// ---- backward passes -------------------------------------------------------------------
// Sizes that take the few-rows gradients.  Small matrices are ahead on the tiles (both gradients, tiles against this:
// bf16 32 x 1024 x 1024 10.9 and 11.2 us, 32 x 512 x 8192 17.8 and 14.0; fp32 32 x 1024 x 1024 13.5
// and 14.7, 32 x 4096 x 512 19.5 and 15.0).  Two blocks of rows leave one wave on a SIMD, which
// pays for large ones in bf16 (64 x 4096 x 4096 37.2 and 37.5, 64 x 11008 x 4096 84 and 58), and
// not in fp32, where the matrix pipes bind (64 x 4096 x 4096 69 and 69, 48 x 4096 x 512 21.6 and 21.9).
// At 720 more pairs of columns and depths (1 MB to 1 GB of weights, gated and not) it is within 2% of
// the faster of the two in the mean of every kind, within 10% at nine of ten.
inline bool few_rows_grad(int64_t rows, int64_t weight_bytes, int esz) {
  return rows <= 32 ? weight_bytes > (int64_t(4) << 20)
                    : rows <= 64 && esz == 2 && weight_bytes > (int64_t(32) << 20);
}

// Into how many parts dx's contraction is split over workgroups: one workgroup per CU, and four
// steps or more a wave.
inline int few_rows_dx_splits(int64_t cols, int64_t depth, int esz) {
  const int64_t strips = (cols * esz + 511) / 512, steps = (depth * esz + 31) / 32;
  int64_t splits = 256 / strips;
  if (splits > steps / 16) splits = steps / 16;
  return static_cast<int>(splits < 2 ? 1 : splits > 128 ? 128 : splits);
}

constexpr int kSide = 64;  // dz is computed in tiles of 64 x 64

// Workspace of a backward pass (byte offsets): dz [rows][parts d_out], column sums for dbias,
// parts of split contractions.
struct GradPlan {
  int64_t dz, sums, part[2], total;
  bool few;
  PairPlan pair;  // dx, dW: the same whichever of the two is asked for, and so are their sums
};

inline GradPlan plan_grad(int64_t rows, int64_t n, int64_t k, int act, int gated, int esz) {
  GradPlan g{};
  const int64_t parts = gated ? 2 : 1;
  auto take = [&](int64_t bytes) {
    const int64_t at = g.total;
    g.total += (bytes + 255) / 256 * 256;
    return at;
  };
  g.dz = take(gated || act != ADA_ACT_NONE ? rows * parts * n * esz : 0);
  g.sums = take((rows + kSide - 1) / kSide * parts * n * 4);
  const Product dx{rows, k, parts * n, esz}, dw{parts * n, k, rows, esz};
  g.few = few_rows_grad(rows, parts * n * k * esz, esz);
  if (g.few)
    g.pair = {true, {{0, few_rows_dx_splits(k, parts * n, esz), 1.f}, {0, 1, 0.f}}};
  else
    g.pair = plan_pair(dx, dw);
  g.part[0] = take(part_bytes(dx, g.pair.plan[0].splits));
  g.part[1] = take(part_bytes(dw, g.pair.plan[1].splits));
  return g;
}

}  // namespace
}  // namespace ada
