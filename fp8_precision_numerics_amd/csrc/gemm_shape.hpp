// Tile shape and split of K of the dense GEMMs, by an estimate of their time.  Plain
// host C++, so that a test can ask for the choice without a device.
#pragma once

#include <cstddef>
#include <cstdint>

namespace fp8mi {

constexpr int kShapeStep = 128;  // K bytes of a main-loop step

// The larger tiles need fewer operand bytes a product; the smaller ones fill the chip
// with fewer rows and columns, and a split of K fills it where even those are few (only
// with a workspace for the parts).  64 x 128 tiles with three stages of loads (two
// workgroups a compute unit instead of three) take a shorter step where few of them
// share a compute unit.  The choice is the least of an estimate in microseconds, from
// step times (a K step of 128) measured on MI355X:
//
//   L = the most workgroups that any compute unit gets, S = K steps of a part
//   start + S max(alone, L each odd) + (split: second launch + traffic of the partials)
//
// `alone` is the step of a lone workgroup (latency-bound), `each` the step's share of a
// busy compute unit, `odd` its growth where K is no multiple of 128 and the 128 bytes
// of a row and step lie in two cache lines (8192 x 4096 on the FP8 cores: 108 us at
// K = 4096, 133 at 4112).  The constants are a least-squares fit to 100 products of
// random and of round sizes; over them the choice is 4 % slower than the best shape
// and split of each, 30 % at worst.  Measured for some M x N x K (exact mode, cold weights, us; 256, 128, 64
// and 64t stand for the shapes, t for three stages, /s for the best split tried, * for the choice
// with a workspace of 64 MiB):
//   8192 x 4096 x 16384   256*: 718   128: 777    64: 876     64t: 963
//   1003 x 16384 x 4096   256*: 99    128: 109    64: 122     64t: 138
//   2048 x 4096 x 4096    256/2: 75   128*: 56    64: 66      64t: 70
//   500 x 4096 x 16384    256/6: 73   128/4*: 65  64/3: 68    64t/2: 70
//   64 x 4096 x 16384                             64/13: 24   64t/6*: 23
//   24 x 4096 x 16384                             64/13*: 21  64t/6: 21
struct TileChoice {
  int shape;  // 0: 256 x 256, 1: 128 x 128, 2: 64 x 128, 3: 64 x 128 in three stages
  int split;
  double us;  // the estimate
};

struct TileCost {
  int bm, bn;
  double start, alone, each, odd;
};
inline const TileCost* tile_costs(bool fp8_cores) {
  static constexpr TileCost kExact[4] = {{256, 256, 10.5, 2.13, 2.22, 1.04},
                                         {128, 128, 6.9, 0.86, 0.72, 1.11},
                                         {64, 128, 6.4, 0.60, 0.43, 1.20},
                                         {64, 128, 6.6, 0.48, 0.49, 1.12}};
  static constexpr TileCost kFp8[4] = {{256, 256, 9.0, 1.00, 1.27, 1.23},
                                       {128, 128, 6.3, 0.77, 0.50, 1.23},
                                       {64, 128, 5.7, 0.60, 0.34, 1.32},
                                       {64, 128, 5.9, 0.39, 0.35, 1.27}};
  return fp8_cores ? kFp8 : kExact;
}

// The estimate for one shape and split.
inline double tile_time(const TileCost& c, int split, int64_t M, int64_t brows, int64_t K, int64_t cus) {
  const int64_t steps = (K + kShapeStep - 1) / kShapeStep;
  const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((brows + c.bn - 1) / c.bn);
  const double traffic = (double)split * M * brows * 4.0;
  const int64_t load = (tiles * split + cus - 1) / cus;
  const double busy = load * c.each * (K % kShapeStep ? c.odd : 1.0);
  const double step = c.alone > busy ? c.alone : busy;
  return c.start + (double)((steps + split - 1) / split) * step + (split > 1 ? 2.0 + 2.0 * traffic / 5.2e6 : 0.0);
}

// `brows`: rows of B; `cus`: compute units of the device.
inline TileChoice choose_tile(int64_t M, int64_t brows, int64_t K, bool fp8_cores, size_t workspace_bytes,
                              int64_t cus) {
  const TileCost* costs = tile_costs(fp8_cores);
  const int64_t steps = (K + kShapeStep - 1) / kShapeStep;
  TileChoice best{2, 1, 1e300};
  for (int i = 0; i < 4; ++i) {
    const TileCost& c = costs[i];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((brows + c.bn - 1) / c.bn);
    for (int split = 1; split <= 32 && split <= steps; split = split < 4 ? split + 1 : split + split / 2) {
      const double traffic = (double)split * M * brows * 4.0;
      if (split > 1 && (traffic > (double)workspace_bytes || tiles * split > 4 * cus)) break;
      const double t = tile_time(c, split, M, brows, K, cus);
      if (t < best.us) best = TileChoice{i, split, t};
    }
  }
  return best;
}

}  // namespace fp8mi
