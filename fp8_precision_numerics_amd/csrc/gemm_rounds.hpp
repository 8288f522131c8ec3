// Products cut where their tiles leave most of the last round of compute units idle.
// Plain host C++, as gemm_shape.hpp.
#pragma once

#include "gemm_shape.hpp"

namespace fp8mi {

// A product whose 256 x 256 tiles would leave the last round of the compute units nearly empty goes in two
// launches where the estimate prefers it: as many tiles as whole rounds hold, and the rest on the tiles that suit it.  `fixed` and `free`
// are its two sides, `free` (rows or columns) the one that may be cut.
struct Rounds {
  int64_t first;  // rows or columns of the first launch (all of them: no second one)
  double us;      // estimate of both
};
// Measured on MI355X: the loss of 1003 x 50021 x 4096, exact (784 tiles on 256 compute units, so 768 and the
// rest) 308 us against 349.
inline Rounds plan_rounds(int64_t fixed, int64_t free, int64_t K, bool fp8_cores, size_t workspace_bytes, int64_t cus) {
  const TileChoice whole = choose_tile(fixed, free, K, fp8_cores, workspace_bytes, cus);
  const TileCost& c = tile_costs(fp8_cores)[0];
  const int64_t across = (fixed + 255) / 256, tiles = across * ((free + 255) / 256);
  const int64_t first = tiles / cus * cus / across * 256;
  if (whole.split == 1 && first > 0 && first < free) {
    const double t = tile_time(c, 1, fixed, first, K, cus) + choose_tile(fixed, free - first, K, fp8_cores, workspace_bytes, cus).us;
    if (t < 0.97 * whole.us) return Rounds{first, t};
  }
  return Rounds{free, whole.us};
}

}  // namespace fp8mi
