// How the products of few rows (gemm_few_rows.hip) share their columns and K among waves.
// Plain host C++, as gemm_shape.hpp.
#pragma once

#include <stdint.h>

namespace fp8mi {

constexpr int64_t kFewRows = 16;  // rows that the kernel takes at most: the matrix instruction's
constexpr int kWavesFew = 8;      // a workgroup's

// Workgroups of a product of N columns, `split` waves a tile of 16.
inline int64_t few_groups(int64_t N, int split) {
  const int64_t tiles = (N + 15) / 16, tiles_wg = kWavesFew / split;
  return (tiles + tiles_wg - 1) / tiles_wg;
}

// Waves that share a tile's K: as many as make `waves` (about 8 a compute unit), in no more than `most` workgroups.
inline int few_split(int64_t N, int64_t waves, int64_t most = INT64_MAX) {
  const int64_t tiles = (N + 15) / 16;
  int split = 1;
  while (split < kWavesFew && tiles * split < waves && few_groups(N, 2 * split) <= most) split *= 2;
  return split;
}

}  // namespace fp8mi
