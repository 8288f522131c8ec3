// Sum of a column of fp32 partial rows, in a fixed order: a workgroup takes 16
// columns, 64 lanes down the rows of each, then a tree in LDS.
#pragma once

#include "device_common.hpp"

namespace fp8mi {

constexpr int kSumLanes = 64;

// Column c of partials [count x pitch] (`valid`: it exists), for a workgroup of 16 * kSumLanes
// threads, all of which call it; threads of the same number mod 16 name the same column.
// The sum is threads 0 .. 15's.
__device__ __forceinline__ float column_sum(const float* __restrict__ partials, int count, int64_t pitch, int64_t c,
                                            bool valid) {
  __shared__ float buf[kSumLanes][17];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  float v = 0.0f;
  if (valid) {
    int r = ry;
    for (; r + 7 * kSumLanes < count; r += 8 * kSumLanes) {
      float p[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) p[u] = partials[(int64_t)(r + u * kSumLanes) * pitch + c];
      v += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    }
    for (; r < count; r += kSumLanes) v += partials[(int64_t)r * pitch + c];
  }
  buf[ry][cx] = v;
  __syncthreads();
#pragma unroll
  for (int half = kSumLanes / 2; half > 0; half >>= 1) {
    if (ry < half) buf[ry][cx] += buf[ry + half][cx];
    __syncthreads();
  }
  return buf[0][cx];
}

}  // namespace fp8mi
