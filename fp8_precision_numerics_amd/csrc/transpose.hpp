// A 128 x 128 tile of codes staged row-major in LDS (row pitch 132 B), written out
// transposed: each lane takes 4 columns x 16 rows: 16 LDS words, a 4x4 byte
// transpose per 4 rows with V_PERM_B32, and four 16-B stores into 4 rows of the
// transpose (eight lanes cover 128 contiguous bytes of one row).
#pragma once

#include "device_common.hpp"

namespace fp8mi {

constexpr int kTile = 128;
constexpr int kPitch = 132;

__device__ __forceinline__ void transpose4x4(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t& c0,
                                             uint32_t& c1, uint32_t& c2, uint32_t& c3) {
  // w_r holds columns 0..3 of row r (byte k = column k); c_k gets rows 0..3 of column k.
  const uint32_t t0 = __builtin_amdgcn_perm(w1, w0, 0x05010400u);  // w0.b0 w1.b0 w0.b1 w1.b1
  const uint32_t t1 = __builtin_amdgcn_perm(w3, w2, 0x05010400u);  // w2.b0 w3.b0 w2.b1 w3.b1
  const uint32_t t2 = __builtin_amdgcn_perm(w1, w0, 0x07030602u);  // w0.b2 w1.b2 w0.b3 w1.b3
  const uint32_t t3 = __builtin_amdgcn_perm(w3, w2, 0x07030602u);  // w2.b2 w3.b2 w2.b3 w3.b3
  c0 = __builtin_amdgcn_perm(t1, t0, 0x05040100u);
  c1 = __builtin_amdgcn_perm(t1, t0, 0x07060302u);
  c2 = __builtin_amdgcn_perm(t3, t2, 0x05040100u);
  c3 = __builtin_amdgcn_perm(t3, t2, 0x07060302u);
}

// The staged tile's columns col0.. and rows row0.. into q_t [cols x rows], by 256
// threads (thread t); rows and cols are multiples of 16.
__device__ __forceinline__ void transposed_store(const uint8_t* tile, uint8_t* q_t, int64_t rows, int64_t cols,
                                                 int64_t row0, int64_t col0, int t) {
  const int rg = t & 7, cq = t >> 3;
  const int64_t c = col0 + cq * 4, r = row0 + rg * 16;
  if (c < cols && r < rows) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = *reinterpret_cast<const uint32_t*>(tile + (rg * 16 + j) * kPitch + cq * 4);
    uint32_t o[4][4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
      transpose4x4(w[4 * b], w[4 * b + 1], w[4 * b + 2], w[4 * b + 3], o[b][0], o[b][1], o[b][2], o[b][3]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4*>(q_t + (c + k) * rows + r) = make_uint4(o[0][k], o[1][k], o[2][k], o[3][k]);
  }
}

}  // namespace fp8mi
