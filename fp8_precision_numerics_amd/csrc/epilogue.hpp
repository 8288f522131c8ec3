// The epilogue of the feed-forward GEMMs, eight consecutive columns at a time.
//
//   fused   z = c + bias;   y = act(z) + residual
//   gated   y = act(c_gate) * c_up
//   product y = c + add
//
// with c the fp32 GEMM result already times sinv_a * sinv_b.  z (gated: both
// projections) may be kept in bf16 for the gradient; it is rounded from the fp32
// value that the activation is taken of, so the forward does not see the
// rounding.  y leaves as fp32, bf16 or FP8 codes of fp32(y * out_scale), with the
// amax of the unscaled y and the saturation count.  Everything up to the last
// rounding is fp32.
#pragma once

#include "activation.hpp"
#include "stats.hpp"

namespace fp8mi {

// Output kinds besides kF32 and kBF16 (the values gemm_kernel.hpp's kOutE4M3 and
// kOutE5M2 have).
enum : int { kYE4M3 = 2, kYE5M2 = 3 };

struct EpiArgs {
  void* y;                  // [M x N]
  uint16_t* z;              // bf16 [M x N], gated [M x 2N] (gate, then up), or null
  const uint16_t* bias;     // bf16 [N], or null (not gated)
  const uint16_t* residual; // bf16 [M x N], or null (not gated)
  const float* out_scale;   // FP8 outputs
  uint32_t* amax_bits;      // may be null
  unsigned long long* sat;  // may be null
  int act;
  int out;                  // kF32, kBF16, kYE4M3, kYE5M2
  // Split products: `split` workgroups share a tile's K, and each writes its fp32
  // sums (not yet scaled) to partials [split x M x N] (gated [split x M x 2N]),
  // which epilogue_partials_kernel adds up and finishes.  1: no split.
  float* partials;
  int split;
};

template <class T>
struct is_epilogue {
  static constexpr bool value = false;
};
// Epilogues that take the accumulators of a whole tile (gemm_kernel.hpp) specialise this.
template <class T>
struct is_tile_epilogue {
  static constexpr bool value = false;
};
// The epilogues as kernel arguments of their own types.
struct FusedEpi : EpiArgs {};
struct GatedEpi : EpiArgs {};
// A product whose A rows are padded: lda bytes apart, a multiple of 128, zeros from K on
// (K itself may be any number), added to the fp32 matrix `add` [M x N] (may be null, or y where y is fp32).
struct ProductEpi : EpiArgs {
  const float* add;
  int lda;
};
template <>
struct is_epilogue<ProductEpi> {
  static constexpr bool value = true;
};
template <>
struct is_epilogue<FusedEpi> {
  static constexpr bool value = true;
};
template <>
struct is_epilogue<GatedEpi> {
  static constexpr bool value = true;
};

__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[2 * k], f[2 * k + 1]}, v2bf));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = bf16_lo(w[k]);
    f[2 * k + 1] = bf16_hi(w[k]);
  }
}

// Streamed past the caches: no kernel of the library reads an output again before
// other data has passed.
__device__ __forceinline__ void store16_nt(void* p, const uint4& v) {
  typedef unsigned int vec4 __attribute__((ext_vector_type(4)));
  vec4 r;
  r[0] = v.x;
  r[1] = v.y;
  r[2] = v.z;
  r[3] = v.w;
  __builtin_nontemporal_store(r, reinterpret_cast<vec4*>(p));
}

// Row m, columns n .. n + 7 (`left` of them inside the matrix).  `c` holds the
// GEMM result (gated: of the gate; `up` of the up projection) and is overwritten.
// `vec`: N is a multiple of 8, so a chunk lies inside the matrix or outside and
// every store is whole and aligned; `left` is then 8.  bias and res are the
// chunk's bias and residual values, zero where there are none.
template <bool GATED>
__device__ __forceinline__ void epilogue8(const EpiArgs& a, float* c, const float* up, const float* bias,
                                          const float* res, int64_t m, int64_t n, int64_t N, bool vec, int left,
                                          float scale, LaneStats& st) {
  if constexpr (!GATED) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] += bias[e];
  }
  if (a.z) {
    uint16_t* z = a.z + m * (GATED ? 2 * N : N) + n;
    const uint4 zc = pack_bf16x8(c);
    if (vec) {
      store16_nt(z, zc);
      if constexpr (GATED) store16_nt(z + N, pack_bf16x8(up));
    } else {
      const uint32_t w[4] = {zc.x, zc.y, zc.z, zc.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) z[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      if constexpr (GATED) {
        const uint4 zu = pack_bf16x8(up);
        const uint32_t wu[4] = {zu.x, zu.y, zu.z, zu.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) z[N + e] = (uint16_t)(wu[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
  if (a.act == kActGelu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = act_value<kActGelu>(c[e]);
  } else if (a.act == kActSilu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = act_value<kActSilu>(c[e]);
  } else if (a.act == kActRelu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = act_value<kActRelu>(c[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = GATED ? c[e] * up[e] : c[e] + res[e];
  if (a.out == kYE4M3 || a.out == kYE5M2) {
    if (!vec) {  // columns past the edge take no part in the statistics
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= left) c[e] = 0.0f;
    }
    const bool amax = a.amax_bits != nullptr, sat = a.sat != nullptr;
    const uint2 q = a.out == kYE4M3 ? encode8<kE4M3>(c, scale, amax, sat, st) : encode8<kE5M2>(c, scale, amax, sat, st);
    uint8_t* y = reinterpret_cast<uint8_t*>(a.y) + m * N + n;
    if (vec) {
      typedef unsigned int vec2 __attribute__((ext_vector_type(2)));
      vec2 r;
      r[0] = q.x;
      r[1] = q.y;
      __builtin_nontemporal_store(r, reinterpret_cast<vec2*>(y));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) y[e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    }
  } else if (a.out == kBF16) {
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + m * N + n;
    const uint4 v = pack_bf16x8(c);
    if (vec) {
      store16_nt(y, v);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) y[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* y = reinterpret_cast<float*>(a.y) + m * N + n;
    if (vec) {
      store16_nt(y, make_uint4(f2u(c[0]), f2u(c[1]), f2u(c[2]), f2u(c[3])));
      store16_nt(y + 4, make_uint4(f2u(c[4]), f2u(c[5]), f2u(c[6]), f2u(c[7])));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) y[e] = c[e];
    }
  }
}

// Eight bf16 values (bias, residual) of which `left` exist; zeros past them.
__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* p, bool vec, int left) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight fp32 values, likewise (to is zero on entry).
__device__ __forceinline__ void load_f32x8(const float* p, bool vec, int left, v4f* to) {
  if (vec) {
    to[0] = reinterpret_cast<const v4f*>(p)[0];
    to[1] = reinterpret_cast<const v4f*>(p)[1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) to[e >> 2][e & 3] = p[e];
  }
}

// A workgroup's amax and count into the outputs (cleared beforehand): the waves meet in
// `scratch` (LDS, two words a wave, free of other use), then one device-scope atomic a
// workgroup, skipped where it would change nothing (the outputs only grow).  One
// atomic a wave, contended by every wave that finishes its tile at the same time, cost
// 18 us (8192 x 4096 x 16384, FP8 cores: 397 against 379 us without the amax).
// All threads of the workgroup call it.
__device__ __forceinline__ void publish_epilogue_stats(const EpiArgs& a, const LaneStats& st, uint32_t* scratch) {
  const uint32_t m = wave_max_u32(st.amax()), cnt = wave_sum_u32(st.sat);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    scratch[2 * (threadIdx.x >> 6)] = m;
    scratch[2 * (threadIdx.x >> 6) + 1] = cnt;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t top = m;
    unsigned long long total = cnt;
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) {
      top = scratch[2 * w] > top ? scratch[2 * w] : top;
      total += scratch[2 * w + 1];
    }
    if (a.amax_bits && top > __hip_atomic_load(a.amax_bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
      atomicMax(a.amax_bits, top);
    if (a.sat && total) atomicAdd(a.sat, total);
  }
}

// Clears the outputs that a later kernel's publish_epilogue_stats adds to.
__device__ __forceinline__ void clear_epilogue_stats(const EpiArgs& a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (a.amax_bits) *a.amax_bits = 0u;
    if (a.sat) *a.sat = 0ull;
  }
}

// One staged pass of a tile: fp32 results in LDS rows of BN values (TileWriter's
// layout), taken out eight columns at a time.  Gated tiles hold PAIR gate columns,
// then the same PAIR columns of the up projection, and so on; an output tile is
// BN / 2 wide.  A thread keeps its columns over its rows, so it loads the bias
// once; its residual values are requested two rows ahead, the first two before the
// pass is staged.
// The row loop is rolled on purpose: unrolled, the kernel had 85 KiB of code, each
// instruction of the epilogue ran once a pass, and fetching them from memory cost
// about 40 us a launch (2048 x 4096 x 4096 exact on these tiles:
// 105 us against 84).  The next row's values are read from LDS while the present row is
// worked on (8192 x 2 x 16384 x 4096 exact: 1552 against 1474 us, a plain GEMM of that
// size beside them 1511 and 1451).
// PRODUCT: a ProductEpi's, which flush_product writes.
template <int BN, int NT, int PASS, int PAIR, bool PRODUCT, class TW>
struct EpiPass {
  static constexpr bool GATED = PAIR != 0;
  static constexpr int CPR = (GATED ? BN / 2 : BN) / 8;  // chunks per row
  static constexpr int SWEEP = NT / CPR;                 // rows per sweep
  static constexpr int ROWS = PASS / SWEEP;              // rows per thread
  static_assert(NT % CPR == 0 && PASS % SWEEP == 0, "whole sweeps");
  const EpiArgs& a;
  int64_t M, N, m0, n;
  int r0, left, col;
  bool vec;
  float bias[8];
  uint4 res[2];
  float scale;
  const float* add = nullptr;
  template <class ARGS>
  __device__ __forceinline__ EpiPass(const ARGS& a_, int64_t M_, int64_t N_, int64_t m_base, int64_t n_base, int t)
      : a(a_), M(M_), N(N_), m0(m_base) {
    const int c = t % CPR;
    r0 = t / CPR;
    n = n_base + c * 8;
    constexpr int P = GATED ? PAIR : 8;
    col = GATED ? (c * 8 / P) * 2 * P + c * 8 % P : c * 8;  // staged column of the first value
    left = n < N ? (int)(N - n < 8 ? N - n : 8) : 0;
    vec = (N & 7) == 0;
    uint4 b = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!GATED && !PRODUCT) {
      if (a.bias && left) b = load_bf16x8(a.bias + n, vec, left);
    }
    if constexpr (PRODUCT) add = a_.add;
    unpack_bf16x8(b, bias);
    res[0] = res[1] = make_uint4(0u, 0u, 0u, 0u);
    scale = (a.out == kYE4M3 || a.out == kYE5M2) ? *a.out_scale : 1.0f;
  }
  __device__ __forceinline__ void request(int pass_row, int i, uint4* to) const {
    if constexpr (!GATED && !PRODUCT) {
      const int64_t m = m0 + pass_row + r0 + i * SWEEP;
      if (a.residual && left && i < ROWS && m < M) *to = load_bf16x8(a.residual + m * N + n, vec, left);
    }
  }
  __device__ __forceinline__ void prefetch(int pass_row) {
    if (a.split > 1) return;
    request(pass_row, 0, &res[0]);
    request(pass_row, 1, &res[1]);
  }
  __device__ __forceinline__ void take(const TW& tw, int r, int from, float* to) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4f f = *reinterpret_cast<const v4f*>(tw.lds + tw.pos(r, (from + 4 * h) * 4));
#pragma unroll
      for (int e = 0; e < 4; ++e) to[4 * h + e] = f[e];
    }
  }
  // A split product's pass: the sums as they are, into this part's partials.
  __device__ __forceinline__ void flush_partials(const TW& tw, int pass_row, float* partials) const {
    if (!left) return;
    const int64_t ld = GATED ? 2 * N : N;
#pragma unroll 1
    for (int r = r0; r < PASS; r += SWEEP) {
      const int64_t m = m0 + pass_row + r;
      if (m >= M) break;
#pragma unroll
      for (int p = 0; p < (GATED ? 2 : 1); ++p) {
        float* dst = partials + m * ld + p * N + n;
        float v[8];
        take(tw, r, col + p * PAIR, v);
        if (vec) {
          reinterpret_cast<v4f*>(dst)[0] = (v4f){v[0], v[1], v[2], v[3]};
          reinterpret_cast<v4f*>(dst)[1] = (v4f){v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < left) dst[e] = v[e];
        }
      }
    }
  }
  // A product's pass: y = c + add and no more, N a multiple of 8, several rows at a time: tiles of one or two K steps spend
  // more time here than on the steps (dw of 50021 x 2048 from 219 rows, its logits before it: 155 us row by row as below, 137 so; of 32000 x 4096 from 64, 137 and 111).
  __device__ __forceinline__ void flush_product(const TW& tw, int pass_row) const {
    if (!left) return;
    constexpr int U = ROWS % 4 == 0 ? 4 : 1;
#pragma unroll 1
    for (int i = 0; i < ROWS; i += U) {
      const int64_t first = m0 + pass_row + r0 + i * SWEEP;
      if (first >= M) break;
      v4f v[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u][0] = v[u][1] = (v4f){0.f, 0.f, 0.f, 0.f};
        if (add && first + u * SWEEP < M) load_f32x8(add + (first + u * SWEEP) * N + n, true, 8, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float c[8];
        take(tw, r0 + (i + u) * SWEEP, col, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e >> 2][e & 3] = c[e] + v[u][e >> 2][e & 3];
      }
      if (a.out == kBF16) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float c[8] = {v[u][0][0], v[u][0][1], v[u][0][2], v[u][0][3], v[u][1][0], v[u][1][1], v[u][1][2], v[u][1][3]};
          if (first + u * SWEEP < M) store16_nt(reinterpret_cast<uint16_t*>(a.y) + (first + u * SWEEP) * N + n, pack_bf16x8(c));
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float* y = reinterpret_cast<float*>(a.y) + (first + u * SWEEP) * N + n;
          if (first + u * SWEEP < M) {
            store16_nt(y, make_uint4(f2u(v[u][0][0]), f2u(v[u][0][1]), f2u(v[u][0][2]), f2u(v[u][0][3])));
            store16_nt(y + 4, make_uint4(f2u(v[u][1][0]), f2u(v[u][1][1]), f2u(v[u][1][2]), f2u(v[u][1][3])));
          }
        }
      }
    }
  }
  __device__ __forceinline__ void flush(const TW& tw, int pass_row, LaneStats& st) {
    if (!left) return;
    // the next row's values come from LDS while the present row is worked on
    float nv[8], nu[GATED ? 8 : 1];
    take(tw, r0, col, nv);
    if constexpr (GATED) take(tw, r0, col + PAIR, nu);
#pragma unroll 1
    for (int i = 0; i < ROWS; ++i) {
      const int r = r0 + i * SWEEP;
      const int64_t m = m0 + pass_row + r;
      if (m >= M) break;
      float v[8], up[8], rs[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = nv[e];
        if constexpr (GATED) up[e] = nu[e];
      }
      unpack_bf16x8(res[0], rs);
      res[0] = res[1];
      request(pass_row, i + 2, &res[1]);
      const int rn = i + 1 < ROWS ? r + SWEEP : r;
      take(tw, rn, col, nv);
      if constexpr (GATED) take(tw, rn, col + PAIR, nu);
      epilogue8<GATED>(a, v, up, bias, rs, m, n, N, vec, left, scale, st);
    }
  }
};

}  // namespace fp8mi
