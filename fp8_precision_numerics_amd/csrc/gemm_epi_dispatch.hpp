// Host-side launch of the dense GEMM kernel with a feed-forward epilogue: tile
// shape per problem size and accumulation mode, and the operand-format switch.
// Shared by gemm_fused.hip and gemm_gated.hip, which instantiate it.
#pragma once

#include "gemm_kernel.hpp"

namespace fp8mi {

// The sums of a split product's parts, scaled, through the epilogue: eight columns
// of a row a thread.
template <bool GATED>
__global__ __launch_bounds__(256) void epilogue_partials_kernel(EpiArgs a, int64_t M, int64_t N,
                                                               const float* __restrict__ sinv_a,
                                                               const float* __restrict__ sinv_b) {
  const int64_t cpr = (N + 7) / 8, total = M * cpr, ld = GATED ? 2 * N : N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  LaneStats st;
  const uint32_t seen = a.amax_bits ? __hip_atomic_load(a.amax_bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
  if (i < total) {
    const int64_t m = i / cpr, n = (i - m * cpr) * 8;
    const bool vec = (N & 7) == 0;
    const int left = (int)(N - n < 8 ? N - n : 8);
    const float sc = sinv_a[0] * sinv_b[0];
    float v[GATED ? 2 : 1][8], bias[8], res[8];
    uint4 bb = make_uint4(0u, 0u, 0u, 0u), rr = bb;
    if constexpr (!GATED) {
      if (a.bias) bb = load_bf16x8(a.bias + n, vec, left);
      if (a.residual) rr = load_bf16x8(a.residual + m * N + n, vec, left);
    }
#pragma unroll
    for (int p = 0; p < (GATED ? 2 : 1); ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[p][e] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < a.split; ++s) {
#pragma unroll
      for (int p = 0; p < (GATED ? 2 : 1); ++p) {
        const float* src = a.partials + ((int64_t)s * M + m) * ld + p * N + n;
        if (vec) {
          const v4f lo = reinterpret_cast<const v4f*>(src)[0], hi = reinterpret_cast<const v4f*>(src)[1];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[p][e] += lo[e];
            v[p][4 + e] += hi[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < left) v[p][e] += src[e];
        }
      }
    }
#pragma unroll
    for (int p = 0; p < (GATED ? 2 : 1); ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[p][e] *= sc;
    unpack_bf16x8(bb, bias);
    unpack_bf16x8(rr, res);
    const float scale = (a.out == kYE4M3 || a.out == kYE5M2) ? *a.out_scale : 1.0f;
    epilogue8<GATED>(a, v[0], v[GATED ? 1 : 0], bias, res, m, n, N, vec, left, scale, st);
  }
  if (a.amax_bits || a.sat) publish_epilogue_stats(a, st, seen, threadIdx.x & 63);
}

// `split` > 1: that many workgroups share a tile's K (no part is empty) over
// epi.partials, and a second kernel finishes.
template <int BM, int BN, int WM, int WN, int FA, int FB, int MODE, class EPI>
inline hipError_t epi_run(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                          const float* sb, EPI epi, int split, hipStream_t st) {
  constexpr bool GATED = std::is_same<EPI, GatedEpi>::value;
  constexpr int OUT_BN = GATED ? BN / 2 : BN;
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (int)((N + OUT_BN - 1) / OUT_BN);
  const int group_m = 4;  // bands of 4 tile-rows, as the plain GEMM's
  const int64_t steps = (K + kBK - 1) / kBK;
  const int64_t per = (steps + split - 1) / split;
  epi.split = (int)((steps + per - 1) / per);
  hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, FA, FB, kF32, MODE, false, EPI>),
                     dim3((unsigned)(tiles_m * tiles_n * epi.split)), dim3(64 * WM * WN), 0, st, A, B, (int)M, (int)N,
                     (int)K, sa, sb, (void*)nullptr, tiles_m, tiles_n, group_m, epi, MxScales{nullptr, nullptr});
  if (epi.split > 1) {
    const int64_t chunks = M * ((N + 7) / 8);
    hipLaunchKernelGGL(epilogue_partials_kernel<GATED>, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, st,
                       static_cast<const EpiArgs&>(epi), M, N, sa, sb);
  }
  return hipGetLastError();
}

// Tile shape and split of K.  A compute unit holds one 256 x 256 tile, two of
// 128 x 128 or three of 64 x 128; the larger ones need fewer operand bytes a
// product, the smaller ones fill the chip with fewer rows and columns, and a split
// fills it where even those are few.  The choice is the least of an estimate in
// microseconds, from step times (a K step of 128) measured on MI355X:
//
//   L = the most workgroups that any compute unit gets, S = K steps of a part
//   start + S max(alone, L each) + (split: second launch + traffic of the partials)
//
// `alone` is the step of a lone workgroup (latency-bound), `each` the step's share
// of a busy compute unit.  At M x N x K the choices measured (exact mode, us; 256,
// 128 and 64 stand for the three shapes, /s for the split):
//   8192 x 4096 x 16384   256: 715   128: 784   64: 876
//   1003 x 16384 x 4096   256: 103   128: 115   64: 127
//   2048 x 4096 x 4096    256: 84    128: 58    64: 67
//   500 x 4096 x 16384    256/6: 74  128/4: 66  64/2: 70   64: 96
//   64 x 4096 x 16384     64: 96     64/4: 34   64/8: 24   64/16: 30
struct EpiShape {
  int shape;  // 0: 256 x 256, 1: 128 x 128, 2: 64 x 128
  int split;
};

inline EpiShape choose_epi_shape(int64_t M, int64_t brows, int64_t K, int mode, size_t workspace_bytes) {
  struct Cost {
    int bm, bn;
    double start, alone, each;
  };
  static constexpr Cost kExact[3] = {{256, 256, 14.0, 2.4, 2.8}, {128, 128, 6.0, 0.90, 0.80}, {64, 128, 4.0, 0.73, 0.45}};
  static constexpr Cost kFp8[3] = {{256, 256, 8.0, 1.25, 1.5}, {128, 128, 5.0, 0.90, 0.52}, {64, 128, 3.5, 0.73, 0.33}};
  const Cost* costs = mode == kAccumMfma8 ? kFp8 : kExact;
  const int64_t cus = persistent_groups(1), steps = (K + kBK - 1) / kBK;
  EpiShape best{2, 1};
  double least = 1e300;
  for (int i = 0; i < 3; ++i) {
    const Cost& c = costs[i];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((brows + c.bn - 1) / c.bn);
    for (int split = 1; split <= 32 && split <= steps; split = split < 4 ? split + 1 : split + split / 2) {
      const double traffic = (double)split * M * brows * 4.0;
      if (split > 1 && (traffic > (double)workspace_bytes || tiles * split > 4 * cus)) break;
      const int64_t load = (tiles * split + cus - 1) / cus;
      const double step = c.alone > load * c.each ? c.alone : load * c.each;
      const double t = c.start + (double)((steps + split - 1) / split) * step +
                       (split > 1 ? 4.0 + 2.0 * traffic / 5.0e6 : 0.0);
      if (t < least) {
        least = t;
        best = EpiShape{i, split};
      }
    }
  }
  return best;
}

template <int FA, int FB, int MODE, class EPI>
inline hipError_t epi_shape(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                            const float* sb, const EPI& epi, size_t workspace_bytes, hipStream_t st) {
  constexpr int64_t W = std::is_same<EPI, GatedEpi>::value ? 2 : 1;  // B rows per output column
  const EpiShape c = choose_epi_shape(M, W * N, K, MODE, workspace_bytes);
  if (c.shape == 0) {
    // 8 wavefronts either way, arranged as the plain GEMM's of that mode
    if constexpr (MODE == kAccumExact) return epi_run<256, 256, 2, 4, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
    else return epi_run<256, 256, 4, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
  }
  if (c.shape == 1) return epi_run<128, 128, 2, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
  return epi_run<64, 128, 2, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
}

template <int MODE, class EPI>
inline hipError_t epi_fmt(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                          const float* sa, const float* sb, const EPI& epi, size_t workspace_bytes,
                          hipStream_t st) {
  if (fa == kE4M3 && fb == kE4M3) return epi_shape<kE4M3, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  if (fa == kE5M2 && fb == kE4M3) return epi_shape<kE5M2, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  if (fa == kE4M3 && fb == kE5M2) return epi_shape<kE4M3, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  return epi_shape<kE5M2, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
}

template <class EPI>
inline hipError_t epi_launch(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                             const float* sa, const float* sb, const EPI& epi, int accum, size_t workspace_bytes,
                             hipStream_t st) {
  if (epi.amax_bits || epi.sat) {
    const hipError_t e = launch_clear_stats(reinterpret_cast<float*>(epi.amax_bits), epi.sat, st);
    if (e != hipSuccess) return e;
  }
  if (M == 0 || N == 0) return hipSuccess;
  if (M <= kFewRows) return launch_gemm_few_rows(A, fa, B, fb, M, N, K, sa, sb, epi, std::is_same<EPI, GatedEpi>::value, st);
  if (accum == kAccumMfma8) return epi_fmt<kAccumMfma8, EPI>(A, fa, B, fb, M, N, K, sa, sb, epi, workspace_bytes, st);
  return epi_fmt<kAccumExact, EPI>(A, fa, B, fb, M, N, K, sa, sb, epi, workspace_bytes, st);
}

}  // namespace fp8mi
