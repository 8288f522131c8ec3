// Host-side launch of the dense GEMM kernel with a feed-forward epilogue: tile
// shape per problem size and accumulation mode, and the operand-format switch.
// Shared by gemm_fused.hip and gemm_gated.hip, which instantiate it.
#pragma once

#include "gemm_kernel.hpp"
#include "gemm_shape.hpp"
#include "launch.hpp"

namespace fp8mi {

// The sums of a split product's parts, scaled, through the epilogue: eight columns
// of a row a thread.
template <class EPI>
__global__ __launch_bounds__(256) void epilogue_partials_kernel(EPI a, int64_t M, int64_t N,
                                                               const float* __restrict__ sinv_a,
                                                               const float* __restrict__ sinv_b) {
  constexpr bool GATED = std::is_same<EPI, GatedEpi>::value, PRODUCT = std::is_same<EPI, ProductEpi>::value;
  const int64_t cpr = (N + 7) / 8, total = M * cpr, ld = GATED ? 2 * N : N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  LaneStats st;
  __shared__ uint32_t scratch[8];
  if (i < total) {
    const int64_t m = i / cpr, n = (i - m * cpr) * 8;
    const bool vec = (N & 7) == 0;
    const int left = (int)(N - n < 8 ? N - n : 8);
    const float sc = sinv_a[0] * sinv_b[0];
    float v[GATED ? 2 : 1][8], bias[8], res[8];
    uint4 bb = make_uint4(0u, 0u, 0u, 0u), rr = bb;
    if constexpr (!GATED && !PRODUCT) {
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
    if constexpr (PRODUCT) {
      v4f sum[2] = {(v4f){0.f, 0.f, 0.f, 0.f}, (v4f){0.f, 0.f, 0.f, 0.f}};
      if (a.add) load_f32x8(a.add + m * N + n, vec, left, sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) res[e] = sum[e >> 2][e & 3];
    }
    const float scale = (a.out == kYE4M3 || a.out == kYE5M2) ? *a.out_scale : 1.0f;
    epilogue8<GATED>(a, v[0], v[GATED ? 1 : 0], bias, res, m, n, N, vec, left, scale, st);
  }
  if (a.amax_bits || a.sat) publish_epilogue_stats(a, st, scratch);
}

// `split` > 1: that many workgroups share a tile's K (no part is empty) over
// epi.partials, and a second kernel finishes.
template <int BM, int BN, int WM, int WN, int FA, int FB, int MODE, class EPI, int STAGES = 2, bool BT = false>
inline hipError_t epi_run(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                          const float* sb, EPI epi, int split, hipStream_t st) {
  constexpr bool GATED = std::is_same<EPI, GatedEpi>::value;
  constexpr int OUT_BN = GATED ? BN / 2 : BN;
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (int)((N + OUT_BN - 1) / OUT_BN);
  const int group_m = 4;  // bands of 4 tile-rows, as the plain GEMM's
  const int64_t steps = (K + kBK - 1) / kBK;
  const int64_t per = (steps + split - 1) / split;
  epi.split = (int)((steps + per - 1) / per);
  if (epi.split == 1 && (epi.amax_bits || epi.sat)) {  // a split product's first kernel clears them itself
    const hipError_t e = launch_clear_stats(reinterpret_cast<float*>(epi.amax_bits), epi.sat, st);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, FA, FB, kF32, MODE, BT, EPI, STAGES>),
                     dim3((unsigned)(tiles_m * tiles_n * epi.split)), dim3(64 * WM * WN), 0, st, A, B, (int)M, (int)N,
                     (int)K, sa, sb, (void*)nullptr, tiles_m, tiles_n, group_m, epi, MxScales{nullptr, nullptr});
  if (epi.split > 1) {
    const int64_t chunks = M * ((N + 7) / 8);
    hipLaunchKernelGGL(epilogue_partials_kernel<EPI>, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, st, epi, M,
                       N, sa, sb);
  }
  return hipGetLastError();
}

template <int FA, int FB, int MODE, class EPI>
inline hipError_t epi_shape(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                            const float* sb, const EPI& epi, size_t workspace_bytes, hipStream_t st) {
  constexpr int64_t W = std::is_same<EPI, GatedEpi>::value ? 2 : 1;  // B rows per output column
  const TileChoice c = choose_tile(M, W * N, K, MODE == kAccumMfma8, workspace_bytes, persistent_groups(1));
  if (c.shape == 0) {
    // 8 wavefronts either way, arranged as the plain GEMM's of that mode
    if constexpr (MODE == kAccumExact) return epi_run<256, 256, 2, 4, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
    else return epi_run<256, 256, 4, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
  }
  if (c.shape == 1) return epi_run<128, 128, 2, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
  if (c.shape == 2) return epi_run<64, 128, 2, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, c.split, st);
  return epi_run<64, 128, 2, 2, FA, FB, MODE, EPI, 3>(A, B, M, N, K, sa, sb, epi, c.split, st);
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
  const bool empty = M == 0 || N == 0;
  if ((empty || M <= kFewRows) && (epi.amax_bits || epi.sat)) {
    const hipError_t e = launch_clear_stats(reinterpret_cast<float*>(epi.amax_bits), epi.sat, st);
    if (e != hipSuccess) return e;
  }
  if (empty) return hipSuccess;
  if (M <= kFewRows) return launch_gemm_few_rows(A, fa, B, fb, M, N, K, sa, sb, epi, std::is_same<EPI, GatedEpi>::value, st);
  if (accum == kAccumMfma8) return epi_fmt<kAccumMfma8, EPI>(A, fa, B, fb, M, N, K, sa, sb, epi, workspace_bytes, st);
  return epi_fmt<kAccumExact, EPI>(A, fa, B, fb, M, N, K, sa, sb, epi, workspace_bytes, st);
}

}  // namespace fp8mi
