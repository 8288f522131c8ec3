// Host-side launch of the dense GEMM kernel with a feed-forward epilogue: tile
// shape per problem size and accumulation mode, and the operand-format switch.
// Shared by gemm_fused.hip and gemm_gated.hip, which instantiate it.
#pragma once

#include "gemm_kernel.hpp"

namespace fp8mi {

template <int BM, int BN, int WM, int WN, int FA, int FB, int MODE, class EPI>
inline hipError_t epi_run(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                          const float* sb, const EPI& epi, hipStream_t st) {
  constexpr int OUT_BN = std::is_same<EPI, GatedEpi>::value ? BN / 2 : BN;
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (int)((N + OUT_BN - 1) / OUT_BN);
  const int group_m = 4;  // bands of 4 tile-rows, as the plain GEMM's
  hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, FA, FB, kF32, MODE, false, EPI>),
                     dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WM * WN), 0, st, A, B, (int)M, (int)N, (int)K, sa,
                     sb, (void*)nullptr, tiles_m, tiles_n, group_m, epi, MxScales{nullptr, nullptr});
  return hipGetLastError();
}

template <int FA, int FB, int MODE, class EPI>
inline hipError_t epi_shape(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa,
                            const float* sb, const EPI& epi, hipStream_t st) {
  constexpr int64_t W = std::is_same<EPI, GatedEpi>::value ? 2 : 1;  // B rows per output column
  if (M >= 1024 && W * N >= 1024) {
    if constexpr (MODE == kAccumExact) return epi_run<256, 256, 2, 4, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, st);
    else return epi_run<256, 256, 4, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, st);
  }
  return epi_run<128, 128, 2, 2, FA, FB, MODE, EPI>(A, B, M, N, K, sa, sb, epi, st);
}

template <int MODE, class EPI>
inline hipError_t epi_fmt(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                          const float* sa, const float* sb, const EPI& epi, hipStream_t st) {
  if (fa == kE4M3 && fb == kE4M3) return epi_shape<kE4M3, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, st);
  if (fa == kE5M2 && fb == kE4M3) return epi_shape<kE5M2, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, st);
  if (fa == kE4M3 && fb == kE5M2) return epi_shape<kE4M3, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, st);
  return epi_shape<kE5M2, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, st);
}

template <class EPI>
inline hipError_t epi_launch(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                             const float* sa, const float* sb, const EPI& epi, int accum, hipStream_t st) {
  if (epi.amax_bits || epi.sat) {
    const hipError_t e = launch_clear_stats(reinterpret_cast<float*>(epi.amax_bits), epi.sat, st);
    if (e != hipSuccess) return e;
  }
  if (M == 0 || N == 0) return hipSuccess;
  if (M <= kFewRows) return launch_gemm_few_rows(A, fa, B, fb, M, N, K, sa, sb, epi, std::is_same<EPI, GatedEpi>::value, st);
  if (accum == kAccumMfma8) return epi_fmt<kAccumMfma8, EPI>(A, fa, B, fb, M, N, K, sa, sb, epi, st);
  return epi_fmt<kAccumExact, EPI>(A, fa, B, fb, M, N, K, sa, sb, epi, st);
}

}  // namespace fp8mi
