// Host-side launch of the dense GEMM kernel with a tile epilogue of the vocabulary's
// cross entropy: tile shape per problem size, operand-format switch.
#pragma once

#include "gemm_kernel.hpp"
#include "gemm_shape.hpp"
#include "launch.hpp"
#include "vocab.hpp"

namespace fp8mi {

// The shape by the dense GEMM's estimate (a vocabulary's columns fill the chip without a split of
// K); its three-stage form of 64 x 128 tiles is not built here: where the rows are few, the tiles of
// a vocabulary share the compute units.
inline int vocab_shape(const VocabOperands& o, int64_t N, int accum) {
  const int shape = choose_tile(o.M, N, o.K, accum == kAccumMfma8, 0, persistent_groups(1)).shape;
  return shape == 3 ? 2 : shape;
}

template <int BM, int BN, int WM, int WN, int FA, int FB, int MODE, class EPI>
inline hipError_t vocab_run(const VocabOperands& o, const uint8_t* b, int64_t N, const EPI& epi, hipStream_t st) {
  const int tiles_m = (int)((o.M + BM - 1) / BM), tiles_n = (int)((N + BN - 1) / BN);
  const int group_m = 4;  // bands of 4 tile-rows, as the plain GEMM's
  hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, FA, FB, kF32, MODE, false, EPI>), dim3((unsigned)(tiles_m * tiles_n)),
                     dim3(64 * WM * WN), 0, st, o.a, b, (int)o.M, (int)N, (int)o.K, o.sinv_a, o.sinv_b, (void*)nullptr,
                     tiles_m, tiles_n, group_m, epi, MxScales{nullptr, nullptr});
  return hipGetLastError();
}

template <int FA, int FB, int MODE, class EPI>
inline hipError_t vocab_shaped(const VocabOperands& o, const uint8_t* b, int64_t N, const EPI& epi, hipStream_t st) {
  const int shape = vocab_shape(o, N, MODE);
  if (shape == 0) {
    // 8 wavefronts either way, arranged as the plain GEMM's of that mode
    if constexpr (MODE == kAccumExact) return vocab_run<256, 256, 2, 4, FA, FB, MODE>(o, b, N, epi, st);
    else return vocab_run<256, 256, 4, 2, FA, FB, MODE>(o, b, N, epi, st);
  }
  if (shape == 1) return vocab_run<128, 128, 2, 2, FA, FB, MODE>(o, b, N, epi, st);
  return vocab_run<64, 128, 2, 2, FA, FB, MODE>(o, b, N, epi, st);
}

template <int MODE, class EPI>
inline hipError_t vocab_fmt(const VocabOperands& o, const uint8_t* b, int64_t N, const EPI& epi, hipStream_t st) {
  if (o.fa == kE4M3 && o.fb == kE4M3) return vocab_shaped<kE4M3, kE4M3, MODE>(o, b, N, epi, st);
  if (o.fa == kE5M2 && o.fb == kE4M3) return vocab_shaped<kE5M2, kE4M3, MODE>(o, b, N, epi, st);
  if (o.fa == kE4M3 && o.fb == kE5M2) return vocab_shaped<kE4M3, kE5M2, MODE>(o, b, N, epi, st);
  return vocab_shaped<kE5M2, kE5M2, MODE>(o, b, N, epi, st);
}

// One launch on columns [col, col + N).
template <class EPI>
inline hipError_t vocab_launch(const VocabOperands& o, int64_t col, int64_t N, const EPI& epi, int accum, hipStream_t st) {
  const uint8_t* b = o.b + col * o.K;
  if (accum == kAccumMfma8) return vocab_fmt<kAccumMfma8>(o, b, N, epi, st);
  return vocab_fmt<kAccumExact>(o, b, N, epi, st);
}

}  // namespace fp8mi
