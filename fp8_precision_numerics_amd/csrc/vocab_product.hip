// The gradient products of the vocabulary's cross entropy: the dense kernel
// (gemm_kernel.hpp) on a first operand whose rows are padded to whole 16-byte
// granules, so that the number of tokens and of the vocabulary's columns, which are their K, may be any,
// with the fp32 sum of earlier pieces added in the epilogue.
#include "gemm_few_rows.hpp"
#include "gemm_epi_dispatch.hpp"
#include "launch.hpp"
#include "vocab.hpp"

namespace fp8mi {
namespace {

template <int FA, int FB, int MODE>
hipError_t product_shape(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K, const float* sa, const float* sb,
                         const ProductEpi& epi, size_t workspace_bytes, hipStream_t st) {
  const TileChoice c = choose_tile(M, N, K, MODE == kAccumMfma8, workspace_bytes, persistent_groups(1));
  if (c.shape == 0) {
    if constexpr (MODE == kAccumExact) return epi_run<256, 256, 2, 4, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
    else return epi_run<256, 256, 4, 2, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
  }
  if (c.shape == 1) return epi_run<128, 128, 2, 2, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
  if (c.shape == 2) return epi_run<64, 128, 2, 2, FA, FB, MODE, ProductEpi, 2, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
  return epi_run<64, 128, 2, 2, FA, FB, MODE, ProductEpi, 3, true>(A, B, M, N, K, sa, sb, epi, c.split, st);
}

template <int MODE>
hipError_t product_fmt(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K, const float* sa,
                       const float* sb, const ProductEpi& epi, size_t workspace_bytes, hipStream_t st) {
  if (fa == kE4M3 && fb == kE4M3) return product_shape<kE4M3, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  if (fa == kE5M2 && fb == kE4M3) return product_shape<kE5M2, kE4M3, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  if (fa == kE4M3 && fb == kE5M2) return product_shape<kE4M3, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
  return product_shape<kE5M2, kE5M2, MODE>(A, B, M, N, K, sa, sb, epi, workspace_bytes, st);
}

}  // namespace

hipError_t launch_vocab_product(const uint8_t* A, int64_t lda, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                                const float* sinv_a, const float* sinv_b, const float* add, void* y, int ytype, int accum,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  ProductEpi epi{};
  epi.y = y;
  epi.act = kActNone;
  epi.out = ytype;
  epi.partials = reinterpret_cast<float*>(workspace);
  epi.split = 1;
  epi.add = add;
  epi.lda = (int)lda;
  if (accum == kAccumMfma8) return product_fmt<kAccumMfma8>(A, fa, B, fb, M, N, K, sinv_a, sinv_b, epi, workspace_bytes, stream);
  return product_fmt<kAccumExact>(A, fa, B, fb, M, N, K, sinv_a, sinv_b, epi, workspace_bytes, stream);
}

}  // namespace fp8mi
