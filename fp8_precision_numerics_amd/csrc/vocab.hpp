// What the files of the vocabulary's cross entropy (vocab_*.hip) launch of each other.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_few_rows.hpp"
#include "gemm_rounds.hpp"
#include "gemm_tile.hpp"
#include "vocab_epilogue.hpp"
#include "vocab_pieces.hpp"

namespace fp8mi {

// Few rows have exact products in either mode, the gradient's as the loss's: they have to be of the same logits.
inline int logits_mode(int64_t M, int accum) { return M <= kFewRows ? (int)kAccumExact : accum; }

// One product of the loss: codes A [M x K] (hidden states) and B [N x K] (a piece of the
// vocabulary's weight) with their formats and inverse scales.
struct VocabOperands {
  const uint8_t* a;
  const uint8_t* b;
  int fa, fb;
  const float* sinv_a;
  const float* sinv_b;
  int64_t M, K;
};

// The products with either epilogue (M > 0, N > 0), on columns [col, col + N) of the vocabulary;
// *tiles: the loss's pairs a row.
hipError_t launch_vocab_logits(const VocabOperands& o, int64_t col, int64_t N, const LossEpi& epi, int accum, int* tiles,
                               hipStream_t stream);
hipError_t launch_vocab_grad(const VocabOperands& o, int64_t col, int64_t N, const LogitGradEpi& epi, int accum, hipStream_t stream);

// y [M x N] = (A [M x lda] B [K x N]) sinv_a sinv_b + add; K is any number, A's rows hold zeros from K
// to lda = up128(K); K * N < 2^31, N a multiple of 16; `workspace` for the parts of a split K.
hipError_t launch_vocab_product(const uint8_t* A, int64_t lda, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                                const float* sinv_a, const float* sinv_b, const float* add, void* y, int ytype, int accum,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

}  // namespace fp8mi
