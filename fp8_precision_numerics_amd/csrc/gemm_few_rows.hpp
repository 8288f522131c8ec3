// Launcher of the GEMM for few rows (gemm_few_rows.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "epilogue.hpp"
#include "few_rows_shape.hpp"

namespace fp8mi {

// A [M x K], B [N x K] (gated: [2N x K]) codes, K contiguous; M in [1, kFewRows].
hipError_t launch_gemm_few_rows(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                                const float* sinv_a, const float* sinv_b, const EpiArgs& epi, bool gated,
                                hipStream_t stream);

struct LossEpi;  // vocab_epilogue.hpp

// The same with the loss over the vocabulary behind it; *groups: the workgroups of that product, for each of which epi.partials
// holds a pair a row.  There are `slots` of those, one for every 128 columns at least.
hipError_t launch_loss_few_rows(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                                const float* sinv_a, const float* sinv_b, const LossEpi& epi, int64_t slots, int* groups,
                                hipStream_t stream);

}  // namespace fp8mi
