// Launcher of the GEMM for few rows (gemm_few_rows.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "epilogue.hpp"

namespace fp8mi {

// Rows that the kernel takes at most.
constexpr int64_t kFewRows = 16;

// A [M x K], B [N x K] (gated: [2N x K]) codes, K contiguous; M in [1, kFewRows].
hipError_t launch_gemm_few_rows(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                                const float* sinv_a, const float* sinv_b, const EpiArgs& epi, bool gated,
                                hipStream_t stream);

}  // namespace fp8mi
