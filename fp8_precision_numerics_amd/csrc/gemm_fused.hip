// Matrix product with bias, activation and residual in its epilogue:
//
//   z = (A B^T) sinv_a sinv_b + bias,   y = act(z) + residual
//
// The dense kernel (gemm_kernel.hpp) with the epilogue of epilogue.hpp: the tile
// is staged in LDS as fp32 once the K loop is done and taken out eight columns a
// thread, whole rows at a time, so the bias, the residual, the kept z and y each
// move between HBM and the registers once, coalesced, and the product itself
// never leaves the chip.
#include "launch.hpp"
#include "gemm_few_rows.hpp"
#include "gemm_epi_dispatch.hpp"

namespace fp8mi {

hipError_t launch_gemm_fused(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                             const float* sinv_a, const float* sinv_b, const EpiArgs& args, int accum,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  FusedEpi epi;
  static_cast<EpiArgs&>(epi) = args;
  epi.partials = reinterpret_cast<float*>(workspace);
  return epi_launch(A, fa, B, fb, M, N, K, sinv_a, sinv_b, epi, accum, workspace ? workspace_bytes : 0, stream);
}

}  // namespace fp8mi
