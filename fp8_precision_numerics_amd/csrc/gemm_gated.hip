// Gated feed-forward product, both projections in one kernel:
//
//   g = (A Wg^T) s,  u = (A Wu^T) s,  s = sinv_a sinv_b,   h = act(g) u
//
// B holds the gate's F rows, then the up projection's F rows.  The dense kernel
// (gemm_kernel.hpp) loads its B tile as alternating blocks of gate and up rows
// (SlabLoader's PAIR), one matrix-core block wide, so that both projections of
// an output column meet in one tile and A is read once for both; the epilogue
// (epilogue.hpp) multiplies them before anything is stored.
#include "launch.hpp"
#include "gemm_few_rows.hpp"
#include "gemm_epi_dispatch.hpp"

namespace fp8mi {

hipError_t launch_gemm_gated(const uint8_t* A, int fa, const uint8_t* B, int fb, int64_t M, int64_t N, int64_t K,
                             const float* sinv_a, const float* sinv_b, const EpiArgs& args, int accum,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  GatedEpi epi;
  static_cast<EpiArgs&>(epi) = args;
  epi.partials = reinterpret_cast<float*>(workspace);
  return epi_launch(A, fa, B, fb, M, N, K, sinv_a, sinv_b, epi, accum, workspace ? workspace_bytes : 0, stream);
}

}  // namespace fp8mi
