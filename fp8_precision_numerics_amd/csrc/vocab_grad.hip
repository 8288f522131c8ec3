// The vocabulary's cross entropy, backward: the logits of a piece of the vocabulary
// again, as codes of their gradient (vocab_epilogue.hpp), and the two products on those.
//
//   d = dloss (exp(z - lse) - [column = target]),  codes q = round_to_fp8(d scale)
//   dx = (q W) sinv_d sinv_w,  dw = (q^T x) sinv_d sinv_x
//
// Three products of 2 M V K operations on the matrix cores.  Of the M x V gradients only a piece's
// codes exist at a time, row-major and transposed, the orientations in which the two products read
// their first operand; dx grows over the pieces in fp32.
// Measured on MI355X: 8192 x 65536 x 4096 on the FP8 cores in four pieces 5.13 ms (2.57 PFLOP/s of the three products: each piece's
// codes 465 us, dx 412, dw 403); 219 x 50021 x 2048 exact, one piece, 202-207 us, which writes 205 MB of dw.
#include "launch.hpp"
#include "model_ends.hpp"
#include "vocab_dispatch.hpp"

namespace fp8mi {

hipError_t launch_vocab_grad(const VocabOperands& o, int64_t col, int64_t N, const LogitGradEpi& epi, int accum, hipStream_t stream) {
  const int mode = logits_mode(o.M, accum);
  const int64_t first = plan_rounds(o.M, N, o.K, mode == kAccumMfma8, 0, persistent_groups(1)).first;
  hipError_t status = vocab_launch(o, col, first, epi, mode, stream);
  if (status != hipSuccess || first == N) return status;
  LogitGradEpi rest = epi;
  rest.col0 += first;
  if (rest.q) rest.q += first;
  if (rest.q_t) rest.q_t += first * epi.ldt;
  return vocab_launch(o, col + first, N - first, rest, mode, stream);
}

hipError_t launch_vocab_cross_entropy_backward(const VocabOperands& o, int64_t V, const Targets& targets, const float* lse,
                                               const float* dloss, int fmt, const float* scale, const float* scale_inv,
                                               void* dx, int dxtype, void* dw, int dwtype, float* amax,
                                               unsigned long long* sat, int accum, void* workspace,
                                               size_t workspace_bytes, hipStream_t stream) {
  if (amax || sat) {
    const hipError_t e = launch_clear_stats(amax, sat, stream);
    if (e != hipSuccess) return e;
  }
  const int64_t M = o.M, K = o.K, ldt = up128(M);
  const int64_t dwsize = dwtype == kBF16 ? 2 : 4;
  if (M == 0) return dw ? launch_fill_rows(nullptr, dw, V * K * dwsize / 16, stream) : hipSuccess;
  const int64_t P = grad_piece(M, V, K, workspace_bytes, logits_mode(M, accum) == kAccumMfma8, accum == kAccumMfma8, persistent_groups(1));
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  uint8_t* const q = ws;
  uint8_t* const q_t = q + up256(M * up128(P));
  uint8_t* rest = q_t + up256(P * ldt);
  // An fp32 dx is its own sum.
  float* sum = dxtype == kF32 ? reinterpret_cast<float*>(dx) : reinterpret_cast<float*>(rest);
  if (P < V) rest += up256(M * K * 4);
  const size_t left = workspace_bytes > (size_t)(rest - ws) ? workspace_bytes - (size_t)(rest - ws) : 0;
  for (int64_t col = 0; col < V; col += P) {
    const int64_t n = V - col < P ? V - col : P;
    const LogitGradEpi epi{lse, dloss, scale, dx ? q : nullptr, dw ? q_t : nullptr, reinterpret_cast<uint32_t*>(amax), sat, targets,
                           V, col, up128(n), ldt, fmt};
    hipError_t e = launch_vocab_grad(o, col, n, epi, accum, stream);
    if (e != hipSuccess) return e;
    if (dx) {
      const bool first = col == 0, last = col + n >= V;
      e = launch_vocab_product(q, up128(n), fmt, o.b + col * K, o.fb, M, K, n, scale_inv, o.sinv_b, first ? nullptr : sum,
                               last ? dx : (void*)sum, last ? dxtype : (int)kF32, accum, rest, left, stream);
      if (e != hipSuccess) return e;
    }
    if (dw) {
      e = launch_vocab_product(q_t, ldt, fmt, o.a, o.fa, n, K, M, scale_inv, o.sinv_a, nullptr,
                               reinterpret_cast<uint8_t*>(dw) + col * K * dwsize, dwtype, accum, rest, left, stream);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace fp8mi
