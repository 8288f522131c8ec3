// How the vocabulary's cross entropy cuts its vocabulary into pieces, and the scratch that
// takes.  Plain host C++, as gemm_shape.hpp.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace fp8mi {

// Pieces of the vocabulary are multiples of so many columns (the widest tile), but for the last.
constexpr int64_t kPieceCols = 256;

// Rows of codes are padded to whole steps of the products that read them.
inline int64_t up128(int64_t n) { return (n + 127) & ~int64_t(127); }
inline int64_t up16(int64_t n) { return (n + 15) & ~int64_t(15); }
inline int64_t up256(int64_t n) { return (n + 255) & ~int64_t(255); }

// Workspace of the forward for M rows and pieces of P columns: the target's logit and the
// carried pair of each row, then a pair a row for each tile (of at least 128 columns).
inline size_t vocab_loss_bytes(int64_t M, int64_t P) { return (size_t)(up16(M * 4) + up16(M * 8) + M * 8 * ((P + 127) / 128)); }

// Of the gradient: the codes both ways for pieces of P columns, and the fp32 sums of dx where there are several.
inline int64_t grad_bytes(int64_t M, int64_t V, int64_t K, int64_t P) {
  return up256(M * up128(P)) + up256(P * up128(M)) + (P < V ? up256(M * K * 4) : 0);
}

// The longest piece that the gradient's products' offsets reach.
inline int64_t most_columns(int64_t K) {
  const int64_t most = ((int64_t(1) << 31) - 1) / K / kPieceCols * kPieceCols;
  return most < (int64_t(1) << 22) ? most : (int64_t(1) << 22);
}

// Whether a workspace holds the gradient's vocabulary whole.
inline bool grad_whole(int64_t M, int64_t V, int64_t K, size_t workspace_bytes) {
  return V <= most_columns(K) && grad_bytes(M, V, K, V) <= (int64_t)workspace_bytes;
}

// Otherwise: the longest piece that it holds (the entry point has seen to kPieceCols).
inline int64_t grad_longest(int64_t M, int64_t K, size_t workspace_bytes) {
  const int64_t most = most_columns(K);
  int64_t fit = ((int64_t)workspace_bytes - up256(M * K * 4) - 512) / (M + up128(M)) / kPieceCols * kPieceCols;
  fit = fit < kPieceCols ? kPieceCols : fit;
  return fit < most ? fit : most;
}

// Workspace with which M rows, a vocabulary of V and rows of K codes go in `pieces` pieces (0: the least that both
// directions take), or as many more as the longest piece asks for.
inline size_t vocab_workspace(int64_t M, int64_t V, int64_t K, int64_t pieces) {
  if (M == 0) return 0;
  const int64_t asked = pieces > 0 ? up256((V + pieces - 1) / pieces) : kPieceCols, most = most_columns(K);
  // A vocabulary that is longer than the longest piece needs dx's sums, however few pieces are asked for.
  const int64_t P = asked < most ? asked : most;
  size_t back = (size_t)grad_bytes(M, V, K, P < V ? P : V);
  const size_t whole = (size_t)grad_bytes(M, V, K, V), fwd = vocab_loss_bytes(M, asked < V ? asked : V);
  // one piece needs no sums of dx, so it may be the smaller
  if (V <= most && whole < back) back = whole;
  return back > fwd ? back : fwd;
}

}  // namespace fp8mi
