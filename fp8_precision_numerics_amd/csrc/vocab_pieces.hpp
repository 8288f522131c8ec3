// How the vocabulary's cross entropy cuts its vocabulary into pieces, and the scratch that
// takes.  Plain host C++, as gemm_shape.hpp.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gemm_rounds.hpp"

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

// Columns of one launch of the logits' products, whose threads have to be fewer than 2^32: 256 a tile of 64 x 128, and
// 512 for 128 columns of the streaming kernel.
inline int64_t launch_columns(int64_t M) { return ((int64_t(1) << 24) - 1) / ((M + 63) / 64) * 128 / kPieceCols * kPieceCols; }
constexpr int64_t kFewColumns = int64_t(1) << 29;

// The longest piece of the gradient: what its products' offsets reach, and a launch.
inline int64_t most_columns(int64_t M, int64_t K) {
  int64_t most = ((int64_t(1) << 31) - 1) / K / kPieceCols * kPieceCols;
  most = most < (int64_t(1) << 22) ? most : (int64_t(1) << 22);
  return most < launch_columns(M) ? most : launch_columns(M);
}

// Whether a workspace holds the gradient's vocabulary whole.
inline bool grad_whole(int64_t M, int64_t V, int64_t K, size_t workspace_bytes) {
  return V <= most_columns(M, K) && grad_bytes(M, V, K, V) <= (int64_t)workspace_bytes;
}

// Otherwise: the longest piece that it holds (the entry point has seen to kPieceCols).  Whole steps of the codes
// leave nothing to round up, so a size that was asked for pieces of so many columns holds them.
inline int64_t grad_longest(int64_t M, int64_t K, size_t workspace_bytes) {
  const int64_t most = most_columns(M, K);
  int64_t fit = ((int64_t)workspace_bytes - up256(M * K * 4)) / (M + up128(M)) / kPieceCols * kPieceCols;
  fit = fit < kPieceCols ? kPieceCols : fit;
  return fit < most ? fit : most;
}

// Workspace with which M rows, a vocabulary of V and rows of K codes go in `pieces` pieces (0: the least that both
// directions take), or as many more as the longest piece asks for.
inline size_t vocab_workspace(int64_t M, int64_t V, int64_t K, int64_t pieces) {
  if (M == 0) return 0;
  const int64_t asked = pieces > 0 ? up256((V - 1) / pieces + 1) : kPieceCols, most = most_columns(M, K);
  // A vocabulary that is longer than the longest piece needs dx's sums, however few pieces are asked for.
  const int64_t P = asked < most ? asked : most;
  size_t back = (size_t)grad_bytes(M, V, K, P < V ? P : V);
  const size_t whole = (size_t)grad_bytes(M, V, K, V), fwd = vocab_loss_bytes(M, asked < V ? asked : V);
  // one piece needs no sums of dx, so it may be the smaller
  if (V <= most && whole < back) back = whole;
  return back > fwd ? back : fwd;
}

// Estimate of the gradient's passes over pieces of P columns, in microseconds: the three products of each, and its
// passes over dx's fp32 sums.  `fp8_logits`, `fp8`: the logits' and the products' cores.
inline double pieces_time(int64_t M, int64_t V, int64_t K, int64_t P, bool fp8_logits, bool fp8, int64_t cus) {
  double t = 0.0;
  for (int64_t col = 0; col < V; col += P) {
    const int64_t n = V - col < P ? V - col : P;
    double one = plan_rounds(M, n, K, fp8_logits, 0, cus).us + plan_rounds(K, M, n, fp8, 0, cus).us + plan_rounds(K, n, M, fp8, 0, cus).us;
    if (P < V) one += 8.0 * M * K / 5.0e6;
    if (n == P && V / P > 1) {  // all whole pieces at once
      t += one * (double)(V / P);
      col += (V / P - 1) * P;
    } else {
      t += one;
    }
  }
  return t;
}

// Columns of the gradient's pieces: the whole vocabulary where the workspace holds it.  Otherwise equal pieces, as few as
// fit, or up to four more where the estimate prefers them: tiles that fill whole rounds of the compute units are worth another
// pass over dx's sums (8192 x 4096 x 65536 on the FP8 cores over 512 MiB: four pieces of 16384 columns 5.21 ms, the three that fit 5.40).
inline int64_t grad_piece(int64_t M, int64_t V, int64_t K, size_t workspace_bytes, bool fp8_logits, bool fp8, int64_t cus) {
  if (grad_whole(M, V, K, workspace_bytes)) return V;
  const int64_t fit = grad_longest(M, K, workspace_bytes), least = (V + fit - 1) / fit;
  int64_t P = fit;
  double best = 1e300;
  for (int64_t pieces = least; pieces <= least + 4; ++pieces) {
    const int64_t p = up256((V + pieces - 1) / pieces);
    const double t = pieces_time(M, V, K, p, fp8_logits, fp8, cus);
    if (t < best) {
      best = t;
      P = p;
    }
  }
  return P;
}

}  // namespace fp8mi
