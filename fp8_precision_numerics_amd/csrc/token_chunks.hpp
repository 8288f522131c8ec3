// How the gradient of the embedding cuts its sorted tokens, and the scratch that takes.
// Plain host C++, as gemm_shape.hpp.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace fp8mi {

constexpr int64_t kMaxTokens = int64_t(1) << 20;  // the most that one call sorts
constexpr int kSortBlock = 8192;                  // tokens that are ranked among each other
constexpr int64_t kMostChunks = 4096;             // they fill the device

// Sorted tokens a chunk: 16 (two requests of eight rows a lane) until that makes kMostChunks; then longer ones.
inline int64_t chunk_size(int64_t rows) {
  const int64_t c = (rows + kMostChunks - 1) / kMostChunks;
  return c < 16 ? 16 : (c + 7) / 8 * 8;
}

inline int64_t chunk_count(int64_t rows) { return (rows + chunk_size(rows) - 1) / chunk_size(rows); }

// Bytes of an array of a word a token.
inline int64_t token_words(int64_t rows) { return (rows * 4 + 15) & ~int64_t(15); }

// Keys and places (twice where blocks are merged), and two partial rows a chunk.
inline int64_t token_bytes(int64_t rows, int64_t cols, int64_t chunks) {
  return (rows > kSortBlock ? 4 : 2) * token_words(rows) + (chunks > 1 ? chunks * 2 * cols * 4 : 0);
}

// What a call of so many tokens needs.
inline size_t embedding_need(int64_t rows, int64_t cols) { return (size_t)token_bytes(rows, cols, chunk_count(rows)); }

// The most that a call of any number of tokens up to `rows` needs.  The chunks are fewer just behind each step of their length
// (65536 tokens: 4096 chunks of 16, 65537: 2731 of 24), and never more than kMostChunks.
inline size_t embedding_workspace(int64_t rows, int64_t cols) {
  return (size_t)token_bytes(rows, cols, rows > 16 * kMostChunks ? kMostChunks : chunk_count(rows));
}

}  // namespace fp8mi
