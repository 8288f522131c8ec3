// extern "C" entry points of the operators at both ends of a model: argument
// validation and dispatch, as api.hip.
#include <cmath>

#include "api_common.hpp"
#include "device_common.hpp"
#include "model_ends.hpp"
#include "token_chunks.hpp"
#include "vocab.hpp"

using namespace fp8mi;

namespace {

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The dropout argument of a call; FP8MI_OK means "go on".
int make_dropout(float p, const uint64_t* rng, Dropout* out) {
  if (!(p >= 0.0f) || p >= 1.0f) return FP8MI_ERR_SHAPE;
  const long cut = std::lrint((double)p * 65536.0);
  if (cut > 65535) return FP8MI_ERR_SHAPE;
  if (cut && !rng) return FP8MI_ERR_NULL;
  if (cut && !aligned8(rng)) return FP8MI_ERR_ALIGN;
  *out = Dropout{reinterpret_cast<const unsigned long long*>(rng), (uint32_t)cut, 65536.0f / (float)(65536 - cut)};
  return FP8MI_OK;
}

constexpr int64_t kMaxEmbedCols = int64_t(1) << 20;  // workgroups a row, of which a grid has thousands

bool index_ok(int t) { return t == FP8MI_I32 || t == FP8MI_I64; }
bool index_aligned(const void* p, int t) { return (reinterpret_cast<uintptr_t>(p) & (t == FP8MI_I64 ? 7u : 3u)) == 0; }

constexpr int64_t kMaxVocabK = int64_t(1) << 22;  // 256 rows of a piece in a 31-bit offset

// Sizes of the loss and its gradient.
int check_vocab_sizes(int64_t M, int64_t V, int64_t K) {
  if (M < 0 || V < 1 || K <= 0 || M > kMaxGemmK - 16 || V > kMaxDim || K > kMaxVocabK) return FP8MI_ERR_SHAPE;
  if (!dims_ok(M, K) || !dims_ok(V, K) || M * K > kMaxBufferBytes) return FP8MI_ERR_SHAPE;
  if (((M + 63) / 64) * ((V + 127) / 128 + 1) > kMaxDim) return FP8MI_ERR_SHAPE;
  return (K & 15) != 0 ? FP8MI_ERR_ALIGN : FP8MI_OK;
}

// What the loss's two entry points share, M != 0.
int check_vocab(const uint8_t* x, int fx, const uint8_t* w, int fw, int64_t M, int64_t V, int64_t K, const float* sinv_x,
                const float* sinv_w, const void* targets, int itype, int accum, const void* workspace) {
  if (!fmt_ok(fx) || !fmt_ok(fw)) return FP8MI_ERR_FORMAT;
  if (!index_ok(itype)) return FP8MI_ERR_DTYPE;
  if (!accum_ok(accum)) return FP8MI_ERR_ACCUM;
  const int bad = check_vocab_sizes(M, V, K);
  if (bad != FP8MI_OK) return bad;
  if (workspace && !aligned16(workspace)) return FP8MI_ERR_ALIGN;
  if (M == 0) return FP8MI_OK;
  if (!x || !w || !sinv_x || !sinv_w || !targets || !workspace) return FP8MI_ERR_NULL;
  if (!aligned16(x) || !aligned16(w) || !index_aligned(targets, itype)) return FP8MI_ERR_ALIGN;
  return FP8MI_OK;
}

}  // namespace

extern "C" {

int fp8_layernorm_quantize(const void* x, const void* residual, const void* weight, const void* bias, int xtype,
                           int64_t rows, int64_t cols, float eps, float dropout, const uint64_t* rng, int fmt,
                           const float* scale, void* sum_out, uint8_t* q, float* mean, float* rstd, float* amax,
                           unsigned long long* sat, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(xtype)) return FP8MI_ERR_DTYPE;
  if (!fmt_ok(fmt)) return FP8MI_ERR_FORMAT;
  if (!dims_ok(rows, cols) || cols > kMaxDim || !(eps >= 0.0f)) return FP8MI_ERR_SHAPE;
  if ((cols & 15) != 0) return FP8MI_ERR_ALIGN;
  if (workspace && (!aligned16(workspace) || workspace_bytes < 16)) return FP8MI_ERR_ALIGN;
  Dropout drop;
  const int bad = make_dropout(dropout, rng, &drop);
  if (bad != FP8MI_OK) return bad;
  if (rows * cols == 0) {
    if (!amax && !sat) return FP8MI_OK;
  } else {
    if (!x || !weight || !q || !scale) return FP8MI_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(bias) || !aligned16(sum_out) || !aligned16(q))
      return FP8MI_ERR_ALIGN;
  }
  const int dev = check_device();
  if (dev != FP8MI_OK) return dev;
  return launched(launch_layernorm_quantize(x, residual, weight, bias, xtype, rows, cols, eps, drop, fmt, scale, sum_out,
                                            q, mean, rstd, amax, sat, workspace, workspace_bytes, (hipStream_t)stream));
}

int fp8_layernorm_backward(const void* dy, const void* h, const float* mean, const float* rstd, const void* weight,
                           const void* dresidual, int xtype, int64_t rows, int64_t cols, float dropout,
                           const uint64_t* rng, void* dx, void* dbranch, float* dweight, float* dbias, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!dtype_ok(xtype)) return FP8MI_ERR_DTYPE;
  if (!dims_ok(rows, cols) || cols > kMaxDim) return FP8MI_ERR_SHAPE;
  if ((cols & 15) != 0) return FP8MI_ERR_ALIGN;
  if (workspace && !aligned16(workspace)) return FP8MI_ERR_ALIGN;
  Dropout drop;
  const int bad = make_dropout(dropout, rng, &drop);
  if (bad != FP8MI_OK) return bad;
  const bool sums = dweight || dbias;
  if (rows * cols == 0 && (cols == 0 || !sums)) return FP8MI_OK;
  if (!aligned16(dweight) || !aligned16(dbias)) return FP8MI_ERR_ALIGN;
  if (rows != 0) {
    if (!dy || !h || !mean || !rstd || !weight || !dx) return FP8MI_ERR_NULL;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(dresidual) || !aligned16(dx) || !aligned16(dbranch))
      return FP8MI_ERR_ALIGN;
    if (dbranch && dbranch == dx) return FP8MI_ERR_SHAPE;
    if (sums && !workspace) return FP8MI_ERR_NULL;
    if (sums && workspace_bytes < (size_t)((dweight ? 1 : 0) + (dbias ? 1 : 0)) * cols * sizeof(float)) return FP8MI_ERR_WORKSPACE;
  }
  const int dev = check_device();
  if (dev != FP8MI_OK) return dev;
  return launched(launch_layernorm_backward(dy, h, mean, rstd, weight, dresidual, xtype, rows, cols, drop, dx, dbranch,
                                            dweight, dbias, workspace, workspace_bytes, (hipStream_t)stream));
}

int fp8_embedding(const void* tokens, int itype, int64_t rows, const void* table, int ttype, int64_t vocab, int64_t cols,
                  const float* sinv, float scale, void* out, int otype, void* stream) {
  const bool codes = ttype == FP8MI_OUT_E4M3 || ttype == FP8MI_OUT_E5M2;
  if (!index_ok(itype) || !dtype_ok(otype) || (ttype != FP8MI_OUT_F32 && ttype != FP8MI_OUT_BF16 && !codes)) return FP8MI_ERR_DTYPE;
  if (!dims_ok(rows, cols) || !dims_ok(vocab, cols) || vocab > kMaxDim || cols > kMaxEmbedCols) return FP8MI_ERR_SHAPE;
  if ((cols & 15) != 0) return FP8MI_ERR_ALIGN;
  if (rows * cols == 0) return FP8MI_OK;
  if (!tokens || (vocab && !table) || !out || (codes && !sinv)) return FP8MI_ERR_NULL;
  if (!index_aligned(tokens, itype) || !aligned16(table) || !aligned16(out)) return FP8MI_ERR_ALIGN;
  const int dev = check_device();
  if (dev != FP8MI_OK) return dev;
  return launched(launch_embedding(tokens, itype == FP8MI_I64, rows, table, ttype, vocab, cols, sinv, scale, out, otype, (hipStream_t)stream));
}

size_t fp8mi_embedding_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxTokens || cols > kMaxEmbedCols || (cols & 15) != 0) return 0;
  return embedding_workspace(rows, cols);
}

int fp8_embedding_backward(const void* tokens, int itype, int64_t rows, const void* dy, int dytype, int64_t vocab,
                           int64_t cols, float scale, const void* base, void* dtable, int ttype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!index_ok(itype) || !dtype_ok(dytype) || !dtype_ok(ttype)) return FP8MI_ERR_DTYPE;
  if (!dims_ok(rows, cols) || !dims_ok(vocab, cols) || vocab > kMaxDim || cols > kMaxEmbedCols || rows > kMaxTokens) return FP8MI_ERR_SHAPE;
  if ((cols & 15) != 0) return FP8MI_ERR_ALIGN;
  if (workspace && !aligned16(workspace)) return FP8MI_ERR_ALIGN;
  if (vocab * cols == 0 || (rows == 0 && base == dtable)) return FP8MI_OK;
  if (!dtable || (rows && (!tokens || !dy || !workspace))) return FP8MI_ERR_NULL;
  if (!aligned16(dy) || !aligned16(base) || !aligned16(dtable) || !index_aligned(tokens, itype)) return FP8MI_ERR_ALIGN;
  if (rows && workspace_bytes < embedding_need(rows, cols)) return FP8MI_ERR_WORKSPACE;
  const int dev = check_device();
  if (dev != FP8MI_OK) return dev;
  return launched(launch_embedding_backward(tokens, itype == FP8MI_I64, rows, dy, dytype, vocab, cols, scale, base, dtable, ttype, workspace,
                                            (hipStream_t)stream));
}

size_t fp8mi_vocab_workspace(int64_t M, int64_t V, int64_t K, int64_t pieces) {
  if (check_vocab_sizes(M, V, K) != FP8MI_OK || pieces < 0) return 0;
  return vocab_workspace(M, V, K, pieces);
}

int fp8_vocab_cross_entropy(const uint8_t* x, int fx, const uint8_t* w, int fw, int64_t M, int64_t V, int64_t K,
                            const float* sinv_x, const float* sinv_w, const void* targets, int itype, float* loss,
                            float* lse, int accum, void* workspace, size_t workspace_bytes, void* stream) {
  const int bad = check_vocab(x, fx, w, fw, M, V, K, sinv_x, sinv_w, targets, itype, accum, workspace);
  if (bad != FP8MI_OK) return bad;
  if (M == 0) return FP8MI_OK;
  if (!loss && !lse) return FP8MI_ERR_NULL;
  if (workspace_bytes < vocab_loss_bytes(M, V < kPieceCols ? V : kPieceCols)) return FP8MI_ERR_WORKSPACE;
  const int dev = check_device();
  if (dev != FP8MI_OK) return dev;
  const VocabOperands o{x, w, fx, fw, sinv_x, sinv_w, M, K};
  return launched(launch_vocab_cross_entropy(o, V, Targets{targets, itype == FP8MI_I64}, loss, lse, accum, workspace,
                                             workspace_bytes, (hipStream_t)stream));
}

int fp8_vocab_cross_entropy_backward(const uint8_t* x, int fx, const uint8_t* w, int fw, int64_t M, int64_t V, int64_t K,
                                     const float* sinv_x, const float* sinv_w, const void* targets, int itype,
                                     const float* lse, const float* dloss, int fmt, const float* scale,
                                     const float* scale_inv, void* dx, int dxtype, void* dw, int dwtype, float* amax,
                                     unsigned long long* sat, int accum, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (!fmt_ok(fmt)) return FP8MI_ERR_FORMAT;
  if ((dx && !dtype_ok(dxtype)) || (dw && !dtype_ok(dwtype))) return FP8MI_ERR_DTYPE;
  const int bad = check_vocab(x, fx, w, fw, M, V, K, sinv_x, sinv_w, targets, itype, accum, workspace);
  if (bad != FP8MI_OK) return bad;
  if (!aligned16(dx) || !aligned16(dw)) return FP8MI_ERR_ALIGN;
  if (M == 0) {
    if (!dw && !amax && !sat) return FP8MI_OK;
  } else {
    if (!dx && !dw) return FP8MI_ERR_NULL;
    if (!lse || !dloss || !scale || !scale_inv) return FP8MI_ERR_NULL;
    if (workspace_bytes < vocab_workspace(M, V, K, 0)) return FP8MI_ERR_WORKSPACE;
  }
  const int dev = check_device();
  if (dev != FP8MI_OK) return dev;
  const VocabOperands o{x, w, fx, fw, sinv_x, sinv_w, M, K};
  return launched(launch_vocab_cross_entropy_backward(o, V, Targets{targets, itype == FP8MI_I64}, lse, dloss, fmt, scale,
                                                      scale_inv, dx, dxtype, dw, dwtype, amax, sat, accum, workspace,
                                                      workspace_bytes, (hipStream_t)stream));
}

}  // extern "C"
