// extern "C" entry points of the operators at both ends of a model: argument
// validation and dispatch, as api.hip.
#include <cmath>

#include "api_common.hpp"
#include "device_common.hpp"
#include "model_ends.hpp"

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

}  // extern "C"
