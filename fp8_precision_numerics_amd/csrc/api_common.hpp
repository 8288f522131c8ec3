// Limits and checks that the entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8mi.h"

namespace fp8mi {

constexpr int64_t kMaxDim = 0x7FFFFFFF;             // kernels index rows/cols with 32-bit ints
constexpr int64_t kMaxGemmK = int64_t(1) << 23;     // 256 rows x K bytes of a tile slab in a 32-bit buffer offset
constexpr int64_t kMaxGroupedK = int64_t(1) << 22;  // 512 rows x K bytes (the grouped kernels' widest slab)
constexpr int64_t kMaxBufferBytes = 0x7FFFFFFF;     // any offset a buffer load carries in one 32-bit register
constexpr int64_t kMaxBackCols = int64_t(1) << 25;  // 16 rows of d in a 32-bit byte offset (fp32)
constexpr int64_t kMaxElems = (int64_t)1 << 40;     // sanity bound on any one tensor

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool fmt_ok(int f) { return f == FP8MI_E4M3 || f == FP8MI_E5M2; }
inline bool dtype_ok(int d) { return d == FP8MI_F32 || d == FP8MI_BF16; }
inline bool accum_ok(int a) { return a == FP8MI_ACCUM_EXACT || a == FP8MI_ACCUM_MFMA_FP8; }

inline bool act_ok(int a) { return a == FP8MI_ACT_NONE || a == FP8MI_ACT_RELU || a == FP8MI_ACT_SILU || a == FP8MI_ACT_GELU; }

// FP8MI_OK where a gfx950 is current.
int check_device();

inline int launched(hipError_t e) { return e == hipSuccess ? FP8MI_OK : FP8MI_ERR_LAUNCH; }

inline bool dims_ok(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxElems || cols > kMaxElems) return false;
  if (rows != 0 && cols > kMaxElems / rows) return false;
  return true;
}

}  // namespace fp8mi
