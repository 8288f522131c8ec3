// Internal launchers of the operators at both ends of a model (layer norm, vocabulary
// cross entropy, embedding), as those of launch.hpp: arguments are validated by
// api_model_ends.hip, each launcher only enqueues kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "philox.hpp"

namespace fp8mi {

hipError_t launch_layernorm_quantize(const void* x, const void* residual, const void* weight, const void* bias, int xtype,
                                     int64_t rows, int64_t cols, float eps, const Dropout& drop, int fmt,
                                     const float* scale, void* sum_out, uint8_t* q, float* mean, float* rstd,
                                     float* amax, unsigned long long* sat, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream);

hipError_t launch_layernorm_backward(const void* dy, const void* h, const float* mean, const float* rstd,
                                     const void* weight, const void* dres, int xtype, int64_t rows, int64_t cols,
                                     const Dropout& drop, void* dx, void* dbranch, float* dweight, float* dbias,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream);

}  // namespace fp8mi
