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

// `wide`: int64 tokens, else int32.  Table types: an fp8mi_output.
hipError_t launch_embedding(const void* tokens, bool wide, int64_t rows, const void* table, int ttype, int64_t vocab,
                            int64_t cols, const float* sinv, float scale, void* out, int otype, hipStream_t stream);

hipError_t launch_embedding_backward(const void* tokens, bool wide, int64_t rows, const void* dy, int dytype,
                                     int64_t vocab, int64_t cols, float scale, const void* base, void* dtable,
                                     int ttype, void* workspace, hipStream_t stream);

// `words` of 16 bytes from base, or of zeros without one.
hipError_t launch_fill_rows(const void* base, void* to, int64_t words, hipStream_t stream);

struct VocabOperands;  // vocab.hpp
struct Targets;        // vocab_epilogue.hpp

hipError_t launch_vocab_cross_entropy(const VocabOperands& o, int64_t V, const Targets& targets, float* loss, float* lse,
                                      int accum, void* workspace, size_t workspace_bytes, hipStream_t stream);

hipError_t launch_vocab_cross_entropy_backward(const VocabOperands& o, int64_t V, const Targets& targets, const float* lse,
                                               const float* dloss, int fmt, const float* scale, const float* scale_inv,
                                               void* dx, int dxtype, void* dw, int dwtype, float* amax,
                                               unsigned long long* sat, int accum, void* workspace,
                                               size_t workspace_bytes, hipStream_t stream);

}  // namespace fp8mi
