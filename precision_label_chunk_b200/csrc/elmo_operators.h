// elmo_operators.h -- launchers of the scoring operators: 4-bit copies of a
// head and log probabilities of labels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/elmo.h"

struct elmo_head;

namespace elmo {

// q4.cu
cudaError_t launch_q4_pack(const void* W, int64_t L, int32_t d, int w_format, int32_t group, uint8_t* codes,
                           uint16_t* scales, cudaStream_t s);
cudaError_t launch_q4_unpack(const uint8_t* codes, const uint16_t* scales, int64_t L, int32_t d, int32_t group,
                             uint16_t* W, cudaStream_t s);
cudaError_t launch_q4_scores(const uint8_t* codes, const uint16_t* scales, int64_t L, int32_t d, int32_t group,
                             const uint16_t* X, int32_t B, float* Z, int64_t ldz, cudaStream_t s);

// logprob.cu
size_t score_logprobs_workspace(int32_t B, int64_t L, int32_t k);
cudaError_t launch_score_logprobs(const void* Z, bool bf16, int64_t ldz, int32_t B, int64_t L, const int32_t* rowptr,
                                  const int32_t* cols, int32_t nnz, int32_t k, float* logp, float* lse, float* entropy,
                                  int32_t* top_idx, float* top_logp, void* work, cudaStream_t s);
cudaError_t launch_score_backward(const void* Z, bool bf16, int64_t ldz, int32_t B, int64_t L, const int32_t* rowptr,
                                  const int32_t* cols, int32_t nnz, const float* lse, const float* entropy,
                                  const float* g_logp, const float* g_lse, const float* g_entropy, void* dZ,
                                  int64_t lddz, cudaStream_t s);

// label_logprobs.cu
size_t label_logprobs_workspace(const elmo_head* h, int32_t B, int32_t k);
cudaError_t launch_label_logprobs(elmo_head* h, const uint16_t* X, int32_t B, const int32_t* rowptr,
                                  const int32_t* cols, int32_t nnz, int32_t k, float* logp, float* lse, float* entropy,
                                  int32_t* top_idx, float* top_logp, void* work, cudaStream_t s);

}  // namespace elmo
