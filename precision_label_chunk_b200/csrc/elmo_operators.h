// elmo_operators.h -- launchers of the scoring operators: 4-bit copies of a
// head and log probabilities of labels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/elmo.h"

namespace elmo {

// q4.cu
cudaError_t launch_q4_pack(const void* W, int64_t L, int32_t d, int w_format, int32_t group, uint8_t* codes,
                           uint16_t* scales, cudaStream_t s);
cudaError_t launch_q4_unpack(const uint8_t* codes, const uint16_t* scales, int64_t L, int32_t d, int32_t group,
                             uint16_t* W, cudaStream_t s);
cudaError_t launch_q4_scores(const uint8_t* codes, const uint16_t* scales, int64_t L, int32_t d, int32_t group,
                             const uint16_t* X, int32_t B, float* Z, int64_t ldz, cudaStream_t s);

}  // namespace elmo
