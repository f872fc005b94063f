// elmo_operators.h -- launchers of the scoring operators: 4-bit copies of a
// head and log probabilities of labels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/elmo.h"

struct elmo_head;

namespace elmo {

// The dynamic shared memory a kernel may have, set once on a device: `seen`
// (one a kernel) has a bit for each device.
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& seen) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (seen.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) seen.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch that may start before the kernel ahead of it in the stream has
// ended; the kernel waits for that (griddepcontrol.wait) before it touches
// what earlier kernels write.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// SMs of the current device (one where it cannot be asked).
inline int current_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  return n;
}

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
