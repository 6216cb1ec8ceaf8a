// Arguments of the token log-probability kernels (logprobs.cu).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

namespace va {

constexpr int kMaxTop = 128;  // alternatives per token

struct LogprobParams {
  const void* z;  // logits [T, V]
  int64_t z_rs;
  const int32_t* tok;
  int T, V, ignore, k;
  float temperature;
  float scale, scale_lo;  // log2(e) / temperature, and what its rounding leaves
  float inv_t, inv_c;     // 1 / temperature, 1 / scale
  float* logprob; // [T]
  float* entropy; // [T]
  float* lse;     // [T]
  int32_t* top_ids;    // [T, k]
  float* top_logprobs; // [T, k]
  // backward
  const float* dlogprob;  // [T]
  const float* dentropy;  // [T], may be null
  void* grad;
  int64_t g_rs;
  int32_t* status;  // forward: set to VA_ERR_BAD_TARGETS, never cleared; may be null
  int slices;       // backward: blocks that share a row (set by the launcher)
};

cudaError_t launch_logprobs_fwd(LogprobParams p, int bf16, cudaStream_t st);
cudaError_t launch_logprobs_bwd(LogprobParams p, int bf16, cudaStream_t st);

}  // namespace va
