// Arguments of the query / key norm kernels (qk_norm.cu).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

namespace va {

constexpr int kQkMaxDim = 256;     // elements of a head
constexpr int kQkMaxBlocks = 1216; // rows of partial weight gradients a workspace holds

struct QkParams {
  const void* x[2];   // queries, keys
  const void* dy[2];  // backward: the outputs' gradients
  void* y[2];         // outputs, or the inputs' gradients
  int64_t x_rs[2], x_hs[2], dy_rs[2], dy_hs[2], y_rs[2], y_hs[2];  // row and head strides (elements)
  const void* w[2];   // weights [d], may be null
  void* dw[2];        // their gradients, may be null
  const float* inv_freq;  // [rot / 2]
  const int32_t* pos;     // [T]
  float* part;            // [blocks][2][d], null when no weight gradient is wanted
  int T, H[2], d, rot, w_bf16, interleaved;
  float eps;
  int G;                  // set by the launchers: lanes per head
};

size_t qk_norm_bwd_workspace(int d);
cudaError_t launch_qk_norm_fwd(QkParams p, int bf16, cudaStream_t st);
cudaError_t launch_qk_norm_bwd(int stage, QkParams p, int bf16, cudaStream_t st);

}  // namespace va
