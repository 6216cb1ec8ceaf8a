// Arguments of the gated recurrence's kernels (scan.cu).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

namespace va {

struct ScanParams {
  const void* x;       // forward: x; backward: dh
  const void* g;       // log decay
  const void* h;       // backward: the forward's h
  void* out;           // forward: h; backward: dx
  void* dg;            // backward
  int64_t x_rs, g_rs, h_rs, out_rs, dg_rs;  // row strides (elements)
  const int32_t* cu;
  const float* h0;     // [B, D] contiguous, may be null
  const float* dlast;  // backward: gradient of the last states, may be null
  float* last;         // forward: the last states; backward: h0's gradient; may be null
  int B, T, D;
  int tiles, cols;     // tiles of rows, columns of channels (set by the launcher)
  struct WsHeader* hdr;  // workspace header (single tokens: may be null)
  int32_t* ticket;
  int32_t* record;     // [tiles][8] what is known of a tile's segments
  float* agg;          // [tiles][cols * width][2] a tile's map (decay product, state from zero)
  uint64_t wait_ns;    // test hook: tile 0 publishes nothing and waits give up after this; 0: none
  float* carry;        // [groups][cols * width] the state after a group of tiles
};

size_t scan_workspace(int T, int D);
// stage 0: boundary check, empty places and look-ups, 1: the recurrence.  dtypes: 0 fp32, 1 bf16 (h: bf16 only where both are).
cudaError_t launch_scan_fwd(int stage, ScanParams p, int x_bf16, int g_bf16, int h_bf16, void* ws, cudaStream_t st);
cudaError_t launch_scan_bwd(int stage, ScanParams p, int x_bf16, int g_bf16, int h_bf16, void* ws, cudaStream_t st);
// The forward of single tokens (T == B): every state moves on by one step.  One launch.
cudaError_t launch_scan_step(ScanParams p, int x_bf16, int g_bf16, int h_bf16, void* ws, cudaStream_t st);

}  // namespace va
