// Host-side declarations shared by the translation units that implement entry points.
#pragma once

#include "ep_internal.cuh"

struct ep_handle {
  ep_config cfg;
  int device;
  cudaStream_t stream;
  void *dmem;
  ep::LayoutParams lp;
  int64_t rows_alloc;
  int64_t sf_hidden_stride, sf_token_stride, sf_numel, sf_expert_stride;
  float *tok_scale;
};

namespace ep {

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

ep_status cuda_status(cudaError_t e);

// EP_OK if the current device is the handle's.
ep_status check_device(const ep_handle *h);

// The device's memory pool for handles and workspaces (kept until exit).
cudaError_t handle_pool(int device, cudaMemPool_t *out);

// Workspace of one call, stream-ordered on s: from the device's pool, or a
// graph memory node while s is being captured.
cudaError_t workspace_alloc(size_t bytes, cudaStream_t s, void **out);
cudaError_t workspace_free(void *p, cudaStream_t s);

}  // namespace ep
