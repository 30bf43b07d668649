// The global norm of many gradients and their clipping: list and launcher.
#pragma once

#include "ep_internal.cuh"

namespace ep {

// Host arrays of `count` entries; outs may be NULL (the norm only).
struct GradList {
  int count;
  const void *const *grads;
  void *const *outs;
  const int64_t *numels;
  const uint8_t *is_f32;
};

// Bytes of workspace; 0: one cluster does it all, and launch_clip's is NULL.
size_t clip_workspace(const GradList &l, int sms);
cudaError_t launch_clip(const GradList &l, float max_norm, float *norm, void *workspace, int sms,
                        cudaStream_t s);

}  // namespace ep
