// Gradient norms and clipping (implemented in grad.hip).
#pragma once

#include "exec.h"

namespace ar {

enum Norm : int32_t { N_L2 = 0, N_MAX = 1 };

// One gradient tensor; arguments have been validated.
struct Grad {
  const void* data;
  void* out;  // data itself for clipping in place
  int64_t n;
  int32_t dtype, out_dtype;
};

// What the norm is, where it goes and how far the gradient is scaled.
struct Clip {
  int32_t norm = N_L2;
  float max_norm = 0, eps = 0;
  float* total = nullptr;        // device: the norm
  float* each = nullptr;         // device: every tensor's or bucket's own norm, or null
  const float* known = nullptr;  // device: a norm to clip by instead of computing one
  void* workspace = nullptr;     // device scratch, or null for the library's
  size_t workspace_bytes = 0;
  void* start_event = nullptr;
  void* stop_event = nullptr;
};

// Enqueue the norm (scale == false), or the norm and the scaling, of `count` tensors.
RunResult run_grad(const Grad* grads, int64_t count, const Clip& clip, bool scale, void* stream);
size_t grad_workspace(const Grad* grads, int64_t count, const Clip& clip);

// P rank buffers per bucket: bufs[b * P + p] holds n[b] elements.
struct Buckets {
  void* const* bufs;
  const int64_t* n;
  int64_t count;
  int32_t P, dtype, op, coll;
};
RunResult run_allreduce_clip(const Buckets& b, const Clip& clip, void* stream);
size_t allreduce_clip_workspace(const Buckets& b, const Clip& clip);

// Workspaces kept for calls that bring none (one per device and stream).
struct GradCache {
  int64_t live = 0, retired = 0, bytes = 0;
};
GradCache grad_cache();
RunResult grad_cache_wait();  // synchronize every device they belong to
void grad_cache_free();       // after that

}  // namespace ar
