// The launches of a call that enqueues several kernels.
#pragma once

#include <hip/hip_ext.h>

#include "exec.h"
#include "launch.h"

namespace ar {

inline RunResult hip_fail(hipError_t e, const char* what) {
  RunResult r;
  r.status = 4;  // AR_HIP_ERROR
  r.hip_error = int(e);
  r.message = std::string(what) + ": " + hipGetErrorString(e);
  (void)hipGetLastError();  // reported here: not left for a later call that asks for the last error
  return r;
}

// The call's launches in order: the first records the start event, the last the stop event. Errors are
// taken from the launch itself, not from the thread's last one, which may be another call's.
template <typename T> struct Same { using type = T; };
struct Sequence {
  hipStream_t st;
  Evs ev;
  int64_t left;
  bool begun = false;
  hipError_t err = hipSuccess;
  template <typename... A> void launch(void (*k)(A...), int64_t blocks, int threads, typename Same<A>::type... a) {
    launch_lds(k, blocks, threads, 0, a...);
  }
  // The same with dynamic LDS.
  template <typename... A> void launch_lds(void (*k)(A...), int64_t blocks, int threads, size_t lds, typename Same<A>::type... a) {
    if (err != hipSuccess) return;
    --left;
    void* args[] = {static_cast<void*>(&a)...};
    err = hipExtLaunchKernel(reinterpret_cast<const void*>(k), dim3(unsigned(blocks)), dim3(unsigned(threads)), args, lds, st,
                             begun ? nullptr : ev.start, left ? nullptr : ev.stop, 0);
    begun = true;
  }
  RunResult done(const char* what) {
    if (err == hipSuccess && !begun) {  // no launch: both events mark this point of the stream
      if (ev.start) err = hipEventRecord(ev.start, st);
      if (err == hipSuccess && ev.stop) err = hipEventRecord(ev.stop, st);
    }
    return err == hipSuccess ? RunResult{} : hip_fail(err, what);
  }
};

}  // namespace ar
