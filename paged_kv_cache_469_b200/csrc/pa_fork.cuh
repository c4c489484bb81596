// pa_fork.cuh -- two pieces of a call's work side by side, on the caller's stream and on
// one of the library's own.
#pragma once

#include <cuda_runtime_api.h>

namespace pa {

// A side stream and two events, per thread and device, for the calls that run
// the prefill kernel beside the decode kernel.  Created on the first such call
// outside a stream capture; a capture that would need to create them runs the
// kernels one after the other instead, and so does a call on any other stream
// while the side stream is part of a capture.
struct ForkStreams {
  cudaStream_t side = nullptr;
  cudaEvent_t start = nullptr, done = nullptr;
};
ForkStreams* fork_streams(cudaStream_t st);

// aside(stream) queues work on the side stream, behind what `st` holds; here() the rest
// on `st`.  Each says whether it could.  Whatever fails, `st` waits for what the side
// stream was given: the buffers are the caller's again in the order of its own stream,
// and a capture is joined.
template <typename Aside, typename Here>
bool side_by_side(const ForkStreams& f, cudaStream_t st, Aside aside, Here here) {
  if (cudaEventRecord(f.start, st) != cudaSuccess ||
      cudaStreamWaitEvent(f.side, f.start, 0) != cudaSuccess)
    return false;
  const bool queued = aside(f.side) && here();
  const bool joined = cudaEventRecord(f.done, f.side) == cudaSuccess &&
                      cudaStreamWaitEvent(st, f.done, 0) == cudaSuccess;
  return queued && joined;
}

}  // namespace pa
