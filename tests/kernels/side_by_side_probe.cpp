// Test-only program: the two-stream part of a mixed step (pa_fork.cuh) over stand-ins of
// the CUDA calls it makes.  argv[1] names the step that fails ("none", "start", "wait",
// "aside", "here", "done", "join"); every step that is reached is printed.
#include <cstdio>
#include <cstring>

#include "pa_fork.cuh"

static const char* failing = "none";
static bool step(const char* name) {
  std::puts(name);
  return std::strcmp(name, failing) != 0;
}
static const cudaStream_t kMain = (cudaStream_t)16, kSide = (cudaStream_t)32;
static const cudaEvent_t kStart = (cudaEvent_t)48, kDone = (cudaEvent_t)64;

extern "C" cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t s) {
  const char* name = e == kStart && s == kMain ? "start" : e == kDone && s == kSide ? "done" : "?";
  return step(name) ? cudaSuccess : cudaErrorUnknown;
}
extern "C" cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned int) {
  const char* name = e == kStart && s == kSide ? "wait" : e == kDone && s == kMain ? "join" : "?";
  return step(name) ? cudaSuccess : cudaErrorUnknown;
}

int main(int, char** argv) {
  failing = argv[1];
  pa::ForkStreams f;
  f.side = kSide;
  f.start = kStart;
  f.done = kDone;
  const bool ok = pa::side_by_side(
      f, kMain, [](cudaStream_t s) { return step(s == kSide ? "aside" : "?"); },
      [] { return step("here"); });
  std::puts(ok ? "true" : "false");
  return 0;
}
