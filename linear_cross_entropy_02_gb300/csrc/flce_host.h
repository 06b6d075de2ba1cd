// Host-side services of the engine that every entry point uses: the launch
// counter with its optional timing, the per-device cache, the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "flce_head.h"

namespace flce {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr int kMaxDevices = 64;

// Counts one launch, and times it with events while profiling is on.
struct LaunchScope {
  int kernel;
  cudaStream_t stream;
  cudaEvent_t start = nullptr, stop = nullptr;
  LaunchScope(int k, cudaStream_t s);
  ~LaunchScope();
};

#define FLCE_LAUNCH(kid, expr)                         \
  do {                                                 \
    LaunchScope _scope((kid), stream);                 \
    if ((expr) != cudaSuccess) return FLCE_ERR_CUDA;   \
  } while (0)

// SM count and compute capability (10 * major + minor) of the current device.
int device_info(int* sms, int* cc);

// cuTensorMapEncodeTiled, looked up by load_encoder() (false: not available).
extern PFN_cuTensorMapEncodeTiled_v12000 g_encode;
bool load_encoder();

}  // namespace flce
