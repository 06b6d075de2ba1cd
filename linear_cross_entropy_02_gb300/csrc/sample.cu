// One token per row of logits: temperature, top-k, top-p, min-p, and the inverse
// of the kept tokens' distribution function at a given random number.
// (The kernels: sample_device.cuh.)
#include "sample_device.cuh"

namespace flce {

cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t s) {
  return p.dtype == FLCE_DTYPE_F32 ? run_typed<float, false>(p, sms, s) : run_typed<uint16_t, false>(p, sms, s);
}

}  // namespace flce
