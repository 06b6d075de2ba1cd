// The residual's addition with the norm behind it, and its backward pass from the kept
// sum. The kernels are the norm's (norm_device.cuh) with the addition in front: the
// sum is never read back by the forward pass.
#include "model_internal.h"
#include "norm_device.cuh"

namespace flce {

cudaError_t launch_add_norm(const NormParams& p, int sms, cudaStream_t s) {
  if (p.dtype == FLCE_DTYPE_F32) return vectors(p) ? run_fwd<float, 4, kAdd>(p, sms, s) : run_fwd<float, 1, kAdd>(p, sms, s);
  return vectors(p) ? run_fwd<uint16_t, 8, kAdd>(p, sms, s) : run_fwd<uint16_t, 1, kAdd>(p, sms, s);
}

cudaError_t launch_add_norm_bwd(const NormParams& p, int sms, int* partials, cudaStream_t s) {
  return p.dtype == FLCE_DTYPE_F32 ? launch_bwd<float, 4, kAdd>(p, sms, partials, s) : launch_bwd<uint16_t, 8, kAdd>(p, sms, partials, s);
}

}  // namespace flce
