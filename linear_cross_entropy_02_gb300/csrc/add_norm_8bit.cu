// Backward pass of the norm from an 8-bit checkpoint of what it normalised
// (norm_device.cuh, checkpoint_device.cuh).
#include "add_norm_bwd.cuh"
#include "model_internal.h"

namespace flce {

cudaError_t launch_add_norm_bwd_8bit(const AddNormParams& p, int sms, int* partials, cudaStream_t s) {
  if (wide_rows(p)) return p.dtype == FLCE_DTYPE_F32 ? run_wide_bwd<float, true>(p, sms, partials, s) : run_wide_bwd<uint16_t, true>(p, sms, partials, s);
  return p.dtype == FLCE_DTYPE_F32 ? launch_bwd<float, 4, kAdd8>(p, sms, partials, s) : launch_bwd<uint16_t, 8, kAdd8>(p, sms, partials, s);
}

}  // namespace flce
