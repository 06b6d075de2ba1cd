// The residual's addition with the norm behind it, and its backward pass from the kept
// sum. The kernels are the norm's (norm_device.cuh) with the addition in front: the
// sum is never read back by the forward pass.
#include "add_norm_bwd.cuh"
#include "model_internal.h"

namespace flce {

int add_norm_partial_rows(int64_t rows, int64_t hidden, int sms) {
  const int64_t most = static_cast<int64_t>(sms) * (bwd_ctas(hidden) > kMostAddCtas ? bwd_ctas(hidden) : kMostAddCtas);
  return static_cast<int>(rows < most ? rows : most);
}

cudaError_t launch_add_norm(const AddNormParams& p, int sms, cudaStream_t s) {
  if (p.dtype == FLCE_DTYPE_F32) return vectors(p) ? run_fwd<float, 4, kAdd>(p, sms, s) : run_fwd<float, 1, kAdd>(p, sms, s);
  return vectors(p) ? run_fwd<uint16_t, 8, kAdd>(p, sms, s) : run_fwd<uint16_t, 1, kAdd>(p, sms, s);
}

cudaError_t launch_add_norm_bwd(const AddNormParams& p, int sms, int* partials, cudaStream_t s) {
  if (wide_rows(p)) return p.dtype == FLCE_DTYPE_F32 ? run_wide_bwd<float, false>(p, sms, partials, s) : run_wide_bwd<uint16_t, false>(p, sms, partials, s);
  return p.dtype == FLCE_DTYPE_F32 ? launch_bwd<float, 4, kAdd>(p, sms, partials, s) : launch_bwd<uint16_t, 8, kAdd>(p, sms, partials, s);
}

}  // namespace flce
