// Layer norm and RMS norm in front of the head (the kernels: norm_device.cuh).
#include "norm_device.cuh"

namespace flce {

namespace {

// 32 columns per CTA, 32 threads on each: thread k takes partial rows k, k + 32, ...
// and the 32 sums are added in order.
__global__ void __launch_bounds__(1024) norm_wgrad_kernel(const float* part_w, const float* part_b, int partials,
                                                          int64_t hidden, float* grad_w, float* grad_b,
                                                          int accumulate) {
  __shared__ float s[32][33];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* grad = blockIdx.y == 0 ? grad_w : grad_b;
  if (grad == nullptr) return;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.f;
  if (col < hidden) {
#pragma unroll 8
    for (int i = threadIdx.y; i < partials; i += 32) v += part[i * hidden + col];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && col < hidden) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
    grad[col] = accumulate ? grad[col] + a : a;
  }
}

}  // namespace


int norm_partial_rows(int64_t rows, int64_t hidden, int sms) {
  const int64_t most = static_cast<int64_t>(sms) * bwd_ctas(hidden);
  return static_cast<int>(rows < most ? rows : most);
}

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t s) {
  if (p.dtype == FLCE_DTYPE_F32) return vectors(p) ? run_fwd<float, 4, kPlain>(p, sms, s) : run_fwd<float, 1, kPlain>(p, sms, s);
  return vectors(p) ? run_fwd<uint16_t, 8, kPlain>(p, sms, s) : run_fwd<uint16_t, 1, kPlain>(p, sms, s);
}

cudaError_t launch_norm_bwd(const NormParams& p, int sms, int* partials, cudaStream_t s) {
  return p.dtype == FLCE_DTYPE_F32 ? launch_bwd<float, 4, kPlain>(p, sms, partials, s) : launch_bwd<uint16_t, 8, kPlain>(p, sms, partials, s);
}

cudaError_t launch_norm_wgrad(const float* part_w, const float* part_b, int partials, int64_t hidden, float* grad_w,
                              float* grad_b, int accumulate, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((hidden + 31) / 32), grad_b ? 2 : 1);
  norm_wgrad_kernel<<<grid, dim3(32, 32), 0, s>>>(part_w, part_b, partials, hidden, grad_w, grad_b, accumulate);
  return cudaGetLastError();
}

}  // namespace flce
