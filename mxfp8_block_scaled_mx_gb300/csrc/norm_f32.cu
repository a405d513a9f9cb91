// norm_f32.cu -- the norm kernels for FP32 blocks on an FP32 stream.
#include "norm_kernel.cuh"

namespace mx {

cudaError_t norm_forward_f32(const NormParams& p, NormRows kind, int num_sms, cudaStream_t stream) {
  return norm_forward_of<float, float>(p, kind, num_sms, stream);
}

cudaError_t norm_backward_f32(const NormBackParams& p, NormRows kind, int64_t n, cudaStream_t stream) {
  return norm_backward_of<float, float>(p, kind, n, stream);
}

}  // namespace mx
