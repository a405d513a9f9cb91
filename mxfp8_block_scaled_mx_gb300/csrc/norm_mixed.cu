// norm_mixed.cu -- the norm kernels for bf16 blocks on an FP32 stream.
#include "norm_kernel.cuh"

namespace mx {

cudaError_t norm_forward_mixed(const NormParams& p, NormRows kind, int num_sms, cudaStream_t stream) {
  return norm_forward_of<bf16, float>(p, kind, num_sms, stream);
}

cudaError_t norm_backward_mixed(const NormBackParams& p, NormRows kind, int64_t n, cudaStream_t stream) {
  return norm_backward_of<bf16, float>(p, kind, n, stream);
}

}  // namespace mx
