// rotate_f32.cu -- the heads' norms with rotation of FP32 heads (rotate_kernel.cuh).
#include "rotate_kernel.cuh"

namespace mx {

cudaError_t launch_norm_rotate_f32(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return by_layout<float, false>(p, num_sms, stream);
}

}  // namespace mx
