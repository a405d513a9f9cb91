// rotate_back.cu -- their gradient of bf16 heads, its workspace and the choice by type (rotate_kernel.cuh).
#include "rotate_kernel.cuh"

namespace mx {

size_t norm_rotate_backward_workspace(int64_t tokens, int64_t dim) {
  return tokens > 0 ? static_cast<size_t>(kBackBlocks * 2 * dim * sizeof(float)) : 0;
}

cudaError_t launch_norm_rotate_backward(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return p.x_fp32 ? launch_norm_rotate_backward_f32(p, num_sms, stream)
                  : by_layout<bf16, true>(p, num_sms, stream);
}

}  // namespace mx
