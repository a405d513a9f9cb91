// rotate.cu -- the heads' norms with rotation of bf16 heads, and the choice by type (rotate_kernel.cuh).
#include "rotate_kernel.cuh"

namespace mx {

cudaError_t launch_norm_rotate(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return p.x_fp32 ? launch_norm_rotate_f32(p, num_sms, stream)
                  : by_layout<bf16, false>(p, num_sms, stream);
}

}  // namespace mx
