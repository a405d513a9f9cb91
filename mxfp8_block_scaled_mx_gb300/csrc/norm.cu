// norm.cu -- the norms before and after a block, with its gate and residual
// scale, and their gradients.
//
//   res_out = alpha * residual + g * n(block; w_post),  y = n(res_out; w_pre)
//   n(v; w)_c = v_c w_c / sqrt(mean(v^2) + eps)
//
// First form: one block of threads per row, three passes over the row; the
// gradient keeps four numbers per row, from which a second kernel forms the
// column sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load(const void* p, int32_t f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void store(void* p, int32_t f32, int64_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Sum over the block of threads, the same in every thread.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane_id() == 0) part[warp_id()] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) v += part[i];
  return v;
}

__global__ void __launch_bounds__(kThreads) norm_residual_kernel(const NormParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const float cols = static_cast<float>(p.cols);
  const int64_t grow = p.gate ? t / (p.rows / p.gates) * p.cols : 0;
  float scale = 1.f;
  if (p.w_post) {
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      const float b = load(p.block, p.c_fp32, t * p.ldb + c);
      s += b * b;
    }
    scale = 1.f / sqrtf(block_sum(s) / cols + p.eps);
  }
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
    float n = load(p.block, p.c_fp32, t * p.ldb + c) * scale;
    if (p.w_post) n *= load(p.w_post, p.w_fp32, c);
    if (p.gate) n *= load(p.gate, p.w_fp32, grow + c);
    float r = p.alpha * load(p.residual, p.s_fp32, t * p.ldr + c) + n;
    store(p.res_out, p.s_fp32, t * p.ldo + c, r);
    if (!p.s_fp32) r = __bfloat162float(__float2bfloat16_rn(r));
    s += r * r;
  }
  const float rho = 1.f / sqrtf(block_sum(s) / cols + p.eps);
  for (int64_t c = threadIdx.x; c < p.cols; c += kThreads)
    store(p.y, p.c_fp32, t * p.ldy + c,
          load(p.res_out, p.s_fp32, t * p.ldo + c) * rho * load(p.w_pre, p.w_fp32, c));
}

// Row t's numbers: rho, rho^3 mean(w_pre dy r), sigma, sigma^3 mean(w_post u b).
__device__ __forceinline__ float grad_d(const NormBackParams& p, int64_t t, int64_t c, float rho,
                                        float k) {
  const float r = load(p.res_out, p.s_fp32, t * p.ldr + c);
  const float dy = load(p.dy, p.c_fp32, t * p.lddy + c);
  const float d = p.d_res ? load(p.d_res, p.s_fp32, t * p.ldd + c) : 0.f;
  return d + rho * load(p.w_pre, p.w_fp32, c) * dy - r * k;
}

__global__ void __launch_bounds__(kThreads) norm_back_rows_kernel(const NormBackParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const float cols = static_cast<float>(p.cols);
  const int64_t grow = p.gate ? t / (p.rows / p.gates) * p.cols : 0;
  float s = 0.f, q = 0.f;
  for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
    const float r = load(p.res_out, p.s_fp32, t * p.ldr + c);
    s += r * r;
    q += load(p.w_pre, p.w_fp32, c) * load(p.dy, p.c_fp32, t * p.lddy + c) * r;
  }
  const float rho = 1.f / sqrtf(block_sum(s) / cols + p.eps);
  // in this order nothing leaves FP32's range before the product does
  const float k = rho * (rho * (rho * (block_sum(q) / cols)));
  float sigma = 1.f, j = 0.f;
  if (p.w_post) {
    s = q = 0.f;
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      const float b = load(p.block, p.c_fp32, t * p.ldb + c);
      float u = grad_d(p, t, c, rho, k) * load(p.w_post, p.w_fp32, c);
      if (p.gate) u *= load(p.gate, p.w_fp32, grow + c);
      s += b * b;
      q += u * b;
    }
    sigma = 1.f / sqrtf(block_sum(s) / cols + p.eps);
    j = sigma * (sigma * (sigma * (block_sum(q) / cols)));
  }
  float* row = p.workspace + t * 4;
  if (threadIdx.x == 0) {
    row[0] = rho;
    row[1] = k;
    row[2] = sigma;
    row[3] = j;
  }
  for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
    const float d = grad_d(p, t, c, rho, k);
    const float b = load(p.block, p.c_fp32, t * p.ldb + c);
    float u = d * sigma;
    if (p.w_post) u *= load(p.w_post, p.w_fp32, c);
    if (p.gate) u *= load(p.gate, p.w_fp32, grow + c);
    store(p.d_block, p.c_fp32, t * p.lddb + c, u - b * j);
    p.d_copy[t * p.cols + c] = d;
  }
}

// Column sums in row order, one thread per column; then alpha D.
__global__ void __launch_bounds__(kThreads) norm_back_cols_kernel(const NormBackParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= p.cols) return;
  const float wpost = p.w_post ? load(p.w_post, p.w_fp32, c) : 1.f;
  const int64_t gates = p.gate ? p.gates : 1;
  const int64_t per = p.rows / gates;
  float s_pre = 0.f, s_post = 0.f;
  for (int64_t g = 0; g < gates; ++g) {
    float sum = 0.f;
    for (int64_t t = g * per; t < (g + 1) * per; ++t) {
      const float* row = p.workspace + t * 4;
      const float d = p.d_copy[t * p.cols + c];
      s_pre += load(p.dy, p.c_fp32, t * p.lddy + c) * load(p.res_out, p.s_fp32, t * p.ldr + c) * row[0];
      sum += d * load(p.block, p.c_fp32, t * p.ldb + c) * row[2];
      store(p.d_residual, p.s_fp32, t * p.lddr + c, p.alpha * d);
    }
    if (p.gate) {
      if (p.d_gate) p.d_gate[g * p.cols + c] = sum * wpost;
      sum *= load(p.gate, p.w_fp32, g * p.cols + c);
    }
    s_post += sum;
  }
  p.d_w_pre[c] = s_pre;
  if (p.d_w_post) p.d_w_post[c] = s_post;
}

template <typename K, typename P>
cudaError_t launch(K kern, unsigned grid, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

size_t norm_backward_workspace(int64_t rows, int64_t cols, int64_t gates) {
  (void)gates;
  return static_cast<size_t>(rows) * (16 + static_cast<size_t>(cols) * 4);
}

cudaError_t launch_norm_residual(const NormParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  return launch(norm_residual_kernel, static_cast<unsigned>(p.rows), p, stream);
}

cudaError_t launch_norm_residual_backward(const NormBackParams& p, int num_sms,
                                          cudaStream_t stream) {
  (void)num_sms;
  NormBackParams q = p;
  q.d_copy = p.workspace + p.rows * 4;
  if (p.rows > 0) {
    const cudaError_t err =
        launch(norm_back_rows_kernel, static_cast<unsigned>(p.rows), q, stream);
    if (err != cudaSuccess) return err;
  }
  return launch(norm_back_cols_kernel,
                static_cast<unsigned>((p.cols + kThreads - 1) / kThreads), q, stream);
}

}  // namespace mx
