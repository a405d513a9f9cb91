// norm.cu -- the norms around a block: the choice of kernels by type, the
// kernels for bf16 blocks on a bf16 stream, and the joining of the gradient's
// column sums.
#include "norm_kernel.cuh"

namespace mx {

cudaError_t norm_forward_mixed(const NormParams& p, bool vec, int num_sms, cudaStream_t stream);
cudaError_t norm_forward_f32(const NormParams& p, bool vec, int num_sms, cudaStream_t stream);
cudaError_t norm_backward_mixed(const NormBackParams& p, bool vec, int64_t n, cudaStream_t stream);
cudaError_t norm_backward_f32(const NormBackParams& p, bool vec, int64_t n, cudaStream_t stream);

namespace {

constexpr int kSumCols = 32, kSumParts = 32;

// Sums the blocks' parts: job 0 w_pre, job 1 w_post, then the gates whose rows
// several blocks share.  A block takes 32 columns; 32 runs of consecutive
// parts are summed in order side by side, then joined in order.
__global__ void __launch_bounds__(kSumCols* kSumParts)
    norm_backward_sum_kernel(const NormBackParams p, uint32_t n) {
  __shared__ float part[kSumParts][kSumCols + 1];
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t job = blockIdx.y;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kSumCols + threadIdx.x % kSumCols;
  const uint32_t run = threadIdx.x / kSumCols;
  const RowShare share(static_cast<uint32_t>(p.rows), n);
  uint32_t first = 0, count = n, group = 0, per = 0;
  float* out;
  if (job == 0) {
    out = p.d_w_pre;
  } else if (job == 1) {
    if (!p.w_post) return;
    out = p.d_w_post;
  } else {
    per = static_cast<uint32_t>(p.rows / p.gates);
    // the gates themselves, or the gate at the start of each block's rows
    group = p.gates <= n ? job - 2 : share.start(job - 1) / per;
    if (group >= p.gates) return;
    first = share.of(group * per);
    count = share.of((group + 1) * per - 1) - first + 1;
    if (count == 1 || (p.gates > n && first != job - 2)) return;
    out = p.d_gate + group * p.cols;
  }
  float s = 0.f;
  if (col < p.cols) {
    const uint32_t begin = static_cast<uint32_t>(static_cast<uint64_t>(count) * run / kSumParts);
    const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(count) * (run + 1) / kSumParts);
    const float* src;
    int64_t step = p.cols;
    if (job == 0) {
      src = ws_pre(p, first);
    } else if (job == 1) {
      src = ws_post(p, n, first);
    } else {
      // blocks after the first begin inside this gate: their first slot
      src = ws_gate(p, n, 2 * static_cast<int64_t>(first));
      step = 2 * p.cols;
    }
    src += col;
    if (job >= 2 && begin == 0 && end > 0 && share.start(first) < group * per) {
      s = src[p.cols];
      for (uint32_t i = 1; i < end; ++i) s += src[i * step];
    } else {
#pragma unroll 8
      for (uint32_t i = begin; i < end; ++i) s += src[i * step];
    }
  }
  part[run][threadIdx.x % kSumCols] = s;
  __syncthreads();
  if (run == 0 && col < p.cols) {
#pragma unroll
    for (int i = 1; i < kSumParts; ++i) s += part[i][threadIdx.x];
    out[col] = s;
  }
}

}  // namespace

size_t norm_backward_workspace(int64_t rows, int64_t cols, int64_t gates) {
  int fit = 1;  // the most that any types and alignment have
  for (int i = 0; i < 8; ++i) {
    if ((i & 4) && cols > kRunsMaxCols) break;
    const int f = backward_plan(cols, i & 1, i & 2, i & 4).fit;
    fit = f > fit ? f : fit;
  }
  return static_cast<size_t>(backward_blocks(rows, kMaxSms, fit)) * (gates > 0 ? 4 : 2) *
         static_cast<size_t>(cols) * 4;
}

cudaError_t launch_norm_residual(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int64_t ce = p.c_fp32 ? 4 : 8, se = p.s_fp32 ? 4 : 8;
  const bool vec = p.cols % 8 == 0 && aligned16(p.block) && aligned16(p.residual) &&
                   aligned16(p.res_out) && aligned16(p.y) && aligned16(p.w_pre) &&
                   aligned16(p.w_post) && aligned16(p.gate) && p.ldb % ce == 0 &&
                   p.ldy % ce == 0 && p.ldr % se == 0 && p.ldo % se == 0;
  if (p.c_fp32) return norm_forward_f32(p, vec, num_sms, stream);
  if (p.s_fp32) return norm_forward_mixed(p, vec, num_sms, stream);
  return norm_forward_of<bf16, bf16>(p, vec, num_sms, stream);
}

cudaError_t launch_norm_residual_backward(const NormBackParams& p, int num_sms,
                                          cudaStream_t stream) {
  if (p.rows == 0) {
    const size_t bytes = static_cast<size_t>(p.cols) * 4;
    cudaError_t err = cudaMemsetAsync(p.d_w_pre, 0, bytes, stream);
    if (err == cudaSuccess && p.d_w_post) err = cudaMemsetAsync(p.d_w_post, 0, bytes, stream);
    if (err == cudaSuccess && p.d_gate)
      err = cudaMemsetAsync(p.d_gate, 0, bytes * p.gates, stream);
    return err;
  }
  const int64_t ce = p.c_fp32 ? 4 : 8, se = p.s_fp32 ? 4 : 8;
  const bool vec = p.cols % 8 == 0 && p.cols <= kRunsMaxCols && aligned16(p.d_res) && aligned16(p.dy) &&
                   aligned16(p.block) && aligned16(p.res_out) && aligned16(p.w_post) &&
                   aligned16(p.w_pre) && aligned16(p.gate) && aligned16(p.d_block) &&
                   aligned16(p.d_residual) && (!p.d_res || p.ldd % se == 0) && p.lddy % ce == 0 &&
                   p.ldb % ce == 0 && p.ldr % se == 0 && p.lddb % ce == 0 && p.lddr % se == 0;
  const BackPlan plan = backward_plan(p.cols, p.c_fp32, p.s_fp32, vec);
  const int64_t n = backward_blocks(p.rows, num_sms < kMaxSms ? num_sms : kMaxSms, plan.fit);
  cudaError_t err;
  if (p.c_fp32)
    err = norm_backward_f32(p, vec, n, stream);
  else if (p.s_fp32)
    err = norm_backward_mixed(p, vec, n, stream);
  else
    err = norm_backward_of<bf16, bf16>(p, vec, n, stream);
  if (err != cudaSuccess) return err;
  const int64_t jobs = 2 + (p.gates < n ? p.gates : n);
  return launch(norm_backward_sum_kernel,
                dim3(static_cast<unsigned>((p.cols + kSumCols - 1) / kSumCols),
                     static_cast<unsigned>(jobs)),
                kSumCols * kSumParts, 0, stream, p, static_cast<uint32_t>(n));
}

}  // namespace mx
