// norm.cu -- the norms around a block: the choice of kernels by type, the
// kernels for bf16 blocks on a bf16 stream, and the joining of the gradient's
// column sums.
#include "norm_kernel.cuh"

namespace mx {

cudaError_t norm_forward_mixed(const NormParams& p, NormRows kind, int num_sms, cudaStream_t stream);
cudaError_t norm_forward_f32(const NormParams& p, NormRows kind, int num_sms, cudaStream_t stream);
cudaError_t norm_backward_mixed(const NormBackParams& p, NormRows kind, int64_t n, cudaStream_t stream);
cudaError_t norm_backward_f32(const NormBackParams& p, NormRows kind, int64_t n, cudaStream_t stream);

namespace {

constexpr int kSumCols = 32, kSumParts = 32, kSumThreads = kSumCols * kSumParts;

// What the sum kernel's blocks do: blocks [0, wide) take 32 columns of w_pre,
// [wide, 2 wide) of w_post; then `gate_jobs` gates whose rows several blocks
// share, each in `gate_tiles` blocks: of 32 columns too where a gate has many
// parts, else of 1024, a thread each (16384 x 2048, 2 gates: gradient 79.2 us,
// the other way 84.1; 16 gates: 79.9, the other way 86.1).
struct SumPlan {
  uint32_t wide, gate_jobs, gate_tiles;
};
SumPlan sum_plan(int64_t rows, int64_t cols, int64_t gates, int64_t n) {
  SumPlan s;
  s.wide = static_cast<uint32_t>((cols + kSumCols - 1) / kSumCols);
  // (rows == gates: every gate has one row, and no part)
  s.gate_jobs = static_cast<uint32_t>(gates == rows ? 0 : gates < n ? gates : n);
  s.gate_tiles = n >= 64 * gates ? s.wide : static_cast<uint32_t>((cols + kSumThreads - 1) / kSumThreads);
  return s;
}

// Sums the blocks' parts.  Where a block of threads takes 32 columns, 32 runs
// of consecutive parts are summed in order side by side, then joined in order.
__global__ void __launch_bounds__(kSumThreads)
    norm_backward_sum_kernel(const NormBackParams p, uint32_t n, const SumPlan plan) {
  __shared__ float part[kSumParts][kSumCols + 1];
  pdl_wait();
  pdl_launch_dependents();
  const RowShare share(static_cast<uint32_t>(p.rows), n);
  uint32_t first = 0, count = n, tile = blockIdx.x;
  bool narrow = true;                                 // 32 columns a block
  const float* src;
  int64_t step = p.cols, start_of_first = 0;          // floats from part to part
  float* out;
  if (blockIdx.x < plan.wide) {
    src = ws_pre(p, 0);
    out = p.d_w_pre;
  } else if (blockIdx.x < 2 * plan.wide) {
    if (!p.w_post) return;
    tile -= plan.wide;
    src = ws_post(p, n, 0);
    out = p.d_w_post;
  } else {
    const uint32_t job = (blockIdx.x - 2 * plan.wide) / plan.gate_tiles;
    tile = blockIdx.x - 2 * plan.wide - job * plan.gate_tiles;
    narrow = plan.gate_tiles == plan.wide;
    const uint32_t per = static_cast<uint32_t>(p.rows / p.gates);
    // the gates themselves, or the gate at the start of each block's rows
    const uint32_t group = p.gates <= n ? job : share.start(job + 1) / per;
    if (group >= p.gates) return;
    first = share.of(group * per);
    count = share.of((group + 1) * per - 1) - first + 1;
    if (count == 1 || (p.gates > n && first != job)) return;
    // blocks after the first begin inside this gate: their first slot; the
    // first block's is its last if it began in an earlier gate
    src = ws_gate(p, n, 2 * static_cast<int64_t>(first));
    step = 2 * p.cols;
    start_of_first = share.start(first) < group * per ? p.cols : 0;
    out = p.d_gate + group * p.cols;
  }
  if (!narrow) {
    const int64_t col = static_cast<int64_t>(tile) * kSumThreads + threadIdx.x;
    if (col >= p.cols) return;
    float s = src[start_of_first + col];
    for (uint32_t i = 1; i < count; ++i) s += src[i * step + col];
    out[col] = s;
    return;
  }
  const int64_t col = static_cast<int64_t>(tile) * kSumCols + threadIdx.x % kSumCols;
  const uint32_t run = threadIdx.x / kSumCols;
  float s = 0.f;
  if (col < p.cols) {
    uint32_t i = static_cast<uint32_t>(static_cast<uint64_t>(count) * run / kSumParts);
    const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(count) * (run + 1) / kSumParts);
    if (i == 0 && end > 0) s = src[start_of_first + col], i = 1;
#pragma unroll 8
    for (; i < end; ++i) s += src[i * step + col];
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
  int64_t n = 0;  // the most blocks that any types and alignment have
  for (int i = 0; i < 4; ++i)
    for (NormRows kind : {NormRows::kAligned, NormRows::kShifted, NormRows::kAny}) {
      if (kind == NormRows::kShifted && cols > kShiftCols) continue;
      const int64_t m = backward_blocks(rows, kMaxSms, backward_plan(rows, cols, gates, i & 1, i & 2, kind));
      n = m > n ? m : n;
    }
  return static_cast<size_t>(n) * (gates > 0 ? 4 : 2) * static_cast<size_t>(cols) * 4;
}

// Whether rows of another array are as far (in columns modulo 8) into their 16
// bytes as those of the first.
struct InStep {
  uint64_t at;
  int64_t ld;
  static uint64_t column(const void* a, bool fp32) {
    return reinterpret_cast<uintptr_t>(a) / (fp32 ? 4 : 2);
  }
  InStep(const void* a, int64_t ld, bool fp32) : at(column(a, fp32)), ld(ld) {}
  bool with(const void* b, int64_t ldb, bool fp32) const {
    return ((column(b, fp32) ^ at) & 7u) == 0 && ((ld ^ ldb) & 7) == 0;
  }
};

cudaError_t launch_norm_residual(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int64_t ce = p.c_fp32 ? 4 : 8, se = p.s_fp32 ? 4 : 8;
  NormRows kind = NormRows::kAny;
  if (p.cols % 8 == 0 && aligned16(p.block) && aligned16(p.residual) && aligned16(p.res_out) &&
      aligned16(p.y) && aligned16(p.w_pre) && aligned16(p.w_post) && aligned16(p.gate) &&
      p.ldb % ce == 0 && p.ldy % ce == 0 && p.ldr % se == 0 && p.ldo % se == 0) {
    kind = NormRows::kAligned;
  } else if (p.cols + 7 <= 8 * 4 * 512) {  // (what the widest kernel holds)
    const InStep step(p.block, p.ldb, p.c_fp32);
    if (step.with(p.y, p.ldy, p.c_fp32) && step.with(p.residual, p.ldr, p.s_fp32) &&
        step.with(p.res_out, p.ldo, p.s_fp32))
      kind = NormRows::kShifted;
  }
  if (p.c_fp32) return norm_forward_f32(p, kind, num_sms, stream);
  if (p.s_fp32) return norm_forward_mixed(p, kind, num_sms, stream);
  return norm_forward_of<bf16, bf16>(p, kind, num_sms, stream);
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
  // (d_gate is in this: the kernel for aligned rows writes a gate of its own
  // rows there in 16-byte stores.  d_w_pre and d_w_post are not: the sum kernel
  // writes them, and gates of several blocks' rows, float by float.)
  NormRows kind = NormRows::kAny;
  if (p.cols % 8 == 0 && aligned16(p.d_res) && aligned16(p.dy) && aligned16(p.block) &&
      aligned16(p.res_out) && aligned16(p.w_post) && aligned16(p.w_pre) && aligned16(p.gate) &&
      aligned16(p.d_block) && aligned16(p.d_residual) && aligned16(p.d_gate) &&
      (!p.d_res || p.ldd % se == 0) &&
      p.lddy % ce == 0 && p.ldb % ce == 0 && p.ldr % se == 0 && p.lddb % ce == 0 &&
      p.lddr % se == 0) {
    kind = NormRows::kAligned;
  } else if (p.cols <= kShiftCols && (p.gates == 0 || p.rows >= 16 * p.gates) &&
             (p.cols > kOneRun || (p.cols > 1024 && p.rows >= 64 * static_cast<int64_t>(num_sms)))) {
    // Going by phase takes 16-byte accesses, but its sums change hands after
    // each of up to eight phases: 16384 x 2049 144 us (element by element 311),
    // x 1111 100 (122), x 501 61 (58); 3000 x 1111 39 (31); 16 rows a gate 131
    // (134); more than 4096 columns: 16384 x 5001 343 (701), 400 x 5001 31 (29).
    const InStep step(p.block, p.ldb, p.c_fp32);
    if (step.with(p.dy, p.lddy, p.c_fp32) && step.with(p.res_out, p.ldr, p.s_fp32) &&
        (!p.d_res || step.with(p.d_res, p.ldd, p.s_fp32)) &&
        step.with(p.d_block, p.lddb, p.c_fp32) && step.with(p.d_residual, p.lddr, p.s_fp32))
      kind = NormRows::kShifted;
  }
  const BackPlan plan = backward_plan(p.rows, p.cols, p.gates, p.c_fp32, p.s_fp32, kind);
  const int64_t n = backward_blocks(p.rows, num_sms < kMaxSms ? num_sms : kMaxSms, plan);
  cudaError_t err;
  if (p.c_fp32)
    err = norm_backward_f32(p, kind, n, stream);
  else if (p.s_fp32)
    err = norm_backward_mixed(p, kind, n, stream);
  else
    err = norm_backward_of<bf16, bf16>(p, kind, n, stream);
  if (err != cudaSuccess) return err;
  const SumPlan sum = sum_plan(p.rows, p.cols, p.gates, n);
  return launch(norm_backward_sum_kernel,
                dim3(2 * sum.wide + sum.gate_jobs * sum.gate_tiles), kSumThreads, 0, stream, p,
                static_cast<uint32_t>(n), sum);
}

}  // namespace mx
