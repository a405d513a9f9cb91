// norm.cu -- the norms before and after a block, with its gate and residual
// scale, and their gradients.
//
//   res_out = alpha * residual + g * n(block; w_post),  y = n(res_out; w_pre)
//   n(v; w)_c = v_c w_c / sqrt(mean(v^2) + eps)
//
// Both directions are bound by memory: every row is read and written once.
// A thread owns the same columns of every array of a row (eight in a run
// where rows and pointers allow 16-byte accesses, else every T-th one), so
// the only exchange within a row is the sum behind each norm.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ columns of a thread

// The columns that thread `tid` of `threads` owns, NV runs of eight.  VEC:
// run v is columns 8 (v threads + tid) ..+7, accessed 16 bytes at a time;
// else element j of run v is column (8 v + j) threads + tid.
template <bool VEC>
struct Cols {
  int32_t cols, tid, threads;
  __device__ __forceinline__ bool any(int v) const {
    return VEC ? 8 * (v * threads + tid) < cols : 8 * v * threads + tid < cols;
  }
  __device__ __forceinline__ bool has(int v, int j) const {
    return VEC ? any(v) : (8 * v + j) * threads + tid < cols;
  }
  __device__ __forceinline__ int32_t at(int v, int j) const {
    return VEC ? 8 * (v * threads + tid) + j : (8 * v + j) * threads + tid;
  }
};

__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

// Run v of a row; elements past its end read as zero.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, const Cols<VEC>& c, int v, float (&f)[8]) {
  if constexpr (VEC) {
    if (!c.any(v)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.f;
    } else if constexpr (sizeof(T) == 2) {
      unpack(*reinterpret_cast<const uint4*>(row + c.at(v, 0)), f);
    } else {
      const float4 a = *reinterpret_cast<const float4*>(row + c.at(v, 0));
      const float4 b = *reinterpret_cast<const float4*>(row + c.at(v, 4));
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
      f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c.has(v, j) ? to_float(row[c.at(v, j)]) : 0.f;
  }
}

// The same of a weight or gate, whose type is a run-time matter.
template <bool VEC>
__device__ __forceinline__ void load8_w(const void* w, int32_t f32, int64_t off,
                                        const Cols<VEC>& c, int v, float (&f)[8]) {
  if (f32)
    load8(static_cast<const float*>(w) + off, c, v, f);
  else
    load8(static_cast<const bf16*>(w) + off, c, v, f);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, const Cols<VEC>& c, int v, const float (&f)[8]) {
  if constexpr (VEC) {
    if (!c.any(v)) return;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(row + c.at(v, 0)) =
          make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    } else {
      *reinterpret_cast<float4*>(row + c.at(v, 0)) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(row + c.at(v, 4)) = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.has(v, j)) {
        if constexpr (sizeof(T) == 2)
          row[c.at(v, j)] = __float2bfloat16_rn(f[j]);
        else
          row[c.at(v, j)] = f[j];
      }
  }
}

template <typename T>
__device__ __forceinline__ float round_to(float v) {
  return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(v)) : v;
}

// ------------------------------------------------------------------ sums over a row

constexpr int kMaxWarps = 32;

// N sums over the block of threads, the same in every thread and run after
// run.  `part` holds N * 32 floats that the block's previous sum does not
// use (callers alternate between two), so one barrier is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (blockDim.x == 32) return;
  const uint32_t lane = lane_id(), warps = blockDim.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[i * kMaxWarps + warp_id()] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lane < warps ? part[i * kMaxWarps + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
}

__device__ __forceinline__ float rms_inverse(float sum_squares, float cols, float eps) {
  return 1.f / sqrtf(sum_squares / cols + eps);
}

// ------------------------------------------------------------------ forward

template <typename C, typename S, bool VEC, int NV>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const NormParams p) {
  __shared__ float part[2][kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const Cols<VEC> c{static_cast<int32_t>(p.cols), static_cast<int32_t>(threadIdx.x),
                    static_cast<int32_t>(blockDim.x)};
  const float cols = static_cast<float>(p.cols);
  for (int64_t t = blockIdx.x; t < p.rows; t += gridDim.x) {
    const C* brow = static_cast<const C*>(p.block) + t * p.ldb;
    const S* rrow = static_cast<const S*>(p.residual) + t * p.ldr;
    const int64_t goff = p.gate ? t / (p.rows / p.gates) * p.cols : 0;
    float b[NV][8], r[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) load8(brow, c, v, b[v]);
#pragma unroll
    for (int v = 0; v < NV; ++v) load8(rrow, c, v, r[v]);
    float sum[1];
    if (p.w_post) {
      sum[0] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] += b[v][j] * b[v][j];
      block_sum(sum, part[0]);
      const float sigma = rms_inverse(sum[0], cols, p.eps);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float w[8];
        load8_w(p.w_post, p.w_fp32, 0, c, v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[v][j] *= sigma * w[j];
      }
    }
    sum[0] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (p.gate) {
        float g[8];
        load8_w(p.gate, p.w_fp32, goff, c, v, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[v][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[v][j] = round_to<S>(p.alpha * r[v][j] + b[v][j]);
      store8(static_cast<S*>(p.res_out) + t * p.ldo, c, v, r[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[0] += r[v][j] * r[v][j];
    }
    block_sum(sum, part[1]);
    const float rho = rms_inverse(sum[0], cols, p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[8];
      load8_w(p.w_pre, p.w_fp32, 0, c, v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[v][j] *= rho * w[j];
      store8(static_cast<C*>(p.y) + t * p.ldy, c, v, r[v]);
    }
    if (!p.w_post && blockDim.x > 32) __syncthreads();  // part[1] is used in every row
  }
}

// ------------------------------------------------------------------ backward

// Rows of block i of n: [rows i / n, rows (i + 1) / n).
__host__ __device__ __forceinline__ int64_t first_row(int64_t rows, int64_t i, int64_t n) {
  return rows * i / n;
}
// Block whose rows hold row t.
__device__ __forceinline__ int64_t block_of_row(int64_t rows, int64_t t, int64_t n) {
  return ((t + 1) * n - 1) / rows;
}

// Workspace of n blocks: sums over each block's rows, FP32 [n][cols] for
// w_pre, [n][cols] for w_post, and [2n][cols] for gates whose rows several
// blocks share (a block's first such gate, then its last).
__device__ __forceinline__ float* ws_pre(const NormBackParams& p, int64_t i) {
  return p.workspace + i * p.cols;
}
__device__ __forceinline__ float* ws_post(const NormBackParams& p, int64_t n, int64_t i) {
  return p.workspace + (n + i) * p.cols;
}
__device__ __forceinline__ float* ws_gate(const NormBackParams& p, int64_t n, int64_t slot) {
  return p.workspace + (2 * n + slot) * p.cols;
}

// One block of threads goes through its own rows in order.  Rows arrive in
// shared memory by bulk copies, `stages` rows ahead (stages 0: rows whose
// addresses or sizes do not allow those, read in place), and are read from
// there as often as needed, so a thread's registers hold only its column
// sums (w_pre and D b sigma, 8 NV each) and D.
template <typename C, typename S, bool VEC, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
    norm_backward_kernel(const NormBackParams p, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float part[2][3 * kMaxWarps];
  __shared__ uint64_t full[8];
  __shared__ uint32_t abort_word;
  volatile uint32_t* s_abort = &abort_word;
  const Cols<VEC> c{static_cast<int32_t>(p.cols), static_cast<int32_t>(threadIdx.x),
                    static_cast<int32_t>(blockDim.x)};
  const float cols = static_cast<float>(p.cols);
  const int64_t n = gridDim.x, me = blockIdx.x;
  const int64_t lo = first_row(p.rows, me, n), hi = first_row(p.rows, me + 1, n);
  const uint32_t cbytes = static_cast<uint32_t>(p.cols * sizeof(C));
  const uint32_t sbytes = static_cast<uint32_t>(p.cols * sizeof(S));
  const uint32_t stage_bytes = 2 * cbytes + 2 * sbytes;
  // sums of D b sigma g over finished gates (gates > 1), behind the ring
  float* post_sum = reinterpret_cast<float*>(smem + static_cast<size_t>(stages) * stage_bytes);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    abort_word = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  auto issue = [&](int64_t t, int s) {
    uint8_t* dst = smem + static_cast<size_t>(s) * stage_bytes;
    mbar_arrive_expect_tx(&full[s], p.d_res ? stage_bytes : stage_bytes - sbytes);
    bulk_load(dst, static_cast<const C*>(p.dy) + t * p.lddy, cbytes, &full[s]);
    bulk_load(dst + cbytes, static_cast<const C*>(p.block) + t * p.ldb, cbytes, &full[s]);
    bulk_load(dst + 2 * cbytes, static_cast<const S*>(p.res_out) + t * p.ldr, sbytes, &full[s]);
    if (p.d_res)
      bulk_load(dst + 2 * cbytes + sbytes, static_cast<const S*>(p.d_res) + t * p.ldd, sbytes,
                &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && lo + s < hi; ++s) issue(lo + s, s);

  const bool many = p.gates > 1;
  const int64_t per = p.gates ? p.rows / p.gates : p.rows;
  float pre[NV][8], q[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      pre[v][j] = q[v][j] = 0.f;
      if (many && c.has(v, j)) post_sum[c.at(v, j)] = 0.f;
    }
  }
  int stage = 0;
  uint32_t phase = 0;
  int64_t group = lo / per, left = (group + 1) * per - lo;  // rows left of this gate
  for (int64_t t = lo; t < hi; ++t) {
    const C *dy, *block;
    const S *res, *dres;
    if (stages > 0) {
      mbar_wait(&full[stage], phase, s_abort, p.status, p.wait_limit_ns);
      const uint8_t* src = smem + static_cast<size_t>(stage) * stage_bytes;
      dy = reinterpret_cast<const C*>(src);
      block = reinterpret_cast<const C*>(src + cbytes);
      res = reinterpret_cast<const S*>(src + 2 * cbytes);
      dres = reinterpret_cast<const S*>(src + 2 * cbytes + sbytes);
    } else {
      dy = static_cast<const C*>(p.dy) + t * p.lddy;
      block = static_cast<const C*>(p.block) + t * p.ldb;
      res = static_cast<const S*>(p.res_out) + t * p.ldr;
      dres = static_cast<const S*>(p.d_res) + (p.d_res ? t * p.ldd : 0);
    }
    float d[NV][8];
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float x[8], y[8];
      load8(res, c, v, x);
      load8(dy, c, v, y);
      load8_w(p.w_pre, p.w_fp32, 0, c, v, d[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum[0] += x[j] * x[j];
        d[v][j] *= y[j];
        sum[1] += d[v][j] * x[j];
      }
      if (p.w_post) {
        load8(block, c, v, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[2] += x[j] * x[j];
      }
    }
    block_sum(sum, part[0]);
    // past this barrier nobody reads the previous row's stage any more
    if (stages > 0 && threadIdx.x == 0 && t > lo && t - 1 + stages < hi)
      issue(t - 1 + stages, stage == 0 ? stages - 1 : stage - 1);
    const float rho = rms_inverse(sum[0], cols, p.eps);
    // (in this order nothing leaves FP32's range before the product does)
    const float k = rho * (rho * (rho * (sum[1] / cols)));
    const float sigma = p.w_post ? rms_inverse(sum[2], cols, p.eps) : 1.f;
    const int64_t goff = group * p.cols;
    float dot[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float x[8], y[8];
      load8(res, c, v, x);
      load8(dy, c, v, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        pre[v][j] += y[j] * (x[j] * rho);
        d[v][j] = rho * d[v][j] - x[j] * k;
      }
      if (p.d_res) {
        load8(dres, c, v, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[v][j] += x[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = p.alpha * d[v][j];
      store8(static_cast<S*>(p.d_residual) + t * p.lddr, c, v, x);
      load8(block, c, v, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[v][j] += d[v][j] * (x[j] * sigma);
      if (p.gate) {
        load8_w(p.gate, p.w_fp32, goff, c, v, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[v][j] *= y[j];
      }
      if (p.w_post) {
        load8_w(p.w_post, p.w_fp32, 0, c, v, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d[v][j] *= y[j];
          dot[0] += d[v][j] * x[j];
        }
      }
    }
    float m = 0.f;
    if (p.w_post) {
      block_sum(dot, part[1]);
      m = sigma * (sigma * (sigma * (dot[0] / cols)));
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (p.w_post) {
        float x[8];
        load8(block, c, v, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[v][j] = sigma * d[v][j] - x[j] * m;
      }
      store8(static_cast<C*>(p.d_block) + t * p.lddb, c, v, d[v]);
    }
    if (!p.w_post && blockDim.x > 32) __syncthreads();  // part[0] is used in every row
    if (blockDim.x == 32) __syncwarp();  // as the barriers above: this row's reads are done
    if (stages > 0 && ++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    if (--left == 0 || t + 1 == hi) {  // the gate's rows, or this block's, end here
      if (p.gate) {
        const bool whole = group * per >= lo && t + 1 == (group + 1) * per;
        float* slot = ws_gate(p, n, 2 * me + (group == lo / per ? 0 : 1));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float g[8], w[8];
          load8_w(p.gate, p.w_fp32, goff, c, v, g);
          if (p.w_post) load8_w(p.w_post, p.w_fp32, 0, c, v, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (!c.has(v, j)) continue;
            const float dg = p.w_post ? q[v][j] * w[j] : q[v][j];
            (whole ? p.d_gate + goff : slot)[c.at(v, j)] = dg;
            if (many) post_sum[c.at(v, j)] += q[v][j] * g[j];
            q[v][j] = many ? 0.f : q[v][j] * g[j];
          }
        }
      }
      ++group;
      left = per;
    }
  }
  if (stages > 0 && *s_abort) {  // a wait gave up: copies still in flight must land first
    for (int s = 0; s < stages && lo + s < hi; ++s)
      mbar_wait(&full[s], static_cast<uint32_t>((hi - lo - 1 - s) / stages) & 1u, s_abort,
                p.status, p.wait_limit_ns, true);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!c.has(v, j)) continue;
      ws_pre(p, me)[c.at(v, j)] = pre[v][j];
      if (p.w_post) ws_post(p, n, me)[c.at(v, j)] = many ? post_sum[c.at(v, j)] : q[v][j];
    }
}

constexpr int kSumCols = 32, kSumParts = 16;

// Sums the blocks' parts in block order: job 0 w_pre, job 1 w_post, then
// the gates whose rows several blocks share.
__global__ void __launch_bounds__(kSumCols* kSumParts)
    norm_backward_sum_kernel(const NormBackParams p, int64_t n) {
  __shared__ float part[kSumParts][kSumCols + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t job = blockIdx.y;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kSumCols + threadIdx.x % kSumCols;
  const int part_id = threadIdx.x / kSumCols;
  int64_t first = 0, count = n, group = 0;
  float* out;
  if (job == 0) {
    out = p.d_w_pre;
  } else if (job == 1) {
    if (!p.w_post) return;
    out = p.d_w_post;
  } else {
    const int64_t per = p.rows / p.gates;
    // the gates themselves, or the gate at the start of each block's rows
    group = p.gates <= n ? job - 2 : first_row(p.rows, job - 1, n) / per;
    if (group >= p.gates) return;
    first = block_of_row(p.rows, group * per, n);
    count = block_of_row(p.rows, (group + 1) * per - 1, n) - first + 1;
    if (count == 1 || (p.gates > n && first != job - 2)) return;
    out = p.d_gate + group * p.cols;
  }
  float s = 0.f;
  if (col < p.cols) {
    // kSumParts runs of consecutive blocks, each in order
    const int64_t end = count * (part_id + 1) / kSumParts;
    for (int64_t i = count * part_id / kSumParts; i < end; ++i) {
      const int64_t b = first + i;
      if (job == 0)
        s += ws_pre(p, b)[col];
      else if (job == 1)
        s += ws_post(p, n, b)[col];
      else
        s += ws_gate(p, n, 2 * b + (first_row(p.rows, b, n) >= group * (p.rows / p.gates) ? 0 : 1))[col];
    }
  }
  part[part_id][threadIdx.x % kSumCols] = s;
  __syncthreads();
  if (part_id == 0 && col < p.cols) {
#pragma unroll
    for (int i = 1; i < kSumParts; ++i) s += part[i][threadIdx.x];
    out[col] = s;
  }
}

// ------------------------------------------------------------------ launches

template <typename K, typename... A>
cudaError_t launch(K kern, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Threads of a row of `cols` columns held in NV runs of eight per thread.
int row_threads(int64_t cols, int nv) {
  const int64_t runs = (cols + 7) / 8;
  return static_cast<int>(((runs + nv - 1) / nv + 31) / 32 * 32);
}

template <typename C, typename S, bool VEC>
cudaError_t forward(const NormParams& p, int num_sms, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.rows));
  if (p.cols <= 8192 && p.rows <= num_sms)
    return launch(norm_residual_kernel<C, S, VEC, 1>, grid, row_threads(p.cols, 1), 0, stream, p);
  if (p.cols <= 2048)
    return launch(norm_residual_kernel<C, S, VEC, 1>, grid, row_threads(p.cols, 1), 0, stream, p);
  return launch(norm_residual_kernel<C, S, VEC, 2>, grid, row_threads(p.cols, 2), 0, stream, p);
}

// Blocks of the gradient for a row width: those that fit an SM side by side
// with 64 registers a thread, times the SMs.
int64_t backward_blocks(int64_t rows, int64_t cols, int num_sms) {
  const int threads = row_threads(cols, cols <= 8192 ? 1 : 2);
  const int per_sm = threads <= 256 ? 4 : threads <= 512 ? 2 : 1;
  const int64_t n = static_cast<int64_t>(num_sms) * per_sm;
  return rows < n ? rows : n;
}

constexpr int kMaxSms = 192;         // workspaces are sized for this many
constexpr size_t kRingBytes = 216 * 1024;

template <typename C, typename S, bool VEC, int NV, int MAXT, int MINB>
cudaError_t backward_impl(const NormBackParams& p, int64_t n, cudaStream_t stream) {
  auto kern = norm_backward_kernel<C, S, VEC, NV, MAXT, MINB>;
  static PerDeviceOnce setup;
  const cudaError_t err = setup.run([&]() -> cudaError_t {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kRingBytes));
  });
  if (err != cudaSuccess) return err;
  const size_t stage = p.cols * 2 * (sizeof(C) + sizeof(S));
  const size_t post = p.gates > 1 ? p.cols * 4 : 0;
  size_t stages = VEC ? (kRingBytes / MINB - post) / stage : 0;
  stages = stages < 2 ? 0 : stages > 4 ? 4 : stages;
  return launch(kern, dim3(static_cast<unsigned>(n)), row_threads(p.cols, NV), stages * stage + post,
                stream, p, static_cast<int>(stages));
}

template <typename C, typename S, bool VEC>
cudaError_t backward(const NormBackParams& p, int64_t n, cudaStream_t stream) {
  const int threads = row_threads(p.cols, 1);
  if (threads <= 256) return backward_impl<C, S, VEC, 1, 256, 4>(p, n, stream);
  if (threads <= 512) return backward_impl<C, S, VEC, 1, 512, 2>(p, n, stream);
  if (threads <= 1024) return backward_impl<C, S, VEC, 1, 1024, 1>(p, n, stream);
  return backward_impl<C, S, VEC, 2, 1024, 1>(p, n, stream);
}

}  // namespace

size_t norm_backward_workspace(int64_t rows, int64_t cols, int64_t gates) {
  return static_cast<size_t>(backward_blocks(rows, cols, kMaxSms)) * (gates > 0 ? 4 : 2) *
         static_cast<size_t>(cols) * 4;
}

cudaError_t launch_norm_residual(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int64_t ce = p.c_fp32 ? 4 : 8, se = p.s_fp32 ? 4 : 8;
  const bool vec = p.cols % 8 == 0 && aligned16(p.block) && aligned16(p.residual) &&
                   aligned16(p.res_out) && aligned16(p.y) && aligned16(p.w_pre) &&
                   aligned16(p.w_post) && aligned16(p.gate) && p.ldb % ce == 0 &&
                   p.ldy % ce == 0 && p.ldr % se == 0 && p.ldo % se == 0;
  if (p.c_fp32)
    return vec ? forward<float, float, true>(p, num_sms, stream)
               : forward<float, float, false>(p, num_sms, stream);
  if (p.s_fp32)
    return vec ? forward<bf16, float, true>(p, num_sms, stream)
               : forward<bf16, float, false>(p, num_sms, stream);
  return vec ? forward<bf16, bf16, true>(p, num_sms, stream)
             : forward<bf16, bf16, false>(p, num_sms, stream);
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
  const bool vec = p.cols % 8 == 0 && aligned16(p.d_res) && aligned16(p.dy) &&
                   aligned16(p.block) && aligned16(p.res_out) && aligned16(p.w_post) &&
                   aligned16(p.w_pre) && aligned16(p.gate) && aligned16(p.d_block) &&
                   aligned16(p.d_residual) && (!p.d_res || p.ldd % se == 0) && p.lddy % ce == 0 &&
                   p.ldb % ce == 0 && p.ldr % se == 0 && p.lddb % ce == 0 && p.lddr % se == 0;
  const int64_t n =
      backward_blocks(p.rows, p.cols, num_sms < kMaxSms ? num_sms : kMaxSms);
  cudaError_t err;
  if (p.c_fp32)
    err = vec ? backward<float, float, true>(p, n, stream)
              : backward<float, float, false>(p, n, stream);
  else if (p.s_fp32)
    err = vec ? backward<bf16, float, true>(p, n, stream)
              : backward<bf16, float, false>(p, n, stream);
  else
    err = vec ? backward<bf16, bf16, true>(p, n, stream)
              : backward<bf16, bf16, false>(p, n, stream);
  if (err != cudaSuccess) return err;
  const int64_t jobs = 2 + (p.gates < n ? p.gates : n);
  return launch(norm_backward_sum_kernel,
                dim3(static_cast<unsigned>((p.cols + kSumCols - 1) / kSumCols),
                     static_cast<unsigned>(jobs)),
                kSumCols * kSumParts, 0, stream, p, n);
}

}  // namespace mx
