// moe_few.cu -- a whole mixture-of-experts layer for 1 to 64 tokens.
//
//   z = x router^T, the top_k largest per token win, w = softmax share;
//   y = sum over the winners e of w_e down_e (silu(gate_e x) * (up_e x))
//
// First form: four launches, one warp per dot product on the FP32 units.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float bf16(const void* p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Value of code `i` of a row.
__device__ __forceinline__ float decode(const uint8_t* row, int64_t i, int32_t fmt) {
  uint32_t code, ebits, mbits, bias;
  if (fmt == 7) {
    code = (row[i >> 1] >> ((i & 1) * 4)) & 15u;
    ebits = 2, mbits = 1, bias = 1;
  } else {
    code = row[i];
    ebits = fmt == 0 ? 4 : 5, mbits = fmt == 0 ? 3 : 2, bias = fmt == 0 ? 7 : 15;
  }
  const uint32_t e = (code >> mbits) & ((1u << ebits) - 1), m = code & ((1u << mbits) - 1);
  const bool neg = code >> (ebits + mbits);
  if ((fmt == 0 && (code & 0x7Fu) == 0x7Fu) || (fmt == 1 && e == 31u && m != 0))
    return __int_as_float(0x7FC00000);
  if (fmt == 1 && e == 31u) return __int_as_float(neg ? 0xFF800000 : 0x7F800000);
  const float v = e == 0 ? ldexpf(static_cast<float>(m), 1 - static_cast<int>(bias + mbits))
                         : ldexpf(static_cast<float>((1u << mbits) + m),
                                  static_cast<int>(e) - static_cast<int>(bias + mbits));
  return neg ? -v : v;
}

// Scale of block j of row r in an expert's swizzled scale matrix.
__device__ __forceinline__ float block_scale(const uint8_t* s, int64_t r, int64_t j,
                                             int64_t k_tiles) {
  const uint32_t c = s[((r >> 7) * k_tiles + (j >> 2)) * 512 + (r & 31) * 16 +
                       ((r & 127) >> 5) * 4 + (j & 3)];
  return c == 255u ? __int_as_float(0x7FC00000)
                   : __int_as_float(c == 0 ? 0x00400000 : static_cast<int>(c << 23));
}

__global__ void __launch_bounds__(kThreads) moe_logits_kernel(const MoeFewParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  if (w >= static_cast<int64_t>(p.tokens) * p.experts) return;
  const int64_t t = w / p.experts, e = w % p.experts;
  float s = 0.f;
  for (int64_t c = lane_id(); c < p.hidden; c += 32) {
    const float r = p.router_fp32 ? static_cast<const float*>(p.router)[e * p.hidden + c]
                                  : bf16(p.router, e * p.hidden + c);
    s += bf16(p.x, t * p.ldx + c) * r;
  }
  s = warp_sum(s);
  if (lane_id() == 0) p.logits[w] = s;
}

// Order-preserving key of a logit (equal zeros alike, NaN below everything)
// with the expert behind it, so that among equal logits the lowest wins.
__device__ __forceinline__ uint64_t logit_key(float z, uint32_t e) {
  const uint32_t b = __float_as_uint(z + 0.f);
  const uint32_t k = z != z ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return static_cast<uint64_t>(k) << 32 | (0xFFFFFFFFu - e);
}

__global__ void __launch_bounds__(32) moe_select_kernel(const MoeFewParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const float* z = p.logits + t * p.experts;
  float top = -INFINITY;
  for (int e = lane_id(); e < p.experts; e += 32) top = fmaxf(top, z[e]);
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f;
  for (int e = lane_id(); e < p.experts; e += 32) sum += expf(z[e] - top);
  sum = warp_sum(sum);
  uint64_t last = ~0ull;
  float chosen = 0.f;
  for (int k = 0; k < p.top_k; ++k) {
    uint64_t best = 0;
    for (int e = lane_id(); e < p.experts; e += 32) {
      const uint64_t key = logit_key(z[e], e);
      if (key < last && key > best) best = key;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
      if (other > best) best = other;
    }
    last = best;
    const int e = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
    const float w = expf(z[e] - top) / sum;
    chosen += w;
    if (lane_id() == 0) {
      p.ids[t * p.top_k + k] = e;
      p.weights[t * p.top_k + k] = w;
    }
  }
  __syncwarp();
  if (p.renormalize)
    for (int k = lane_id(); k < p.top_k; k += 32) p.weights[t * p.top_k + k] /= chosen;
}

// One warp per (token, choice, channel of the expert).
__global__ void __launch_bounds__(kThreads) moe_gate_up_kernel(const MoeFewParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  if (w >= static_cast<int64_t>(p.tokens) * p.top_k * p.inter) return;
  const int64_t slot = w / p.inter, i = w % p.inter, t = slot / p.top_k;
  const int64_t e = p.ids[slot];
  const int64_t k_tiles = (p.hidden + 127) / 128;
  const int64_t smat = (p.inter + 127) / 128 * k_tiles * 512;
  const int64_t row = p.hidden * p.bits_gu / 8;
  const uint8_t* g = p.gate + (e * p.inter + i) * row;
  const uint8_t* u = p.up + (e * p.inter + i) * row;
  float a = 0.f, b = 0.f;
  for (int64_t c = lane_id(); c < p.hidden; c += 32) {
    const float x = bf16(p.x, t * p.ldx + c);
    a += x * decode(g, c, p.fmt_gu) * block_scale(p.gate_scales + e * smat, i, c >> 5, k_tiles);
    b += x * decode(u, c, p.fmt_gu) * block_scale(p.up_scales + e * smat, i, c >> 5, k_tiles);
  }
  a = warp_sum(a);
  b = warp_sum(b);
  if (lane_id() == 0) p.h[w] = a / (1.f + expf(-a)) * b * p.weights[slot];
}

// One warp per (token, channel of y).
__global__ void __launch_bounds__(kThreads) moe_down_kernel(const MoeFewParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  if (w >= static_cast<int64_t>(p.tokens) * p.hidden) return;
  const int64_t t = w / p.hidden, c = w % p.hidden;
  const int64_t k_tiles = (p.inter + 127) / 128;
  const int64_t smat = (p.hidden + 127) / 128 * k_tiles * 512;
  float s = 0.f;
  for (int k = 0; k < p.top_k; ++k) {
    const int64_t slot = t * p.top_k + k, e = p.ids[slot];
    const uint8_t* d = p.down + (e * p.hidden + c) * (p.inter * p.bits_d / 8);
    for (int64_t i = lane_id(); i < p.inter; i += 32)
      s += p.h[slot * p.inter + i] * decode(d, i, p.fmt_d) *
           block_scale(p.down_scales + e * smat, c, i >> 5, k_tiles);
  }
  s = warp_sum(s);
  if (lane_id() == 0) static_cast<__nv_bfloat16*>(p.y)[t * p.ldy + c] = __float2bfloat16_rn(s);
}

template <typename K>
cudaError_t launch(K kern, int64_t grid, int threads, const MoeFewParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

size_t moe_few_workspace(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                         int32_t top_k) {
  (void)hidden;
  return static_cast<size_t>(tokens) *
         ((static_cast<size_t>(experts) + 3) / 4 * 16 + static_cast<size_t>(top_k) * inter * 4);
}

cudaError_t launch_moe_few(const MoeFewParams& q, cudaStream_t stream) {
  MoeFewParams p = q;
  p.logits = static_cast<float*>(q.workspace);
  p.h = p.logits + static_cast<int64_t>(p.tokens) * ((p.experts + 3) / 4 * 4);
  constexpr int64_t kWarps = kThreads / 32;
  const int64_t t = p.tokens;
  cudaError_t err = launch(moe_logits_kernel, (t * p.experts + kWarps - 1) / kWarps, kThreads, p, stream);
  if (err == cudaSuccess) err = launch(moe_select_kernel, t, 32, p, stream);
  if (err == cudaSuccess)
    err = launch(moe_gate_up_kernel, (t * p.top_k * p.inter + kWarps - 1) / kWarps, kThreads, p, stream);
  if (err == cudaSuccess)
    err = launch(moe_down_kernel, (t * p.hidden + kWarps - 1) / kWarps, kThreads, p, stream);
  return err;
}

}  // namespace mx
