// rotate.cu -- the norms of query and key heads with the rotation by position,
// in one pass, and their gradient.  For every token t and head row x of D
// channels:
//
//   n_c = x_c w_c / sqrt(mean(x^2) + eps)
//   (y_a, y_b) = (n_a c - n_b s, n_a s + n_b c),  c, s = scale cos, sin(pos_t f_i)
//
// for the pairs (a, b) of the first R channels: (i, i + R/2) or (2 i, 2 i + 1); the
// other channels are n.  Gradient: dn is dy rotated back, then
//   dx = rho (w dn - x rho^2 mean(w dn x)),  dw = sum over rows of dn x rho.
//
// Bound by memory: a row is read once and written once.  A row belongs to a
// group of lanes, each of which holds both channels of its pairs, so that the
// only exchange is the sum (the gradient: two sums) over the row.  Angles are
// shared by a token's heads: a block computes the cosines and sines of its tokens
// once, in shared memory.  An angle is a product in turns: the frequency becomes
// a 64-bit fraction of a turn per position, the product with the position keeps
// its low 64 bits, which are the fraction of a turn -- exact to 2^-64 turns times
// the position however far that is, in integers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTable = 2048;  // pairs of cosine and sine of a block

// Fraction of a turn per position, in units of 2^-64, of a frequency in radians:
// the 53-bit significand times 2^66 / (2 pi), shifted to the binary point (and
// taken modulo a turn).
__device__ __forceinline__ uint64_t turns_of(double frequency) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(frequency));
  const int e = static_cast<int>((b >> 52) & 0x7FF);
  if (e == 0) return 0;  // below 2^-1022
  const uint64_t m = (b & 0xFFFFFFFFFFFFFull) | (1ull << 52);
  constexpr uint64_t kTurn = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi)
  const uint64_t hi = __umul64hi(m, kTurn), lo = m * kTurn;
  const int sh = 1077 - e;  // the product is turns * 2^(64 + sh)
  uint64_t v;
  if (sh >= 128) v = 0;
  else if (sh >= 64) v = hi >> (sh - 64);
  else if (sh > 0) v = (lo >> sh) | (hi << (64 - sh));
  else v = sh > -64 ? lo << -sh : 0;
  return (b >> 63) ? 0 - v : v;
}

__device__ __forceinline__ float2 angle(const RotateParams& p, int64_t token, int32_t i) {
  const int64_t pos = p.positions_64 ? static_cast<const int64_t*>(p.positions)[token]
                                     : static_cast<const int32_t*>(p.positions)[token];
  const uint64_t turn = static_cast<uint64_t>(pos) * turns_of(p.frequencies[i]);
  // signed half turns: the top 32 bits, rounded
  const int32_t top = static_cast<int32_t>((turn + (1ull << 31)) >> 32);
  float s, c;
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  return make_float2(c * p.scale, s * p.scale);
}

__device__ __forceinline__ float weight_of(const void* w, int32_t f32, int32_t i) {
  return f32 ? static_cast<const float*>(w)[i]
             : __bfloat162float(static_cast<const bf16*>(w)[i]);
}

// C consecutive elements as loaded.
template <typename T, int C>
struct Chunk;
template <>
struct Chunk<bf16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ void store(bf16* p, const float* f) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
};
template <>
struct Chunk<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Chunk<bf16, 1> {
  bf16 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *p; }
  __device__ __forceinline__ void get(float* f) const { f[0] = __bfloat162float(v); }
  static __device__ __forceinline__ void store(bf16* p, const float* f) {
    *p = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct Chunk<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void get(float* f) const { f[0] = v; }
  static __device__ __forceinline__ void store(float* p, const float* f) { *p = f[0]; }
};

// A lane's share of a row: S slots of two chunks of C channels, which hold whole
// pairs where the slot is one of the rotated part.
template <int C, int LPR, int S, bool INTER>
struct Lane {
  int32_t a[S], b[S];  // first channels of the chunks, -1 where there is none
  int32_t pair[S];     // first pair, or -1
  __device__ __forceinline__ Lane(const RotateParams& p, int32_t lane) {
    const int32_t turned = p.rotary / (2 * C);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int32_t g = lane + s * LPR;
      pair[s] = g < turned ? C * g : -1;
      if (g < turned) {
        a[s] = INTER ? 2 * C * g : C * g;
        b[s] = INTER ? a[s] + C : p.rotary / 2 + C * g;
      } else {
        a[s] = p.rotary + 2 * C * (g - turned);
        b[s] = a[s] + C;
        if (a[s] >= p.dim) a[s] = -1;
        if (b[s] >= p.dim) b[s] = -1;
      }
    }
  }
};

template <typename T, int C, int S>
struct Row {
  Chunk<T, C> a[S], b[S];
  template <typename L>
  __device__ __forceinline__ void load(const T* p, const L& l) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (l.a[s] >= 0) a[s].load(p + l.a[s]);
      if (l.b[s] >= 0) b[s].load(p + l.b[s]);
    }
  }
  // values of slot s, zero where there is no channel
  template <typename L>
  __device__ __forceinline__ void get(int s, const L& l, float* f) const {
    if (l.a[s] >= 0) {
      a[s].get(f);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) f[i] = 0.f;
    }
    if (l.b[s] >= 0) {
      b[s].get(f + C);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) f[C + i] = 0.f;
    }
  }
};

// Turns the pairs of a slot by their angles (sign -1: back).
template <int C, bool INTER>
__device__ __forceinline__ void turn(float* f, const float2* tab, float sign) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float& u = f[INTER ? 2 * i : i];
    float& v = f[INTER ? 2 * i + 1 : C + i];
    const float c = tab[i].x, s = tab[i].y * sign;
    const float y = u * c - v * s;
    v = u * s + v * c;
    u = y;
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Rows of a block: tokens [t0, t0 + nt) x heads [h0, h0 + nh) of queries, then keys.
struct Rows {
  int32_t t0, nt, h0, nh;
  __device__ __forceinline__ int32_t count() const { return nt * nh; }
};

template <int C, int S>
__device__ __forceinline__ void load_weights(const RotateParams& p, const int32_t* a,
                                             const int32_t* b, float (*wq)[2 * C],
                                             float (*wk)[2 * C]) {
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < 2 * C; ++i) {
      const int32_t at = i < C ? (a[s] < 0 ? -1 : a[s] + i) : (b[s] < 0 ? -1 : b[s] + i - C);
      wq[s][i] = at < 0 ? 0.f : weight_of(p.w_q, p.w_fp32, at);
      wk[s][i] = at < 0 ? 0.f : weight_of(p.w_k, p.w_fp32, at);
    }
}

__device__ __forceinline__ void fill_table(const RotateParams& p, const Rows& r, float2* tab) {
  const int32_t half = p.rotary / 2;
  for (int32_t i = threadIdx.x; i < r.nt * half; i += kThreads) {
    const int32_t t = i / half;
    tab[i] = angle(p, r.t0 + t, i - t * half);
  }
}

template <typename T, int C, int LPR, int S, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rotate_kernel(const RotateParams p) {
  extern __shared__ float2 tab[];
  constexpr int kGroups = kThreads / LPR;
  constexpr int U = S == 1 ? 2 : 1;  // rows under way
  const int32_t lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  Rows r;
  r.t0 = blockIdx.x * p.tokens_per_block;
  r.nt = min(p.tokens_per_block, p.tokens - r.t0);
  r.h0 = blockIdx.y * p.heads_per_block;
  r.nh = min(p.heads_per_block, p.q_heads + p.k_heads - r.h0);
  const Lane<C, LPR, S, INTER> l(p, lane);
  pdl_wait();
  pdl_launch_dependents();
  const int32_t rows = r.count();
  Row<T, C, S> x[U];
  auto row_at = [&](int32_t i, const T*& src, T*& dst, bool& is_q, int32_t& t) {
    t = i / r.nh;
    const int32_t h = r.h0 + i - t * r.nh;
    const int64_t token = r.t0 + t;
    is_q = h < p.q_heads;
    const int64_t hh = is_q ? h : h - p.q_heads;
    src = static_cast<const T*>(is_q ? p.q : p.k) + token * (is_q ? p.q_st : p.k_st) +
          hh * (is_q ? p.q_sh : p.k_sh);
    dst = static_cast<T*>(is_q ? p.out_q : p.out_k) + token * (is_q ? p.oq_st : p.ok_st) +
          hh * (is_q ? p.oq_sh : p.ok_sh);
  };
  auto load = [&](int32_t base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t i = base + u * kGroups;
      if (i >= rows) continue;
      const T* src;
      T* dst;
      bool is_q;
      int32_t t;
      row_at(i, src, dst, is_q, t);
      x[u].load(src, l);
    }
  };
  load(group);
  float wq[S][2 * C], wk[S][2 * C];
  load_weights<C, S>(p, l.a, l.b, wq, wk);
  fill_table(p, r, tab);
  __syncthreads();
  const float inv_dim = 1.f / static_cast<float>(p.dim);
  // (every lane of a warp runs the same rounds: the sums are over whole warps)
  for (int32_t base = 0; base < rows; base += U * kGroups) {
    if (base > 0) load(base + group);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t i = base + group + u * kGroups;
      const bool here = i < rows;
      float f[S][2 * C];
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        x[u].get(s, l, f[s]);
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) sum = fmaf(f[s][j], f[s][j], sum);
      }
      sum = row_sum<LPR>(sum);
      if (!here) continue;
      const float rho = rsqrtf(fmaf(sum, inv_dim, p.eps));
      const T* src;
      T* dst;
      bool is_q;
      int32_t t;
      row_at(i, src, dst, is_q, t);
#pragma unroll
      for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) f[s][j] = f[s][j] * rho * (is_q ? wq[s][j] : wk[s][j]);
        if (l.pair[s] >= 0)
          turn<C, INTER>(f[s], tab + t * (p.rotary / 2) + l.pair[s], 1.f);
        if (l.a[s] >= 0) Chunk<T, C>::store(dst + l.a[s], f[s]);
        if (l.b[s] >= 0) Chunk<T, C>::store(dst + l.b[s], f[s] + C);
      }
    }
  }
}

// Gradient: persistent blocks, whose sums of dw end in a part of the workspace each.
template <typename T, int C, int LPR, int S, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rotate_backward_kernel(const RotateParams p) {
  extern __shared__ float2 tab[];  // two tables; at the end [warps][2][dim] sums
  constexpr int kGroups = kThreads / LPR;
  const int32_t lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int32_t heads = p.q_heads + p.k_heads;
  const int32_t half = p.rotary / 2;
  const Lane<C, LPR, S, INTER> l(p, lane);
  pdl_wait();
  pdl_launch_dependents();
  float wq[S][2 * C], wk[S][2 * C], gq[S][2 * C], gk[S][2 * C];
  load_weights<C, S>(p, l.a, l.b, wq, wk);
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < 2 * C; ++j) gq[s][j] = gk[s][j] = 0.f;
  const float inv_dim = 1.f / static_cast<float>(p.dim);
  const int32_t units = (p.tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  int32_t buf = 0;
  for (int32_t unit = blockIdx.x; unit < units; unit += gridDim.x, buf ^= 1) {
    Rows r;
    r.t0 = unit * p.tokens_per_block;
    r.nt = min(p.tokens_per_block, p.tokens - r.t0);
    r.h0 = 0;
    r.nh = heads;
    float2* table = tab + buf * p.tokens_per_block * half;
    fill_table(p, r, table);
    __syncthreads();  // (and every thread is past the table before the last one)
    const int32_t rows = r.count();
    for (int32_t base = 0; base < rows; base += kGroups) {
      const int32_t i = base + group;
      const bool here = i < rows;
      const int32_t t = here ? i / heads : 0;
      const int32_t h = here ? i - t * heads : 0;
      const int64_t token = r.t0 + t;
      const bool is_q = h < p.q_heads;
      const int64_t hh = is_q ? h : h - p.q_heads;
      Row<T, C, S> x, d;
      if (here) {
        x.load(static_cast<const T*>(is_q ? p.q : p.k) + token * (is_q ? p.q_st : p.k_st) +
                   hh * (is_q ? p.q_sh : p.k_sh),
               l);
        d.load(static_cast<const T*>(is_q ? p.d_q : p.d_k) + token * (is_q ? p.dq_st : p.dk_st) +
                   hh * (is_q ? p.dq_sh : p.dk_sh),
               l);
      }
      float f[S][2 * C], g[S][2 * C];
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        x.get(s, l, f[s]);
        d.get(s, l, g[s]);
        if (l.pair[s] >= 0) turn<C, INTER>(g[s], table + t * half + l.pair[s], -1.f);
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) {
          sum = fmaf(f[s][j], f[s][j], sum);
          dot = fmaf(g[s][j] * (is_q ? wq[s][j] : wk[s][j]), f[s][j], dot);
        }
      }
      sum = row_sum<LPR>(sum);
      dot = row_sum<LPR>(dot);
      if (!here) continue;
      const float rho = rsqrtf(fmaf(sum, inv_dim, p.eps));
      const float back = rho * rho * dot * inv_dim;
      T* dst = static_cast<T*>(is_q ? p.out_q : p.out_k) + token * (is_q ? p.oq_st : p.ok_st) +
               hh * (is_q ? p.oq_sh : p.ok_sh);
#pragma unroll
      for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) {
          const float dwj = g[s][j] * f[s][j] * rho;
          gq[s][j] += is_q ? dwj : 0.f;
          gk[s][j] += is_q ? 0.f : dwj;
          g[s][j] = rho * fmaf(g[s][j], is_q ? wq[s][j] : wk[s][j], -f[s][j] * back);
        }
        if (l.a[s] >= 0) Chunk<T, C>::store(dst + l.a[s], g[s]);
        if (l.b[s] >= 0) Chunk<T, C>::store(dst + l.b[s], g[s] + C);
      }
    }
  }
  // sums of the rows of a warp, then of the block's warps, in a fixed order
  __syncthreads();
  float* sums = reinterpret_cast<float*>(tab);
  const int32_t warp = threadIdx.x / 32;
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < 2 * C; ++j) {
      float vq = gq[s][j], vk = gk[s][j];
#pragma unroll
      for (int d = LPR; d < 32; d <<= 1) {
        vq += __shfl_xor_sync(0xffffffffu, vq, d);
        vk += __shfl_xor_sync(0xffffffffu, vk, d);
      }
      const int32_t at = j < C ? l.a[s] : l.b[s];
      if (at >= 0 && (threadIdx.x & 31) < LPR) {
        sums[(warp * 2 + 0) * p.dim + at + j % C] = vq;
        sums[(warp * 2 + 1) * p.dim + at + j % C] = vk;
      }
    }
  __syncthreads();
  for (int32_t i = threadIdx.x; i < 2 * p.dim; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w * 2 * p.dim + i];
    p.workspace[static_cast<int64_t>(blockIdx.x) * 2 * p.dim + i] = v;
  }
}

// dw_q and dw_k from the blocks' parts: 32 columns a block, 8 rows of parts side
// by side.
__global__ void __launch_bounds__(256) norm_rotate_sums_kernel(const RotateParams p,
                                                               int32_t parts) {
  __shared__ float s[8][32];
  pdl_wait();
  pdl_launch_dependents();
  const int32_t x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int32_t col = blockIdx.x * 32 + x;
  float v = 0.f;
  if (col < 2 * p.dim)
    for (int32_t i = y; i < parts; i += 8)
      v += p.workspace[static_cast<int64_t>(i) * 2 * p.dim + col];
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && col < 2 * p.dim) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][x];
    (col < p.dim ? p.dw_q : p.dw_k)[col < p.dim ? col : col - p.dim] = v;
  }
}

struct Shape {
  int chunk, lanes, slots;
};

// Chunks of four channels where every array allows them, else single ones; as
// few lanes a row as hold it in one slot each.
Shape shape_of(const RotateParams& p) {
  if (p.chunks) {
    const int n = p.dim / 8;
    return n <= 8 ? Shape{4, 8, 1} : n <= 16 ? Shape{4, 16, 1} : n <= 32 ? Shape{4, 32, 1}
                                                                         : Shape{4, 32, 2};
  }
  const int n = (p.dim + 1) / 2;
  return n <= 32 ? Shape{1, 32, 1} : n <= 64 ? Shape{1, 32, 2} : n <= 128 ? Shape{1, 32, 4}
                                                                          : Shape{1, 32, 8};
}

// Blocks of the gradient at most: four an SM.
constexpr int32_t kBackBlocks = 4 * 152;

template <typename T, int C, int LPR, int S, bool INTER>
cudaError_t launch(RotateParams p, bool back, int num_sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / LPR;
  const int32_t heads = p.q_heads + p.k_heads, half = p.rotary / 2;
  // whole tokens a block, as many as give every group of lanes two rows
  int32_t per = heads >= 2 * kGroups ? 1 : 2 * kGroups / heads;
  if (per > kMaxTable / half) per = kMaxTable / half;
  // (no more than leave every SM a block)
  if (per > (p.tokens + num_sms - 1) / num_sms) per = (p.tokens + num_sms - 1) / num_sms;
  p.tokens_per_block = per;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (!back) {
    // few tokens: their heads over several blocks
    p.heads_per_block = p.tokens < num_sms && heads > kGroups ? kGroups : heads;
    cfg.gridDim = dim3((p.tokens + per - 1) / per,
                       (heads + p.heads_per_block - 1) / p.heads_per_block);
    cfg.dynamicSmemBytes = sizeof(float2) * per * half;
    return cudaLaunchKernelEx(&cfg, norm_rotate_kernel<T, C, LPR, S, INTER>, p);
  }
  const int32_t units = (p.tokens + per - 1) / per;
  const int32_t blocks = units < kBackBlocks ? units : kBackBlocks;
  const size_t tables = sizeof(float2) * 2 * per * half;
  const size_t sums = sizeof(float) * kWarps * 2 * p.dim;
  cfg.gridDim = dim3(blocks);
  cfg.dynamicSmemBytes = tables > sums ? tables : sums;
  cudaError_t err =
      cudaLaunchKernelEx(&cfg, norm_rotate_backward_kernel<T, C, LPR, S, INTER>, p);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3((2 * p.dim + 31) / 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, norm_rotate_sums_kernel, p, blocks);
}

template <typename T, bool INTER>
cudaError_t by_shape(const RotateParams& p, bool back, int num_sms, cudaStream_t stream) {
  const Shape s = shape_of(p);
  if (s.chunk == 4) {
    if (s.slots == 2) return launch<T, 4, 32, 2, INTER>(p, back, num_sms, stream);
    if (s.lanes == 8) return launch<T, 4, 8, 1, INTER>(p, back, num_sms, stream);
    if (s.lanes == 16) return launch<T, 4, 16, 1, INTER>(p, back, num_sms, stream);
    return launch<T, 4, 32, 1, INTER>(p, back, num_sms, stream);
  }
  switch (s.slots) {
    case 1: return launch<T, 1, 32, 1, INTER>(p, back, num_sms, stream);
    case 2: return launch<T, 1, 32, 2, INTER>(p, back, num_sms, stream);
    case 4: return launch<T, 1, 32, 4, INTER>(p, back, num_sms, stream);
    default: return launch<T, 1, 32, 8, INTER>(p, back, num_sms, stream);
  }
}

cudaError_t by_type(const RotateParams& p, bool back, int num_sms, cudaStream_t stream) {
  if (p.x_fp32)
    return p.interleaved ? by_shape<float, true>(p, back, num_sms, stream)
                         : by_shape<float, false>(p, back, num_sms, stream);
  return p.interleaved ? by_shape<bf16, true>(p, back, num_sms, stream)
                       : by_shape<bf16, false>(p, back, num_sms, stream);
}

}  // namespace

// (a block has at least one token)
size_t norm_rotate_backward_workspace(int64_t tokens, int64_t dim) {
  const int64_t blocks = tokens < kBackBlocks ? tokens : kBackBlocks;
  return static_cast<size_t>(blocks * 2 * dim * sizeof(float));
}

cudaError_t launch_norm_rotate(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return by_type(p, false, num_sms, stream);
}

cudaError_t launch_norm_rotate_backward(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return by_type(p, true, num_sms, stream);
}

}  // namespace mx
