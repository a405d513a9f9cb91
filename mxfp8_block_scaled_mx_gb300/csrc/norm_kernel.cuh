// norm_kernel.cuh -- the norms before and after a block, with its gate and
// residual scale, and their gradients: kernels and their launches, which
// norm.cu, norm_mixed.cu and norm_f32.cu instantiate for the types of blocks and
// stream (three files, so that they compile side by side).
//
//   res_out = alpha * residual + g * n(block; w_post),  y = n(res_out; w_pre)
//   n(v; w)_c = v_c w_c / sqrt(mean(v^2) + eps)
//
// Both directions are bound by memory: every row is read and written once.
// A thread owns the same columns of every array of a row (runs of eight where
// rows and pointers allow 16-byte accesses, else every T-th one), so the only
// exchange within a row is the sum behind each norm.  Arithmetic is FP32, two
// columns an instruction (f32x2): at memory speed a row leaves an SM about 20
// instructions per column pair and direction, so their number counts.
// Measured on one GB300 (part of the measured copy bandwidth, 6.68 TB/s):
//   forward   16384 x 7168 bf16: 155 us, 0.91; 8192 x 2048, FP32 stream, four
//             gates: 34.7 us, 0.87; one row of 7168: 3.1 us, the latency of a
//             launch, two loads and two sums; 777 x 1111 FP32: 4.9 us, 0.42
//   gradient  16384 x 7168 bf16: 217 us, 0.97; 8192 x 2048, FP32 stream, four
//             gates: 55 us, 0.82 (5.5 us of it the sums over rows); 333 x 1111:
//             10.5 us, a row's latency, then the sums over 333 parts
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mx {

// What a pass's arrays allow: 16-byte accesses from each row's first
// column on; from the same column of a row on in all of them (rows of an odd
// length); neither.
enum class NormRows { kAligned, kShifted, kAny };

namespace {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ pairs of columns

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ void store1(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// ------------------------------------------------------------------ columns of a thread

// How a thread's NV runs of eight columns lie in a row:
// kWhole  run v is columns 8 (v threads + tid) ..+7, 16 bytes an access, and
//         the row has exactly 8 NV threads columns;
// kRuns   the same with an end inside (whole runs of eight);
// kShift  run v is columns 8 (v threads + tid) - phase ..+7, with the row's phase
//         (0..7) such that its runs lie on 16 bytes; first and last may be cut
//         (`open`: they may be read whole, rows lie on either side);
// kSingle element j of run v is column (8 v + j) threads + tid, one at a time.
enum Mode { kWhole, kRuns, kShift, kSingle };

template <Mode M>
struct Cols {
  int32_t cols, tid, threads, phase = 0;
  bool open = false;
  __device__ __forceinline__ int32_t at(int v, int j) const {
    return M == kSingle  ? (8 * v + j) * threads + tid
           : M == kShift ? 8 * (v * threads + tid) - phase + j
                         : 8 * (v * threads + tid) + j;
  }
  __device__ __forceinline__ bool has(int v, int j) const {
    return M == kWhole || (M == kShift ? static_cast<uint32_t>(at(v, j)) < static_cast<uint32_t>(cols)
                                       : at(v, M == kRuns ? 0 : j) < cols);
  }
  // run v lies inside the row, with `margin` columns to spare on either side
  __device__ __forceinline__ bool inside(int v, int margin = 0) const {
    return at(v, 0) >= margin && at(v, 0) + 8 + margin <= cols;
  }
};

// A run of eight elements as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<bf16> {
  uint32_t w[4];
  __device__ __forceinline__ float2 get(int i) const { return unpack2(w[i]); }
};
template <>
struct Raw<float> {
  float2 f[4];
  __device__ __forceinline__ float2 get(int i) const { return f[i]; }
};

__device__ __forceinline__ uint32_t bits(bf16 v) { return *reinterpret_cast<const uint16_t*>(&v); }

// Sixteen bytes of global memory that are read once: they take no place of the
// weights' in L1.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Run v of a row; elements past its ends read as zero (of an open row: as
// anything, until trimmed).  ONCE: a row of global memory that is not read again.
template <typename T, Mode M>
__device__ __forceinline__ Raw<T> load8_singly(const T* row, const Cols<M>& c, int v) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool a = c.has(v, 2 * i), b = c.has(v, 2 * i + 1);
    if constexpr (sizeof(T) == 2)
      r.w[i] = (a ? bits(row[c.at(v, 2 * i)]) : 0u) | (b ? bits(row[c.at(v, 2 * i + 1)]) << 16 : 0u);
    else
      r.f[i] = make_float2(a ? row[c.at(v, 2 * i)] : 0.f, b ? row[c.at(v, 2 * i + 1)] : 0.f);
  }
  return r;
}
template <bool ONCE = false, typename T, Mode M>
__device__ __forceinline__ Raw<T> load8(const T* row, const Cols<M>& c, int v) {
  if constexpr (M == kSingle) return load8_singly(row, c, v);
  if constexpr (M == kShift)
    if (!c.open && !c.inside(v)) return load8_singly(row, c, v);
  Raw<T> r;
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  if (M == kShift ? c.at(v, 0) < c.cols : c.has(v, 0)) {
    const uint4* p = reinterpret_cast<const uint4*>(row + c.at(v, 0));
    x = ONCE ? load_once(p) : p[0];
    if constexpr (sizeof(T) == 4) y = ONCE ? load_once(p + 1) : p[1];
  }
  if constexpr (sizeof(T) == 2) {
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
  } else {
    r.f[0] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
    r.f[1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
    r.f[2] = make_float2(__uint_as_float(y.x), __uint_as_float(y.y));
    r.f[3] = make_float2(__uint_as_float(y.z), __uint_as_float(y.w));
  }
  return r;
}

// Clears what lies past the row's ends (rows beside it, which another block may
// be writing in place: nothing of it is used).
template <typename T, Mode M>
__device__ __forceinline__ void trim(Raw<T>& r, const Cols<M>& c, int v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool a = c.has(v, 2 * i), b = c.has(v, 2 * i + 1);
    if constexpr (sizeof(T) == 2)
      r.w[i] = (a ? r.w[i] & 0xFFFFu : 0u) | (b ? r.w[i] & 0xFFFF0000u : 0u);
    else
      r.f[i] = make_float2(a ? r.f[i].x : 0.f, b ? r.f[i].y : 0.f);
  }
}

// Run v of a weight or gate.  Under kShift it lies anywhere: the 16-byte
// pieces that hold it (inside the row wherever this is done), then the words
// moved into place.
template <typename T, Mode M>
__device__ __forceinline__ Raw<T> load8_weight(const T* row, const Cols<M>& c, int v) {
  if constexpr (M != kShift) {
    return load8(row, c, v);
  } else {
    if (!c.inside(v, 8)) return load8_singly(row, c, v);
    constexpr int N = sizeof(T) * 2 + 4;                 // words of the pieces
    const uintptr_t a = reinterpret_cast<uintptr_t>(row + c.at(v, 0));
    const uint4* p = reinterpret_cast<const uint4*>(a & ~uintptr_t(15));
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = p[i];
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
    const uint32_t by = static_cast<uint32_t>(a) & 15u;  // bytes
#pragma unroll
    for (int i = 0; i + 2 < N; ++i) w[i] = by & 8u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) w[i] = by & 4u ? w[i + 1] : w[i];
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2)
        r.w[i] = __funnelshift_r(w[i], w[i + 1], by & 2u ? 16u : 0u);
      else
        r.f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    return r;
  }
}

// Asks for a row's lines, one a thread (rows have fewer lines than threads).
template <typename T, Mode M>
__device__ __forceinline__ void prefetch_row(const T* row, const Cols<M>& c) {
  constexpr int kLine = 128 / sizeof(T);
  if (c.tid * kLine < c.cols)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c.tid * kLine));
}

// f *= a run.
template <typename T>
__device__ __forceinline__ void times(float2 (&f)[4], const Raw<T>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], r.get(i));
}
// f *= run v of a weight or gate.
template <typename W, Mode M>
__device__ __forceinline__ void times_w(float2 (&f)[4], const void* w, int64_t off,
                                        const Cols<M>& c, int v) {
  times(f, load8_weight(static_cast<const W*>(w) + off, c, v));
}

__device__ __forceinline__ void store_once(uint4* p, const uint4& v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// ONCE: a bf16 row of global memory that takes no place in L1 (16384 x 4096: 81.6
// us, with a place 83.3; FP32 rows are written in two halves that L1 joins:
// 16384 x 7168 with an FP32 stream 217, past L1 221).
template <bool ONCE = false, typename T, Mode M>
__device__ __forceinline__ void store8(T* row, const Cols<M>& c, int v, const Raw<T>& r) {
  if (M == kSingle || (M == kShift && !c.inside(v))) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.has(v, j)) {
        if constexpr (sizeof(T) == 2)
          row[c.at(v, j)] = __ushort_as_bfloat16(static_cast<uint16_t>(r.w[j / 2] >> (j % 2 * 16)));
        else
          row[c.at(v, j)] = j % 2 ? r.f[j / 2].y : r.f[j / 2].x;
      }
  } else {
    if (!c.has(v, 0)) return;
    uint4* p = reinterpret_cast<uint4*>(row + c.at(v, 0));
    if constexpr (sizeof(T) == 2) {
      const uint4 x = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
      if constexpr (ONCE)
        store_once(p, x);
      else
        *p = x;
    } else {
      p[0] = make_uint4(__float_as_uint(r.f[0].x), __float_as_uint(r.f[0].y),
                        __float_as_uint(r.f[1].x), __float_as_uint(r.f[1].y));
      p[1] = make_uint4(__float_as_uint(r.f[2].x), __float_as_uint(r.f[2].y),
                        __float_as_uint(r.f[3].x), __float_as_uint(r.f[3].y));
    }
  }
}

// Eight FP32 values in type T (one rounding).
template <typename T>
__device__ __forceinline__ Raw<T> round8(const float2 (&f)[4]) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2)
      r.w[i] = pack2(f[i]);
    else
      r.f[i] = f[i];
  }
  return r;
}

// ------------------------------------------------------------------ sums over a row

constexpr int kMaxWarps = 32;

// N sums over the block of threads, the same in every thread and run after
// run.  `part` holds N * 32 floats (zeros past the last warp) that the block's
// previous sum does not use (callers alternate between two), so one barrier
// is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (blockDim.x == 32) return;
  if (lane_id() == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[i * kMaxWarps + warp_id()] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (uint32_t w = 0; w < blockDim.x / 32; w += 4)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(part + i * kMaxWarps + w);
      v[i] += (f.x + f.y) + (f.z + f.w);
    }
}

// 1 / sqrt(mean + eps): the hardware's estimate and one Newton step, which
// leaves an error of about one unit in the last place (and 1 / 0 and 1 / inf
// as they are, where the step would make NaN).
__device__ __forceinline__ float rms_inverse(float sum_squares, float inv_cols, float eps) {
  const float m = sum_squares * inv_cols + eps;
  const float r = rsqrtf(m);
  const float s = r + r * 0.5f * (1.f - m * r * r);
  return m > 0.f && m < INFINITY ? s : r;
}

// ------------------------------------------------------------------ forward

// A block of threads goes through every gridDim.x-th row, as many blocks as the
// SMs hold.  A row's registers are free once the stream's row is formed, so
// the next row is loaded there, behind the second norm: a row's 57 KB (7168
// columns of bf16) wait for nothing but memory.  Weights (from L1) are asked for
// before the sums that they wait behind.  Only the outputs are rounded (to
// their types); the second norm reads the stream as it was rounded.
template <typename C, typename S, typename W, Mode M, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_residual_kernel(const NormParams p) {
  __shared__ __align__(16) float part[2][kMaxWarps];
  if (threadIdx.x < 2 * kMaxWarps) part[0][threadIdx.x] = 0.f;
  if (blockDim.x == 32) part[1][threadIdx.x] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  Cols<M> c{static_cast<int32_t>(p.cols), static_cast<int32_t>(threadIdx.x),
            static_cast<int32_t>(blockDim.x)};
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  const float2 alpha = both(p.alpha);
  const uint32_t rows = static_cast<uint32_t>(p.rows);
  const uint32_t per = p.gate ? rows / static_cast<uint32_t>(p.gates) : 1u;
  Raw<C> b[NV];
  Raw<S> r[NV];
  auto set_row = [&](Cols<M>& c, uint32_t t) {  // (of every array's row t the same)
    if constexpr (M == kShift) {
      const uintptr_t row = reinterpret_cast<uintptr_t>(static_cast<const C*>(p.block) + t * p.ldb);
      c.phase = static_cast<int32_t>(row / sizeof(C) & 7u);
      c.open = t >= 8 && t + 8 < rows;
    }
  };
  auto fetch = [&](uint32_t t, const Cols<M>& c) {
#pragma unroll
    for (int v = 0; v < NV; ++v) b[v] = load8<true>(static_cast<const C*>(p.block) + t * p.ldb, c, v);
#pragma unroll
    for (int v = 0; v < NV; ++v) r[v] = load8<true>(static_cast<const S*>(p.residual) + t * p.ldr, c, v);
  };
  uint32_t t = blockIdx.x;
  set_row(c, t);
  fetch(t, c);
  while (true) {
    float sum[1];
    float2 sigma = both(1.f);
    Raw<W> w[NV] = {};
#pragma unroll
    for (int v = 0; M == kShift && v < NV; ++v)
      if (!c.inside(v)) {
        trim(b[v], c, v);
        trim(r[v], c, v);
      }
    if (p.w_post) {
#pragma unroll
      for (int v = 0; v < NV; ++v) w[v] = load8_weight(static_cast<const W*>(p.w_post), c, v);
      float2 s = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(b[v].get(i), b[v].get(i), s);
      sum[0] = s.x + s.y;
      block_sum(sum, part[0]);
      sigma = both(rms_inverse(sum[0], inv_cols, p.eps));
    }
    const int64_t goff = p.gate ? t / per * p.cols : 0;
    Raw<S> out[NV];
    float2 s = both(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(b[v].get(i), sigma);
      if (p.w_post) times(f, w[v]);
      if (p.gate) times_w<W>(f, p.gate, goff, c, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = fma2(alpha, r[v].get(i), f[i]);
      out[v] = round8<S>(f);
      store8<true>(static_cast<S*>(p.res_out) + t * p.ldo, c, v, out[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(out[v].get(i), out[v].get(i), s);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) w[v] = load8_weight(static_cast<const W*>(p.w_pre), c, v);
    const uint32_t next = t + gridDim.x;
    Cols<M> c_next = c;
    set_row(c_next, next);
    if (next < rows) fetch(next, c_next);
    sum[0] = s.x + s.y;
    block_sum(sum, part[1]);
    const float2 rho = both(rms_inverse(sum[0], inv_cols, p.eps));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(out[v].get(i), rho);
      times(f, w[v]);
      store8<true>(static_cast<C*>(p.y) + t * p.ldy, c, v, round8<C>(f));
    }
    if (next >= rows) return;
    t = next;
    c = c_next;
    if (!p.w_post && blockDim.x > 32) __syncthreads();  // part[1] is used in every row
  }
}

// ------------------------------------------------------------------ backward

// Rows of block i of n: q each, the first r blocks one more.
struct RowShare {
  uint32_t q, r;
  __host__ __device__ RowShare(uint32_t rows, uint32_t n) : q(rows / n), r(rows - rows / n * n) {}
  __device__ __forceinline__ uint32_t start(uint32_t i) const { return i * q + (i < r ? i : r); }
  // block whose rows hold row t
  __device__ __forceinline__ uint32_t of(uint32_t t) const {
    const uint32_t m = r * (q + 1);
    return t < m ? t / (q + 1) : r + (t - m) / q;
  }
};

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

constexpr int kBackThreads = 512;   // at most

// The sums behind a row's gradient.  With t = w_pre dy and h = w_post g block,
//   D = d_res + rho t - rho^3 mean(t r) r,   dot = sum of h D
//     = sum h d_res + rho sum h t - rho^3 mean(t r) sum h r,
// so that one pass over the row gives all of them, before rho is known.
enum RowSum { kRR, kTR, kBB, kHA, kHT, kHR, kRowSums };

// Eight sums over a warp in nine exchanges: lane l gets that of v[l / 4].
__device__ __forceinline__ float warp_sum8(float (&v)[8]) {
  const uint32_t lane = lane_id();
#pragma unroll
  for (int o = 16, n = 4; n > 0; o >>= 1, n >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// One block of threads goes through its own rows in order.  Rows arrive in
// shared memory by bulk copies, `stages` of them at most (0: rows that do not
// fit, read in place); a thread takes its columns to registers once, where
// they stay across the row's one barrier, behind which the next copy starts.
// (16384 x 7168: all six sums of a row in one pass 315 -> 306 us, the columns in
// registers across one barrier instead of two with re-reads 306 -> 278.)
// A thread also keeps the sums of its columns over the rows and the factors
// w_post g of its columns for the current gate, which every row wants twice (in
// FP32, the first run's in registers, the second's behind the ring).  w_pre (from
// L1) is asked for before the wait for the row, where registers hold it that long.
// `post` (more gates than one): the sums of D b sigma g over finished gates lie
// behind ring and factors, else in the workspace.
// CL: blocks of a cluster that share a row (two for rows longer than a block's
// registers hold, exchanging sums through distributed shared memory).
// kShift: a thread's columns depend on the row's phase, so a gate's rows are
// taken by phase (every `stride`-th row has the same), and after each phase the
// sums go to shared memory by column.  Rows are read in place.
template <typename C, typename S, typename W, Mode M, int NV, int CL>
__global__ void __launch_bounds__(kBackThreads)
    norm_backward_kernel(const NormBackParams p, int stages, bool post) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float part[2][CL * kBackThreads / 32 * 8];
  __shared__ uint64_t full[8];
  __shared__ uint32_t abort_word;
  volatile uint32_t* s_abort = &abort_word;
  // this block's columns: all, or its half in a cluster of two
  const uint32_t rank = CL == 1 ? 0u : cluster_ctarank();
  const int32_t width = static_cast<int32_t>(p.cols);
  const int32_t half = CL == 1 ? width : (width / 8 + 1) / 2 * 8;
  const int32_t off = rank * half, mine = rank == 0 ? half : width - half;
  Cols<M> c{mine, static_cast<int32_t>(threadIdx.x), static_cast<int32_t>(blockDim.x)};
  const Cols<M == kSingle ? M : kWhole> slots{c.cols, c.tid, c.threads};  // of the factors
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  const uint32_t n = gridDim.x / CL, me = blockIdx.x / CL, lane = lane_id();
  const RowShare share(static_cast<uint32_t>(p.rows), n);
  const uint32_t lo = share.start(me), hi = share.start(me + 1);
  const uint32_t cbytes = mine * sizeof(C), sbytes = mine * sizeof(S);
  const uint32_t stage_bytes = 2 * cbytes + 2 * sbytes;
  for (uint32_t i = threadIdx.x; i < CL * kBackThreads / 32 * 16; i += blockDim.x) part[0][i] = 0.f;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    abort_word = 0;
    fence_mbarrier_init();
  }
  if constexpr (CL == 1)
    __syncthreads();
  else
    cluster_sync();  // both blocks' sums are cleared before either adds to them
  pdl_wait();
  pdl_launch_dependents();
  auto issue = [&](uint32_t t, int s) {
    uint8_t* dst = smem + s * stage_bytes;
    mbar_arrive_expect_tx(&full[s], p.d_res ? stage_bytes : stage_bytes - sbytes);
    bulk_load(dst, static_cast<const C*>(p.dy) + t * p.lddy + off, cbytes, &full[s]);
    bulk_load(dst + cbytes, static_cast<const C*>(p.block) + t * p.ldb + off, cbytes, &full[s]);
    bulk_load(dst + 2 * cbytes, static_cast<const S*>(p.res_out) + t * p.ldr + off, sbytes, &full[s]);
    if (p.d_res)
      bulk_load(dst + 2 * cbytes + sbytes, static_cast<const S*>(p.d_res) + t * p.ldd + off, sbytes,
                &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && lo + s < hi; ++s) issue(lo + s, s);

  const uint32_t per = static_cast<uint32_t>(p.gates ? p.rows / p.gates : p.rows);
  const float2 alpha = both(p.alpha);
  // sums over rows of dy r rho and of D b sigma, the latter over the current
  // gate's rows
  float2 pre[NV][4], q[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) pre[v][i] = q[v][i] = both(0.f);
  constexpr int kHeld = M == kShift && NV > 1 ? 0 : 1;       // runs with factors in registers
  Raw<float> held = {{both(1.f), both(1.f), both(1.f), both(1.f)}};
  float* factor = reinterpret_cast<float*>(smem + stages * stage_bytes);
  auto times_factor = [&](float2 (&f)[4], int v) {
    if (v < kHeld)
      times(f, held);
    else if (p.gate || p.w_post)
      times(f, load8(factor, slots, v - kHeld));
  };
  float* past = factor + 8 * (NV - kHeld) * blockDim.x;
  float* finished = post ? past : p.w_post ? ws_post(p, n, me) + off : nullptr;
  auto set_factors = [&](int64_t goff) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Raw<float> r;
      float2 f[4] = {both(1.f), both(1.f), both(1.f), both(1.f)};
      if (p.w_post) times_w<W>(f, p.w_post, off, c, v);
      if (p.gate) times_w<W>(f, p.gate, goff, c, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.f[i] = f[i];
      if (v < kHeld)
        held = r;
      else
        store8(factor, slots, v - kHeld, r);
    }
  };
  const uint32_t group0 = lo / per;
  uint32_t group = group0, left = (group + 1) * per - lo;  // rows left of this gate
  // kShift: the gate's rows [begin, end) of this block, their sums by column
  const uint32_t stride = p.ldb & 1 ? 8u : p.ldb & 2 ? 4u : p.ldb & 4 ? 2u : 1u;
  uint32_t begin = lo, end = hi - lo < left ? hi : lo + left;
  float* pre_sum = past;
  float* q_sum = pre_sum + mine;
  auto set_phase = [&](uint32_t t) {  // (of every array's row t the same)
    if constexpr (M == kShift)
      c.phase = static_cast<int32_t>(
          reinterpret_cast<uintptr_t>(static_cast<const C*>(p.block) + t * p.ldb) / sizeof(C) & 7u);
  };
  if constexpr (M == kShift)  // (the first row's barrier lies before the first use)
    for (int i = c.tid; i < 2 * mine; i += c.threads) pre_sum[i] = 0.f;
  set_phase(lo);
  if (p.gate || p.w_post) set_factors(group * p.cols + off);
  int stage = 0;
  uint32_t phase = 0;
  for (uint32_t t = lo, done = 0; t < hi; ++done) {
    const uint32_t turn = (M == kShift ? done : t) & 1u;
    Raw<S> x[NV], a[NV] = {};
    Raw<C> y[NV], b[NV];
    constexpr bool kAhead = NV == 1 || sizeof(W) == 2;
    Raw<W> w_pre[NV];
#pragma unroll
    for (int v = 0; kAhead && v < NV; ++v) w_pre[v] = load8_weight(static_cast<const W*>(p.w_pre) + off, c, v);
    auto times_pre = [&](float2 (&f)[4], int v) {
      if constexpr (kAhead)
        times(f, w_pre[v]);
      else
        times_w<W>(f, p.w_pre, off, c, v);
    };
    if (stages > 0) {
      mbar_wait(&full[stage], phase, s_abort, p.status, p.wait_limit_ns);
      const uint8_t* src = smem + stage * stage_bytes;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        y[v] = load8(reinterpret_cast<const C*>(src), c, v);
        b[v] = load8(reinterpret_cast<const C*>(src + cbytes), c, v);
        x[v] = load8(reinterpret_cast<const S*>(src + 2 * cbytes), c, v);
        if (p.d_res) a[v] = load8(reinterpret_cast<const S*>(src + 2 * cbytes + sbytes), c, v);
      }
    } else {
      c.open = t >= 8 && t + 8 < static_cast<uint32_t>(p.rows);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        y[v] = load8<true>(static_cast<const C*>(p.dy) + t * p.lddy + off, c, v);
        b[v] = load8<true>(static_cast<const C*>(p.block) + t * p.ldb + off, c, v);
        x[v] = load8<true>(static_cast<const S*>(p.res_out) + t * p.ldr + off, c, v);
        if (p.d_res) a[v] = load8<true>(static_cast<const S*>(p.d_res) + t * p.ldd + off, c, v);
      }
#pragma unroll
      for (int v = 0; M == kShift && v < NV; ++v)
        if (!c.inside(v)) {
          trim(y[v], c, v);
          trim(b[v], c, v);
          trim(x[v], c, v);
          trim(a[v], c, v);
        }
      const uint32_t soon = t + (M == kShift ? stride : 1u);
      if (soon < (M == kShift ? end : hi)) {
        prefetch_row(static_cast<const C*>(p.dy) + soon * p.lddy + off, c);
        prefetch_row(static_cast<const C*>(p.block) + soon * p.ldb + off, c);
        prefetch_row(static_cast<const S*>(p.res_out) + soon * p.ldr + off, c);
        if (p.d_res) prefetch_row(static_cast<const S*>(p.d_res) + soon * p.ldd + off, c);
      }
    }
    float2 s2[kRowSums];
#pragma unroll
    for (int i = 0; i < kRowSums; ++i) s2[i] = both(0.f);
    float2 f[NV][4];                                       // w_pre dy
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[v][i] = y[v].get(i);
      times_pre(f[v], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s2[kRR] = fma2(x[v].get(i), x[v].get(i), s2[kRR]);
        s2[kTR] = fma2(f[v][i], x[v].get(i), s2[kTR]);
      }
      if (p.w_post) {
        float2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = b[v].get(i);
          s2[kBB] = fma2(h[i], h[i], s2[kBB]);
        }
        times_factor(h, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s2[kHA] = fma2(h[i], a[v].get(i), s2[kHA]);
          s2[kHT] = fma2(h[i], f[v][i], s2[kHT]);
          s2[kHR] = fma2(h[i], x[v].get(i), s2[kHR]);
        }
      }
    }
    float sums[8];
#pragma unroll
    for (int i = 0; i < kRowSums; ++i) sums[i] = s2[i].x + s2[i].y;
    sums[6] = sums[7] = 0.f;
    float s = warp_sum8(sums);
    const uint32_t warps = blockDim.x / 32;
    float* to = &part[turn][(rank * warps + warp_id()) * 8 + lane / 4];
    if constexpr (CL == 1) {
      if ((lane & 3) == 0) *to = s;
      __syncthreads();
    } else {
      if ((lane & 3) == 0) {
        store_cluster(to, 0, s);
        store_cluster(to, 1, s);
      }
      cluster_sync();
    }
    // past this barrier the row is in registers
    if (stages > 0) {
      if (threadIdx.x == 0 && t + stages < hi) issue(t + stages, stage);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    s = 0.f;
#pragma unroll
    for (uint32_t w = 0; w < CL * kBackThreads / 32; w += 4)
      if (w < CL * warps) s += part[turn][(w + lane / 8) * 8 + lane % 8];
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
#pragma unroll
    for (int i = 0; i < kRowSums; ++i) sums[i] = __shfl_sync(0xffffffffu, s, i);
    const float rho1 = rms_inverse(sums[kRR], inv_cols, p.eps);
    // (in this order nothing leaves FP32's range before the product does)
    const float k1 = rho1 * (rho1 * (rho1 * (sums[kTR] * inv_cols)));
    float sigma1 = 1.f, m1 = 0.f;
    if (p.w_post) {
      sigma1 = rms_inverse(sums[kBB], inv_cols, p.eps);
      const float dot = sums[kHA] + (rho1 * sums[kHT] - k1 * sums[kHR]);
      m1 = sigma1 * (sigma1 * (sigma1 * (dot * inv_cols)));
    }
    const float2 rho = both(rho1), sigma = both(sigma1), k = both(-k1), m = both(-m1);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 d[4], o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pre[v][i] = fma2(y[v].get(i), mul2(x[v].get(i), rho), pre[v][i]);
        d[i] = fma2(x[v].get(i), k, fma2(rho, f[v][i], a[v].get(i)));
        o[i] = mul2(alpha, d[i]);
        q[v][i] = fma2(d[i], mul2(b[v].get(i), sigma), q[v][i]);
      }
      store8(static_cast<S*>(p.d_residual) + t * p.lddr + off, c, v, round8<S>(o));
      times_factor(d, v);
      if (p.w_post) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = fma2(b[v].get(i), m, mul2(sigma, d[i]));
      }
      store8(static_cast<C*>(p.d_block) + t * p.lddb + off, c, v, round8<C>(d));
    }
    if constexpr (M == kShift) {
      t += stride;
      if (t < end) continue;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (c.has(v, i)) {
            pre_sum[c.at(v, i)] += i % 2 ? pre[v][i / 2].y : pre[v][i / 2].x;
            q_sum[c.at(v, i)] += i % 2 ? q[v][i / 2].y : q[v][i / 2].x;
          }
          if (i % 2) pre[v][i / 2] = q[v][i / 2] = both(0.f);
        }
      // the next phase's first row; a gate's rows end behind its last phase
      const uint32_t next = (t - begin) % stride + 1;
      t = begin + next;
      if (next == stride || t >= end) {
        __syncthreads();
        if (p.gate) {
          const int64_t goff = group * p.cols;
          const bool whole = group * per >= lo && end == (group + 1) * per;
          float* dst = whole ? p.d_gate + goff : ws_gate(p, n, 2 * me + (group == group0 ? 0 : 1));
          const W* w_post = static_cast<const W*>(p.w_post);
          const W* gate = static_cast<const W*>(p.gate) + goff;
          for (int i = c.tid; i < mine; i += c.threads) {
            const float sum = q_sum[i], g = sum * to_float(gate[i]);
            dst[i] = w_post ? sum * to_float(w_post[i]) : sum;
            if (p.gates > 1 && w_post) finished[i] = group != group0 ? finished[i] + g : g;
            q_sum[i] = p.gates > 1 ? 0.f : g;
          }
        }
        if (end == hi) break;
        ++group;
        begin = t = end;
        end = hi - begin < per ? hi : begin + per;
      }
      set_phase(t);
      if (p.gate || p.w_post) set_factors(group * p.cols);
      continue;
    }
    if (--left == 0 || t + 1 == hi) {  // the gate's rows, or this block's, end here
      if (p.gate) {
        const int64_t goff = group * p.cols + off;
        const bool whole = group * per >= lo && left == 0;
        float* dst = whole ? p.d_gate + goff : ws_gate(p, n, 2 * me + (group == group0 ? 0 : 1)) + off;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float2 dg[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) dg[i] = q[v][i];
          if (p.w_post) times_w<W>(dg, p.w_post, off, c, v);
          Raw<float> out;
#pragma unroll
          for (int i = 0; i < 4; ++i) out.f[i] = dg[i];
          store8(dst, c, v, out);
          times_w<W>(q[v], p.gate, goff, c, v);
          if (p.gates > 1) {
            if (p.w_post) {
              if (group != group0) out = load8(finished, c, v);
#pragma unroll
              for (int i = 0; i < 4; ++i) out.f[i] = group != group0 ? add2(out.f[i], q[v][i]) : q[v][i];
              store8(finished, c, v, out);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) q[v][i] = both(0.f);
          }
        }
      }
      ++group;
      left = per;
      if (p.gate && t + 1 < hi) set_factors(group * p.cols + off);
    }
    ++t;
  }
  if constexpr (M == kShift) {
    float *pre_out = ws_pre(p, me), *post_out = ws_post(p, n, me);
    for (int i = c.tid; i < mine; i += c.threads) {
      pre_out[i] = pre_sum[i];
      if (p.w_post && p.gates <= 1) post_out[i] = q_sum[i];
    }
    return;
  }
  if (stages > 0 && *s_abort) {  // a wait gave up: copies still in flight must land first
    for (uint32_t s = 0; s < static_cast<uint32_t>(stages) && lo + s < hi; ++s)
      mbar_wait(&full[s], (hi - lo - 1 - s) / stages & 1u, s_abort, p.status, p.wait_limit_ns,
                true);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    Raw<float> out;
#pragma unroll
    for (int i = 0; i < 4; ++i) out.f[i] = pre[v][i];
    store8(ws_pre(p, me) + off, c, v, out);
    if (p.w_post && (post || p.gates <= 1)) {
      if (post) {
        out = load8(finished, c, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) out.f[i] = q[v][i];
      }
      store8(ws_post(p, n, me) + off, c, v, out);
    }
  }
}

// The gradient for rows of more than 4096 columns that neither lie on 16-byte
// boundaries nor can go by phase: element by element (16384 x 5001: 700 us, a
// fifth of the copy bandwidth, bound by its accesses; shorter ones keep their
// columns in registers, 16384 x 4095: 404 us, here 586), with the column sums of w_pre and D b sigma and the row's u in shared memory
// (cols floats each).  Sums over finished gates (gates > 1) grow in the
// workspace.  A thread goes through the same columns everywhere, so no two
// threads touch the same sum.
template <typename C, typename S>
__global__ void __launch_bounds__(kBackThreads)
    norm_backward_single_kernel(const NormBackParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float part[2][3 * kMaxWarps];
  const int cols = static_cast<int>(p.cols), tid = static_cast<int>(threadIdx.x);
  const int step = static_cast<int>(blockDim.x);
  const float inv_cols = 1.f / static_cast<float>(p.cols);
  const uint32_t n = gridDim.x, me = blockIdx.x;
  const RowShare share(static_cast<uint32_t>(p.rows), n);
  const uint32_t lo = share.start(me), hi = share.start(me + 1);
  const bool many = p.gates > 1;
  float* pre = reinterpret_cast<float*>(smem);
  float* q = pre + cols;
  float* u_row = q + cols;
  float* post_out = ws_post(p, n, me);
  for (int i = tid; i < 6 * kMaxWarps; i += step) part[0][i] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  for (int c = tid; c < cols; c += step) {
    pre[c] = q[c] = 0.f;
    if (many) post_out[c] = 0.f;
  }
  auto weight = [&](const void* w, int64_t i) {
    return p.w_fp32 ? static_cast<const float*>(w)[i] : to_float(static_cast<const bf16*>(w)[i]);
  };
  const uint32_t per = static_cast<uint32_t>(p.gates ? p.rows / p.gates : p.rows);
  const uint32_t group0 = lo / per;
  uint32_t group = group0, left = (group + 1) * per - lo;
  for (uint32_t t = lo; t < hi; ++t) {
    const C* dy = static_cast<const C*>(p.dy) + t * p.lddy;
    const C* block = static_cast<const C*>(p.block) + t * p.ldb;
    const S* res = static_cast<const S*>(p.res_out) + t * p.ldr;
    const S* dres = p.d_res ? static_cast<const S*>(p.d_res) + t * p.ldd : nullptr;
    const int64_t goff = group * p.cols;
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = tid; c < cols; c += step) {
      const float x = to_float(res[c]), b = to_float(block[c]);
      sum[0] += x * x;
      sum[1] += to_float(dy[c]) * weight(p.w_pre, c) * x;
      sum[2] += b * b;
    }
    block_sum(sum, part[0]);
    const float rho = rms_inverse(sum[0], inv_cols, p.eps);
    const float sigma = p.w_post ? rms_inverse(sum[2], inv_cols, p.eps) : 1.f;
    const float k = rho * (rho * (rho * (sum[1] * inv_cols)));
    float dot[1] = {0.f};
#pragma unroll 2
    for (int c = tid; c < cols; c += step) {
      const float x = to_float(res[c]), y = to_float(dy[c]), b = to_float(block[c]);
      const float d = (dres ? to_float(dres[c]) : 0.f) + (rho * (y * weight(p.w_pre, c)) - x * k);
      store1(static_cast<S*>(p.d_residual) + t * p.lddr + c, p.alpha * d);
      pre[c] += y * (x * rho);
      q[c] += d * (b * sigma);
      float u = d;
      if (p.gate) u *= weight(p.gate, goff + c);
      if (p.w_post) u *= weight(p.w_post, c);
      dot[0] += u * b;
      u_row[c] = u;
    }
    float m = 0.f;
    if (p.w_post) {
      block_sum(dot, part[1]);
      m = sigma * (sigma * (sigma * (dot[0] * inv_cols)));
    }
#pragma unroll 2
    for (int c = tid; c < cols; c += step) {
      const float u = u_row[c];
      store1(static_cast<C*>(p.d_block) + t * p.lddb + c,
             p.w_post ? sigma * u - to_float(block[c]) * m : u);
    }
    if (!p.w_post && blockDim.x > 32) __syncthreads();  // part[0] is used in every row
    if (--left == 0 || t + 1 == hi) {
      if (p.gate) {
        const bool whole = group * per >= lo && t + 1 == (group + 1) * per;
        float* dst = whole ? p.d_gate + goff : ws_gate(p, n, 2 * me + (group == group0 ? 0 : 1));
        for (int c = tid; c < cols; c += step) {
          const float g = q[c] * weight(p.gate, goff + c);
          dst[c] = p.w_post ? q[c] * weight(p.w_post, c) : q[c];
          if (many) post_out[c] += g;
          q[c] = many ? 0.f : g;
        }
      }
      ++group;
      left = per;
    }
  }
  float* pre_out = ws_pre(p, me);
  for (int c = tid; c < cols; c += step) {
    pre_out[c] = pre[c];
    if (p.w_post && !many) post_out[c] = q[c];
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
bool whole(int64_t cols, int nv) { return cols == 8 * static_cast<int64_t>(nv) * row_threads(cols, nv); }

// Blocks of a kernel that an SM holds at once, asked of the runtime once per
// device and number of threads.
class Fit {
 public:
  template <typename K>
  int of(K kern, int threads) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevs) return 1;
    std::atomic<int>& known = fit_[dev][threads / 32];
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) != cudaSuccess || n < 1)
        n = 1;
      known.store(n, std::memory_order_relaxed);
    }
    return n;
  }

 private:
  static constexpr int kDevs = 64;
  std::atomic<int> fit_[kDevs][33] = {};
};

template <typename C, typename S, typename W, Mode M, int NV, int MAXT>
cudaError_t forward_impl(const NormParams& p, int num_sms, cudaStream_t stream) {
  static Fit fit;
  const int threads = row_threads(p.cols + (M == kShift ? 7 : 0), NV);
  auto kern = norm_residual_kernel<C, S, W, M, NV, MAXT>;
  int64_t grid = p.rows;
  if (grid > num_sms) {
    const int64_t most = static_cast<int64_t>(num_sms) * fit.of(kern, threads);
    grid = grid < most ? grid : most;
  }
  return launch(kern, dim3(static_cast<unsigned>(grid)), threads, 0, stream, p);
}

// (kWhole spares the test for the row's end: 16384 x 7168 157 us against 162.)
template <typename C, typename S, typename W, int NV, int MAXT>
cudaError_t forward_runs(const NormParams& p, NormRows kind, int num_sms, cudaStream_t stream) {
  if (kind == NormRows::kShifted) return forward_impl<C, S, W, kShift, NV, MAXT>(p, num_sms, stream);
  return whole(p.cols, NV) ? forward_impl<C, S, W, kWhole, NV, MAXT>(p, num_sms, stream)
                           : forward_impl<C, S, W, kRuns, NV, MAXT>(p, num_sms, stream);
}

// Runs of eight columns a thread: one for short rows, which several blocks of
// threads on an SM then go through side by side (16384 rows of bf16, us: 256
// columns 8.0, with two runs 9.0; 1024 columns 23.3 against 22.7, but one row
// 1.58 against 1.73); up to 4096 two (8192 rows of 2048: 22.5, with one 25.5,
// with four 23.6); above that four (16384 x 7168: 157, with one 238).
// Shifted rows load every weight in two pieces and move it, which waits: one
// run to 2048 (777 x 1111: 4.3 us, with two 5.2; 16384 x 2049: 83.6 and 76.6,
// now 69.8).  Element by element the same rows take 5.7 and 135 us.
template <typename C, typename S, typename W>
cudaError_t forward(const NormParams& p, NormRows kind, int num_sms, cudaStream_t stream) {
  if (kind == NormRows::kAny)
    return p.cols <= 4096 ? forward_impl<C, S, W, kSingle, 2, 256>(p, num_sms, stream)
                          : forward_impl<C, S, W, kSingle, 2, 1024>(p, num_sms, stream);
  const int64_t cols = p.cols + (kind == NormRows::kShifted ? 7 : 0);
  if (cols <= (kind == NormRows::kShifted ? 2048 : 1024))
    return forward_runs<C, S, W, 1, 256>(p, kind, num_sms, stream);
  if (cols <= 4096) return forward_runs<C, S, W, 2, 256>(p, kind, num_sms, stream);
  return forward_runs<C, S, W, 4, 512>(p, kind, num_sms, stream);
}

constexpr int kMaxSms = 192;         // workspaces are sized for this many
// Shared memory for rings, factors and sums of one of `fit` blocks on an SM (228 KB
// in all; a block has 2 KB of its own beside these).  One block alone takes no
// more than 161 KB: what it leaves is L1, where w_pre is read for every row
// (16384 x 7168: a ring of two rows 218 us, of three 224 and with all of the
// memory 234; x 12288: 538, with a row more 577 to 637; all bf16).  Rows of
// which no two fit in it are read in place: FP32 blocks from 4840 columns on (from
// 9672 in a cluster), bf16 blocks on an FP32 stream from 6320 (12632).  For
// those a ring of two in 206 KB is faster where it fits (8192 x 5120 FP32: 209 us
// in place, 191; x 6144: 239, 216; x 6400 on an FP32 stream: 177, 165; x 7168:
// 179, 174), which this one limit does not give them; bf16 x 7168 115, with 206 KB 118.
constexpr size_t kSmemBytes = 161 * 1024;
constexpr size_t kSmemMost = 12 * 16384;  // (row by row element by element)
constexpr size_t smem_of(int fit) {
  const size_t share = 228 * 1024 / fit - 2304;
  return share < kSmemBytes ? share : kSmemBytes;
}

// How a gradient is run: runs of eight columns a thread holds (0: the kernel
// that goes element by element), blocks that share a row, threads of a block,
// rows on an SM side by side (clusters: on two), rows of the ring, bytes of
// shared memory, and bytes more for the sums over finished gates (0: too many).
struct BackPlan {
  int runs, cluster, threads, fit, stages;
  size_t smem, post;
};
constexpr int64_t kOneRun = 8 * kBackThreads;
constexpr int64_t kShiftCols = 2 * kOneRun - 7;  // what two runs hold wherever they begin
BackPlan backward_plan(int64_t rows, int64_t cols, int64_t gates, bool c_fp32, bool s_fp32, NormRows kind) {
  BackPlan p;
  const bool vec = kind == NormRows::kAligned;
  if (kind == NormRows::kShifted) {
    p.cluster = 1, p.stages = 0, p.post = 0;
    p.runs = cols + 7 <= kOneRun ? 1 : 2;
    if (p.runs == 1 && kBackThreads % row_threads(cols + 7, 1) >= kBackThreads / 4) p.runs = 2;
    p.threads = row_threads(cols + 7, p.runs);
    p.smem = static_cast<size_t>(cols) * 8 + (p.runs == 2 ? 64 * static_cast<size_t>(p.threads) : 0);
    p.fit = kBackThreads / p.threads;
    p.fit = p.fit > 8 ? 8 : p.fit;
    while (p.fit > 1 && p.smem > smem_of(p.fit)) --p.fit;
    return p;
  }
  if (!vec && cols > kOneRun) {  // by shared memory
    p.runs = 0, p.cluster = 1, p.stages = 0;
    p.threads = kBackThreads;
    p.smem = static_cast<size_t>(cols) * 12;
    p.post = 0;
    p.fit = p.smem <= smem_of(2) ? 2 : 1;
    return p;
  }
  // by registers (128 a thread) and rings.  A thread holds two
  // runs where a row takes more than 512; where blocks with one would leave a
  // quarter of the SM's 512 threads idle (16384 x 2560 in bf16: 89 us, with one run
  // 161; x 1536: 58 and 84); and with many rows where the SM then holds two such
  // blocks with their rings instead of one (x 4096: 130 and 145; x 3584: 115 and
  // 144).  Else one (100 x 4096: 7.2, with two 8.6; 16384 x 2048: 73 and 76).
  p.cluster = cols <= 2 * kOneRun ? 1 : 2;
  const int64_t mine = p.cluster == 1 ? cols : (cols / 8 + 1) / 2 * 8;
  p.runs = mine <= kOneRun ? 1 : 2;
  const size_t stage = mine * 2 * ((c_fp32 ? 4 : 2) + (s_fp32 ? 4 : 2));
  const size_t factors = 32 * static_cast<size_t>(row_threads(mine, 2));  // of two runs: the second's
  if (vec && p.runs == 1 &&
      (kBackThreads % row_threads(mine, 1) >= kBackThreads / 4 ||
       (mine > 2048 && rows > 2 * kMaxSms && factors + 3 * stage <= smem_of(2))))
    p.runs = 2;
  p.threads = row_threads(mine, p.runs);
  p.fit = kBackThreads / p.threads;
  p.fit = p.fit > 8 ? 8 : p.fit;
  p.stages = 0;
  p.post = gates > 1 ? static_cast<size_t>(mine) * 4 : 0;
  p.smem = p.runs == 2 ? factors : 0;
  if (vec) {
    // Rows of a ring: two for short rows, of which an SM has several under way
    // (16384 x 2048, FP32 stream: 95 us, with three 108, with four 105; x 1024:
    // 52.8 and 56.5), else three or four (x 4096: 130, with two 141).
    const bool few = mine <= 2560;
    while (p.fit > 1 && p.smem + (few ? 2 : 3) * stage > smem_of(p.fit)) --p.fit;
    const size_t ring = (smem_of(p.fit) - p.smem) / stage, most = few ? 2 : 4;
    p.stages = ring < 2 ? 0 : static_cast<int>(ring < most ? ring : most);
    p.smem += p.stages * stage;
  }
  if (p.smem + p.post > smem_of(p.fit)) p.post = 0;
  return p;
}

// Blocks of the gradient: those that fit the SMs.
// (Blocks that share a row count as one.)
int64_t backward_blocks(int64_t rows, int num_sms, const BackPlan& plan) {
  const int64_t most = static_cast<int64_t>(num_sms / plan.cluster) * plan.fit;
  return rows < most ? rows : most;
}

template <typename K>
cudaError_t allow_smem(PerDeviceOnce& setup, K kern) {
  return setup.run([&]() -> cudaError_t {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemMost));
  });
}

template <typename C, typename S, typename W, Mode M, int NV, int CL>
cudaError_t backward_impl(const NormBackParams& p, const BackPlan& plan, int64_t n,
                          cudaStream_t stream) {
  static PerDeviceOnce setup;
  auto kern = norm_backward_kernel<C, S, W, M, NV, CL>;
  const cudaError_t err = allow_smem(setup, kern);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(n * CL));
  cfg.blockDim = dim3(plan.threads);
  cfg.dynamicSmemBytes = plan.smem + plan.post;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = CL == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kern, p, plan.stages, plan.post > 0);
}

template <typename C, typename S>
cudaError_t backward_single(const NormBackParams& p, const BackPlan& plan, int64_t n,
                            cudaStream_t stream) {
  static PerDeviceOnce setup;
  auto kern = norm_backward_single_kernel<C, S>;
  const cudaError_t err = allow_smem(setup, kern);
  if (err != cudaSuccess) return err;
  return launch(kern, dim3(static_cast<unsigned>(n)), plan.threads, plan.smem, stream, p);
}

template <typename C, typename S, typename W>
cudaError_t backward(const NormBackParams& p, NormRows kind, const BackPlan& plan, int64_t n,
                     cudaStream_t stream) {
  if (plan.runs == 0) return backward_single<C, S>(p, plan, n, stream);
  if (kind == NormRows::kAny) return backward_impl<C, S, W, kSingle, 1, 1>(p, plan, n, stream);
  if (kind == NormRows::kShifted)
    return plan.runs == 1 ? backward_impl<C, S, W, kShift, 1, 1>(p, plan, n, stream)
                          : backward_impl<C, S, W, kShift, 2, 1>(p, plan, n, stream);
  if (plan.cluster == 2) return backward_impl<C, S, W, kRuns, 2, 2>(p, plan, n, stream);
  if (plan.runs == 1)
    return whole(p.cols, 1) ? backward_impl<C, S, W, kWhole, 1, 1>(p, plan, n, stream)
                            : backward_impl<C, S, W, kRuns, 1, 1>(p, plan, n, stream);
  return whole(p.cols, 2) ? backward_impl<C, S, W, kWhole, 2, 1>(p, plan, n, stream)
                          : backward_impl<C, S, W, kRuns, 2, 1>(p, plan, n, stream);
}

}  // namespace

// Forward and gradient for blocks of type C and a stream of type S.
template <typename C, typename S>
cudaError_t norm_forward_of(const NormParams& p, NormRows kind, int num_sms, cudaStream_t stream) {
  return p.w_fp32 ? forward<C, S, float>(p, kind, num_sms, stream)
                  : forward<C, S, bf16>(p, kind, num_sms, stream);
}
template <typename C, typename S>
cudaError_t norm_backward_of(const NormBackParams& p, NormRows kind, int64_t n, cudaStream_t stream) {
  const BackPlan plan = backward_plan(p.rows, p.cols, p.gates, p.c_fp32, p.s_fp32, kind);
  return p.w_fp32 ? backward<C, S, float>(p, kind, plan, n, stream)
                  : backward<C, S, bf16>(p, kind, plan, n, stream);
}

}  // namespace mx
