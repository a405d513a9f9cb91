// rotate_kernel.cuh -- the norms of query and key heads with the rotation by
// position, in one pass, and their gradient: kernels and their launches, which
// rotate.cu, rotate_f32.cu, rotate_back.cu and rotate_back_f32.cu instantiate by type
// and direction (four files, so that they compile side by side).  For every token t
// and head row x of D channels:
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
// only exchange is the sum (the gradient: two sums) over the row.  Blocks stay on
// the SMs and go from item to item (some tokens' heads); a row's registers take
// the next item's row as soon as they are read, so that loads are always on their
// way.  Arithmetic is FP32, two channels an instruction.  Angles are shared by a
// token's heads: a block computes the cosines and sines of its next tokens in shared
// memory beside the rows of these.
// Measured on one GB300 (part of the measured copy bandwidth, 6.78 TB/s): 16384
// tokens x 40 heads of 128, bf16: 53 us, 0.93; gradient 97 us, 0.77 (59 % of issue
// slots busy at 16 warps an SM: the registers of five values a channel); one token
// 2.7 us in a graph, 5.3 called.  Half of the channels rotated: 54 and 107 us; 40
// heads of 80 (lanes without channels) 59 and 137; 52 of 128 channels rotated (not
// a multiple of 8: single channels, twice the lanes and four times the accesses) 119
// and 180.
//
// An angle is a product in turns: the frequency becomes a 64-bit fraction of a turn
// per position, the product with the position keeps its low 64 bits, which are the
// fraction of a turn -- in integers, exact to the position times 2^-64 turns (the
// fraction is cut off) and 2^-69 of the frequency in turns (2^66 / (2 pi) is rounded),
// however far that is.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTable = 1024;  // angles of an item's tokens

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

// Cosine and sine, times the scale, of an angle given as a fraction of a turn in
// units of 2^-64: its top 32 bits, rounded, are signed half turns.
__device__ __forceinline__ float2 unit_of(uint64_t turn, float scale) {
  const int32_t top = static_cast<int32_t>((turn + (1ull << 31)) >> 32);
  float s, c;
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ uint64_t position_of(const RotateParams& p, int32_t token) {
  return static_cast<uint64_t>(
      p.positions_64 ? static_cast<const int64_t*>(p.positions)[token]
                     : static_cast<int64_t>(static_cast<const int32_t*>(p.positions)[token]));
}

__device__ __forceinline__ float weight_of(const void* w, int32_t f32, int32_t i) {
  return f32 ? static_cast<const float*>(w)[i]
             : __bfloat162float(static_cast<const bf16*>(w)[i]);
}

// ------------------------------------------------------------------ a lane's share of a row

// A slot is two chunks of C channels, at a and b, whose values a lane holds as
// pairs of floats: with C = 4 the first channels of four pairs, then their
// second ones; with C = 1 a pair (b may be missing at the end of an odd row).
// How much of it is known when compiled: in a full row (2 C LPR S channels) every slot
// has its channels, in a whole one all of them are rotated too, so that their
// distances are constants.
enum Rows { kAny, kFull, kWhole };
template <int C_, int LPR_, int S_, bool INTER_, Rows ROWS>
struct Lane {
  static constexpr int C = C_, LPR = LPR_, S = S_;
  static constexpr bool INTER = INTER_, WHOLE = ROWS == kWhole, FULL = ROWS != kAny;
  static constexpr int kHalves = C == 4 ? 4 : 1;  // float2 of a slot
  static constexpr int kHalf = C * LPR * S;       // pairs of a whole row
  int32_t first;         // WHOLE: first pair
  int32_t at_a[S], at_b[S];  // else: first channels of the chunks, -1 where there is none
  int32_t at_pair[S];        // first pair, or -1: not rotated
  __device__ __forceinline__ Lane(const RotateParams& p, int32_t lane) : first(C * lane) {
    if constexpr (!WHOLE) {
      const int32_t turned = p.rotary / (2 * C);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int32_t g = lane + s * LPR;
        at_pair[s] = g < turned ? C * g : -1;
        if (g < turned) {
          at_a[s] = INTER ? 2 * C * g : C * g;
          at_b[s] = INTER ? at_a[s] + C : p.rotary / 2 + C * g;
        } else {
          at_a[s] = p.rotary + 2 * C * (g - turned);
          at_b[s] = at_a[s] + C;
          if (!FULL && at_a[s] >= p.dim) at_a[s] = -1;
          if (!FULL && at_b[s] >= p.dim) at_b[s] = -1;
        }
      }
    }
  }
  __device__ __forceinline__ int32_t pair(int s) const {
    return WHOLE ? first + s * C * LPR : at_pair[s];
  }
  __device__ __forceinline__ int32_t a(int s) const {
    return WHOLE ? (INTER ? 2 * pair(s) : pair(s)) : at_a[s];
  }
  __device__ __forceinline__ int32_t b(int s) const {
    return WHOLE ? (INTER ? 2 * pair(s) + C : pair(s) + kHalf) : at_b[s];
  }
  __device__ __forceinline__ bool has_a(int s) const { return FULL || at_a[s] >= 0; }
  __device__ __forceinline__ bool has_b(int s) const { return FULL || at_b[s] >= 0; }
  __device__ __forceinline__ bool turns(int s) const { return WHOLE || at_pair[s] >= 0; }
  // Channel of value e (0 .. 2 C - 1, in the order held) of slot s, or -1.
  __device__ __forceinline__ int32_t channel(int s, int e) const {
    if (C == 1) return e == 0 ? a(s) : b(s);
    if (!has_a(s)) return -1;
    if (INTER) return a(s) + (e < C ? 2 * e : 2 * (e - C) + 1);
    return e < C ? a(s) + e : b(s) + e - C;
  }
};

// A slot's values as loaded.
template <typename T, int C>
struct Raw;
template <>
struct Raw<bf16, 4> {
  uint2 a, b;
};
template <>
struct Raw<float, 4> {
  float4 a, b;
};
template <typename T>
struct Raw<T, 1> {
  T a, b;
};

template <typename T, int C, typename L, int S>
__device__ __forceinline__ void load_row(Raw<T, C> (&r)[S], const T* p, const L& l) {
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (l.has_a(s)) r[s].a = *reinterpret_cast<const decltype(r[s].a)*>(p + l.a(s));
    if (l.has_b(s)) r[s].b = *reinterpret_cast<const decltype(r[s].b)*>(p + l.b(s));
  }
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <bool INTER, typename L>
__device__ __forceinline__ void values(const Raw<bf16, 4>& r, int s, const L& l, float2* h) {
  if (!l.has_a(s)) {
    h[0] = h[1] = h[2] = h[3] = both(0.f);
  } else if (INTER) {
    h[0] = make_float2(low(r.a.x), low(r.a.y)), h[1] = make_float2(low(r.b.x), low(r.b.y));
    h[2] = make_float2(high(r.a.x), high(r.a.y)), h[3] = make_float2(high(r.b.x), high(r.b.y));
  } else {
    h[0] = unpack2(r.a.x), h[1] = unpack2(r.a.y), h[2] = unpack2(r.b.x), h[3] = unpack2(r.b.y);
  }
}
template <bool INTER, typename L>
__device__ __forceinline__ void values(const Raw<float, 4>& r, int s, const L& l, float2* h) {
  if (!l.has_a(s)) {
    h[0] = h[1] = h[2] = h[3] = both(0.f);
  } else if (INTER) {
    h[0] = make_float2(r.a.x, r.a.z), h[1] = make_float2(r.b.x, r.b.z);
    h[2] = make_float2(r.a.y, r.a.w), h[3] = make_float2(r.b.y, r.b.w);
  } else {
    h[0] = make_float2(r.a.x, r.a.y), h[1] = make_float2(r.a.z, r.a.w);
    h[2] = make_float2(r.b.x, r.b.y), h[3] = make_float2(r.b.z, r.b.w);
  }
}
__device__ __forceinline__ float wide(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float wide(float v) { return v; }
template <bool INTER, typename T, typename L>
__device__ __forceinline__ void values(const Raw<T, 1>& r, int s, const L& l, float2* h) {
  h[0] = make_float2(!l.has_a(s) ? 0.f : wide(r.a), !l.has_b(s) ? 0.f : wide(r.b));
}

template <bool INTER, typename L>
__device__ __forceinline__ void store(bf16* p, int s, const L& l, const float2 (&h)[4]) {
  if (!l.has_a(s)) return;
  uint2 a, b;
  if (INTER) {
    a = make_uint2(pack2(make_float2(h[0].x, h[2].x)), pack2(make_float2(h[0].y, h[2].y)));
    b = make_uint2(pack2(make_float2(h[1].x, h[3].x)), pack2(make_float2(h[1].y, h[3].y)));
  } else {
    a = make_uint2(pack2(h[0]), pack2(h[1]));
    b = make_uint2(pack2(h[2]), pack2(h[3]));
  }
  *reinterpret_cast<uint2*>(p + l.a(s)) = a;
  *reinterpret_cast<uint2*>(p + l.b(s)) = b;
}
template <bool INTER, typename L>
__device__ __forceinline__ void store(float* p, int s, const L& l, const float2 (&h)[4]) {
  if (!l.has_a(s)) return;
  float4 a, b;
  if (INTER) {
    a = make_float4(h[0].x, h[2].x, h[0].y, h[2].y);
    b = make_float4(h[1].x, h[3].x, h[1].y, h[3].y);
  } else {
    a = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    b = make_float4(h[2].x, h[2].y, h[3].x, h[3].y);
  }
  *reinterpret_cast<float4*>(p + l.a(s)) = a;
  *reinterpret_cast<float4*>(p + l.b(s)) = b;
}
__device__ __forceinline__ void store1(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
template <bool INTER, typename T, typename L>
__device__ __forceinline__ void store(T* p, int s, const L& l, const float2 (&h)[1]) {
  if (l.has_a(s)) store1(p + l.a(s), h[0].x);
  if (l.has_b(s)) store1(p + l.b(s), h[0].y);
}

// Turns a slot's pairs: c and s are the cosines and sines of its first pair on.
template <bool BACK>
__device__ __forceinline__ void turn(float2 (&h)[4], const float* c, const float* s) {
  const float4 c4 = *reinterpret_cast<const float4*>(c), s4 = *reinterpret_cast<const float4*>(s);
  const float2 cc[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
  const float2 ss[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 minus = make_float2(-ss[i].x, -ss[i].y);
    const float2 u = h[i], v = h[2 + i];
    h[i] = fma2(v, BACK ? ss[i] : minus, mul2(u, cc[i]));
    h[2 + i] = fma2(u, BACK ? minus : ss[i], mul2(v, cc[i]));
  }
}
template <bool BACK>
__device__ __forceinline__ void turn(float2 (&h)[1], const float* c, const float* s) {
  const float sn = BACK ? -*s : *s;
  h[0] = make_float2(fmaf(-h[0].y, sn, h[0].x * *c), fmaf(h[0].x, sn, h[0].y * *c));
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// ------------------------------------------------------------------ work of a block

// An item of work: tokens [t0, t0 + nt) x heads [h0, h0 + nh), queries' first.  Its
// rows go round the groups of lanes; the rows of a group have the same places in
// every item.
struct Item {
  int32_t t0, nt, h0, nh;
};
__device__ __forceinline__ Item item_of(const RotateParams& p, int32_t i) {
  Item it;
  const int32_t g = p.chunks_of_heads == 1 ? i : i / p.chunks_of_heads;
  it.t0 = g * p.tokens_per_item;
  it.nt = min(p.tokens_per_item, p.tokens - it.t0);
  it.h0 = (i - g * p.chunks_of_heads) * p.heads_per_item;
  it.nh = min(p.heads_per_item, p.q_heads + p.k_heads - it.h0);
  return it;
}

// What all items of a block share, in shared memory: the frequencies as fractions
// of a turn, the weights in the order that lanes hold values (queries', then
// keys'), two tables of cosines and sines [token][2][pairs].
template <typename L>
struct Shared {
  static constexpr int C = L::C, LPR = L::LPR, S = L::S;
  static constexpr int kRow = 2 * C * LPR * S;  // values of a row's slots
  uint64_t* turns;
  float* weights;
  float* table;
  int32_t half, table_size;
  __device__ __forceinline__ Shared(const RotateParams& p, uint8_t* smem) {
    half = p.rotary / 2;
    weights = reinterpret_cast<float*>(smem);
    table = weights + 2 * kRow;
    table_size = p.tokens_per_item * 2 * half;
    turns = reinterpret_cast<uint64_t*>(table + 2 * table_size);
  }
  static size_t bytes(const RotateParams& p) {
    return sizeof(float) * (2 * kRow + 4 * p.tokens_per_item * (p.rotary / 2)) +
           sizeof(uint64_t) * (p.rotary / 2);
  }
  // A lane's weights: four values, then the next four, so that neighbouring lanes
  // read neighbouring 16 bytes.
  __device__ __forceinline__ const float2* weights_of(bool is_q, int32_t lane) const {
    return reinterpret_cast<const float2*>(weights + (is_q ? 0 : kRow)) + lane * (C == 4 ? 2 : 1);
  }
  static __device__ __forceinline__ constexpr int weight(int s, int j) {
    return C == 4 ? (2 * s + j / 2) * 2 * LPR + j % 2 : s * LPR;
  }
  __device__ __forceinline__ void fill_once(const RotateParams& p, const L& l) {
    for (int32_t i = threadIdx.x; i < half; i += kThreads) turns[i] = turns_of(p.frequencies[i]);
    if (threadIdx.x < 2 * LPR) {
      const bool is_k = threadIdx.x >= LPR;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 2 * C; ++e) {
          const int32_t at = l.channel(s, e);
          float* w = weights + (is_k ? kRow : 0) + threadIdx.x % LPR * (C == 4 ? 4 : 2);
          w[2 * weight(s, e / 2) + e % 2] =
              at < 0 ? 0.f : weight_of(is_k ? p.w_k : p.w_q, p.w_fp32, at);
        }
    }
  }
  // Cosines and sines of an item's tokens; `first` is the position that the
  // thread's first entry needs.
  __device__ __forceinline__ void fill(const RotateParams& p, const Item& it, int buf,
                                       uint64_t first) {
    float* tab = table + buf * table_size;
    for (int32_t i = threadIdx.x; i < it.nt * half; i += kThreads) {
      const int32_t t = i < half ? 0 : i / half, f = i - t * half;
      const uint64_t pos = i < kThreads ? first : position_of(p, it.t0 + t);
      const float2 u = unit_of(pos * turns[f], p.scale);
      tab[t * 2 * half + f] = u.x;
      tab[t * 2 * half + half + f] = u.y;
    }
  }
  __device__ __forceinline__ uint64_t first_position(const RotateParams& p, const Item& it) const {
    const int32_t i = threadIdx.x;
    return i < it.nt * half ? position_of(p, it.t0 + (i < half ? 0 : i / half)) : 0;
  }
};

// Registers that a row's values take as loaded.
template <typename T, int C, int S>
constexpr int raw_regs() {
  return C == 1 ? 2 * S : static_cast<int>(sizeof(T)) * 2 * C * S / 4;
}
// Rows under way in a thread: as many as 32 registers hold (forward), or 20 of each
// array (gradient).
template <typename T, int C, int S, bool BACK>
constexpr int rows_ahead() {
  constexpr int n = (BACK ? 20 : 32) / raw_regs<T, C, S>();
  return n > 5 ? 5 : n < 1 ? 1 : n;
}
// Blocks of an SM that the registers are shared out for.
template <int C, int S, bool BACK>
constexpr int resident() {
  return BACK ? (C * S >= 8 || S >= 4 ? 1 : 2) : (C == 1 && S >= 4) || C * S > 8 ? 2 : 3;
}

// The rows of one kind of array: queries' heads and, behind them, keys', with
// strides in bytes.
template <typename T>
struct Heads {
  char *q, *k;  // (k as if the keys' heads were numbered on from the queries')
  int32_t q_st, q_sh, k_st, k_sh;
  __device__ __forceinline__ Heads(const void* q_, const void* k_, int64_t qt, int64_t qh,
                                   int64_t kt, int64_t kh, int32_t q_heads)
      : q(static_cast<char*>(const_cast<void*>(q_))),
        k(static_cast<char*>(const_cast<void*>(k_)) - q_heads * kh * int64_t{sizeof(T)}),
        q_st(static_cast<int32_t>(qt * sizeof(T))), q_sh(static_cast<int32_t>(qh * sizeof(T))),
        k_st(static_cast<int32_t>(kt * sizeof(T))), k_sh(static_cast<int32_t>(kh * sizeof(T))) {}
  __device__ __forceinline__ T* at(int32_t token, int32_t h, bool is_q) const {
    return reinterpret_cast<T*>((is_q ? q : k) + static_cast<int64_t>(token) * (is_q ? q_st : k_st) +
                                static_cast<int64_t>(h) * (is_q ? q_sh : k_sh));
  }
};

template <typename T, typename LaneT>
__global__ void __launch_bounds__(kThreads, (resident<LaneT::C, LaneT::S, false>()))
    norm_rotate_kernel(const RotateParams p) {
  using L = LaneT;
  constexpr int C = L::C, LPR = L::LPR, S = L::S, H = L::kHalves, G = kThreads / LPR;
  constexpr int U = rows_ahead<T, C, S, false>();
  extern __shared__ __align__(16) uint8_t smem[];
  const int32_t lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const L l(p, lane);
  Shared<L> sh(p, smem);
  // rows of an item: row r is token r / heads_per_item, head r % heads_per_item
  int32_t tu[U], hu[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    tu[u] = (group + u * G) / p.heads_per_item;
    hu[u] = group + u * G - tu[u] * p.heads_per_item;
  }
  pdl_wait();
  pdl_launch_dependents();
  const Heads<T> in(p.q, p.k, p.q_st, p.q_sh, p.k_st, p.k_sh, p.q_heads);
  const Heads<T> out(p.out_q, p.out_k, p.oq_st, p.oq_sh, p.ok_st, p.ok_sh, p.q_heads);
  Raw<T, C> x[U][S];
  auto here = [&](const Item& it, int u) { return tu[u] < it.nt && hu[u] < it.nh; };
  auto load = [&](const Item& it, int u) {
    if (!here(it, u)) return;
    const int32_t h = it.h0 + hu[u];
    load_row<T, C, L, S>(x[u], in.at(it.t0 + tu[u], h, h < p.q_heads), l);
  };
  int32_t i = blockIdx.x;
  Item it = item_of(p, i);
  uint64_t first = sh.first_position(p, it);
#pragma unroll
  for (int u = 0; u < U; ++u) load(it, u);
  sh.fill_once(p, l);
  __syncthreads();
  sh.fill(p, it, 0, first);
  Item next = it;
  if (i + gridDim.x < p.items) {
    next = item_of(p, i + gridDim.x);
    first = sh.first_position(p, next);
  }
  __syncthreads();
  const float inv_dim = 1.f / static_cast<float>(p.dim);
  for (int buf = 0; i < p.items; i += gridDim.x, buf ^= 1) {
    const bool more = i + gridDim.x < p.items;
    if (more) sh.fill(p, next, buf ^ 1, first);
    Item after = next;
    if (i + 2 * gridDim.x < p.items) {
      after = item_of(p, i + 2 * gridDim.x);
      first = sh.first_position(p, after);
    }
    const float* table = sh.table + buf * sh.table_size;
    const int32_t rows = it.nt * p.heads_per_item;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * G >= rows) break;
      float2 f[S][H];
      float2 sum2 = both(0.f);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        values<L::INTER>(x[u][s], s, l, f[s]);
#pragma unroll
        for (int j = 0; j < H; ++j) sum2 = fma2(f[s][j], f[s][j], sum2);
      }
      if (more) load(next, u);  // into the registers that were just read
      const float sum = row_sum<LPR>(sum2.x + sum2.y);
      const float rho = rsqrtf(fmaf(sum, inv_dim, p.eps));
      const int32_t h = it.h0 + hu[u];
      const bool is_q = h < p.q_heads, mine = here(it, u);
      T* dst = out.at(it.t0 + tu[u], h, is_q);
      const float2* w = sh.weights_of(is_q, lane);
      const float* tab = table + (mine ? tu[u] : 0) * 2 * sh.half;
#pragma unroll
      for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int j = 0; j < H; ++j) f[s][j] = mul2(mul2(f[s][j], both(rho)), w[sh.weight(s, j)]);
        if (l.turns(s)) turn<false>(f[s], tab + l.pair(s), tab + sh.half + l.pair(s));
        if (mine) store<L::INTER>(dst, s, l, f[s]);
      }
    }
    it = next;
    next = after;
    __syncthreads();  // the next table is whole, this one may be overwritten
  }
}

// Gradient: the sums of dw of a block end in its part of the workspace.
template <typename T, typename LaneT>
__global__ void __launch_bounds__(kThreads, (resident<LaneT::C, LaneT::S, true>()))
    norm_rotate_backward_kernel(const RotateParams p) {
  using L = LaneT;
  constexpr int C = L::C, LPR = L::LPR, S = L::S, H = L::kHalves, G = kThreads / LPR;
  constexpr int U = rows_ahead<T, C, S, true>();
  extern __shared__ __align__(16) uint8_t smem[];
  const int32_t lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const L l(p, lane);
  Shared<L> sh(p, smem);
  // rows of an item: row r is token r / heads_per_item, head r % heads_per_item
  int32_t tu[U], hu[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    tu[u] = (group + u * G) / p.heads_per_item;
    hu[u] = group + u * G - tu[u] * p.heads_per_item;
  }
  pdl_wait();
  pdl_launch_dependents();
  const Heads<T> in(p.q, p.k, p.q_st, p.q_sh, p.k_st, p.k_sh, p.q_heads);
  const Heads<T> din(p.d_q, p.d_k, p.dq_st, p.dq_sh, p.dk_st, p.dk_sh, p.q_heads);
  const Heads<T> out(p.out_q, p.out_k, p.oq_st, p.oq_sh, p.ok_st, p.ok_sh, p.q_heads);
  Raw<T, C> x[U][S], d[U][S];
  auto here = [&](const Item& it, int u) { return tu[u] < it.nt && hu[u] < it.nh; };
  auto load = [&](const Item& it, int u) {
    if (!here(it, u)) return;
    const int32_t h = it.h0 + hu[u];
    load_row<T, C, L, S>(x[u], in.at(it.t0 + tu[u], h, h < p.q_heads), l);
    load_row<T, C, L, S>(d[u], din.at(it.t0 + tu[u], h, h < p.q_heads), l);
  };
  float2 gq[S][H], gk[S][H];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < H; ++j) gq[s][j] = gk[s][j] = both(0.f);
  int32_t i = blockIdx.x;
  Item it = item_of(p, i);
  uint64_t first = sh.first_position(p, it);
#pragma unroll
  for (int u = 0; u < U; ++u) load(it, u);
  sh.fill_once(p, l);
  __syncthreads();
  sh.fill(p, it, 0, first);
  Item next = it;
  if (i + gridDim.x < p.items) {
    next = item_of(p, i + gridDim.x);
    first = sh.first_position(p, next);
  }
  __syncthreads();
  const float inv_dim = 1.f / static_cast<float>(p.dim);
  for (int buf = 0; i < p.items; i += gridDim.x, buf ^= 1) {
    const bool more = i + gridDim.x < p.items;
    if (more) sh.fill(p, next, buf ^ 1, first);
    Item after = next;
    if (i + 2 * gridDim.x < p.items) {
      after = item_of(p, i + 2 * gridDim.x);
      first = sh.first_position(p, after);
    }
    const float* table = sh.table + buf * sh.table_size;
    const int32_t rows = it.nt * p.heads_per_item;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * G >= rows) break;
      const bool mine = here(it, u);
      const int32_t h = it.h0 + hu[u];
      const bool is_q = h < p.q_heads;
      const float2* w = sh.weights_of(is_q, lane);
      const float* tab = table + (mine ? tu[u] : 0) * 2 * sh.half;
      float2 f[S][H], g[S][H];
      float2 sum2 = both(0.f), dot2 = both(0.f);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        values<L::INTER>(x[u][s], s, l, f[s]);
        values<L::INTER>(d[u][s], s, l, g[s]);
        if (l.turns(s)) turn<true>(g[s], tab + l.pair(s), tab + sh.half + l.pair(s));
#pragma unroll
        for (int j = 0; j < H; ++j) {
          sum2 = fma2(f[s][j], f[s][j], sum2);
          dot2 = fma2(mul2(g[s][j], w[sh.weight(s, j)]), f[s][j], dot2);
        }
      }
      if (more) load(next, u);
      const float sum = row_sum<LPR>(sum2.x + sum2.y), dot = row_sum<LPR>(dot2.x + dot2.y);
      if (mine) {
        const float rho = rsqrtf(fmaf(sum, inv_dim, p.eps));
        const float2 back = both(-rho * rho * rho * dot * inv_dim), rho2 = both(rho);
        T* dst = out.at(it.t0 + tu[u], h, is_q);
#pragma unroll
        for (int s = 0; s < S; ++s) {
#pragma unroll
          for (int j = 0; j < H; ++j) {
            const float2 gr = mul2(g[s][j], rho2);
            if (is_q) gq[s][j] = fma2(gr, f[s][j], gq[s][j]);
            else gk[s][j] = fma2(gr, f[s][j], gk[s][j]);
            g[s][j] = fma2(f[s][j], back, mul2(gr, w[sh.weight(s, j)]));
          }
          store<L::INTER>(dst, s, l, g[s]);
        }
      }
    }
    it = next;
    next = after;
    __syncthreads();
  }
  // sums of the rows of a warp, then of the block's warps, in a fixed order
  float* sums = reinterpret_cast<float*>(smem);  // [warps][2][dim]
  const int32_t warp = threadIdx.x / 32;
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int e = 0; e < 2 * C; ++e) {
      float vq = e & 1 ? gq[s][e / 2].y : gq[s][e / 2].x;
      float vk = e & 1 ? gk[s][e / 2].y : gk[s][e / 2].x;
#pragma unroll
      for (int k = LPR; k < 32; k <<= 1) {
        vq += __shfl_xor_sync(0xffffffffu, vq, k);
        vk += __shfl_xor_sync(0xffffffffu, vk, k);
      }
      const int32_t at = l.channel(s, e);
      if (at >= 0 && (threadIdx.x & 31) < LPR) {
        sums[(warp * 2 + 0) * p.dim + at] = vq;
        sums[(warp * 2 + 1) * p.dim + at] = vk;
      }
    }
  __syncthreads();
  for (int32_t c = threadIdx.x; c < 2 * p.dim; c += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w * 2 * p.dim + c];
    p.workspace[static_cast<int64_t>(blockIdx.x) * 2 * p.dim + c] = v;
  }
}

// dw_q and dw_k from the blocks' parts: 32 columns a block, 32 parts side by side.
__global__ void __launch_bounds__(1024) norm_rotate_sums_kernel(const RotateParams p,
                                                                int32_t parts) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int32_t x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int32_t col = blockIdx.x * 32 + x;
  float v = 0.f;
  if (col < 2 * p.dim) {
#pragma unroll 8
    for (int32_t i = y; i < parts; i += 32)
      v += p.workspace[static_cast<int64_t>(i) * 2 * p.dim + col];
  }
  s[y][x] = v;
  __syncthreads();
  v = s[x][y];  // column blockIdx.x * 32 + y
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int32_t c = blockIdx.x * 32 + y;
  if (x == 0 && c < 2 * p.dim) (c < p.dim ? p.dw_q : p.dw_k)[c < p.dim ? c : c - p.dim] = v;
}

// Blocks of the gradient at most: two an SM.
constexpr int32_t kBackBlocks = 2 * 152;

// Tokens of an item: of those that its rows' places hold, the number that leaves
// fewest of them empty (the largest such).
int32_t tokens_of(int32_t heads, int32_t groups, int32_t most) {
  int32_t best = 1;
  double used = 0.0;
  for (int32_t n = 1; n <= most; ++n) {
    const int32_t rounds = (n * heads + groups - 1) / groups;
    const double u = static_cast<double>(n * heads) / (rounds * groups);
    if (u >= used) best = n, used = u;
  }
  return best;
}

template <typename T, typename L, bool BACK>
cudaError_t launch(RotateParams p, int num_sms, cudaStream_t stream) {
  constexpr int C = L::C, S = L::S, G = kThreads / L::LPR;
  constexpr int kRows = G * rows_ahead<T, C, S, BACK>();  // of an item at most
  const int32_t heads = p.q_heads + p.k_heads, half = p.rotary / 2;
  const int32_t slots = resident<C, S, BACK>() * num_sms;  // blocks side by side
  // tokens of an item, no more than leave every place for a block an item
  int32_t most = kRows / heads;
  if (most > kMaxTable / half) most = kMaxTable / half;
  if (most > (p.tokens + slots - 1) / slots) most = (p.tokens + slots - 1) / slots;
  p.chunks_of_heads = 1;
  p.heads_per_item = heads;
  p.tokens_per_item = most >= 1 ? tokens_of(heads, G, most) : 1;
  if (heads > kRows || p.tokens < num_sms) {
    // one token's heads in equal chunks: as few as hold them, or, where tokens are
    // few, of one row a group
    const int32_t rows = heads > kRows && p.tokens >= num_sms ? kRows : G;
    p.tokens_per_item = 1;
    p.chunks_of_heads = (heads + rows - 1) / rows;
    p.heads_per_item = (heads + p.chunks_of_heads - 1) / p.chunks_of_heads;
  }
  p.items = (p.tokens + p.tokens_per_item - 1) / p.tokens_per_item * p.chunks_of_heads;
  const int32_t blocks = p.items < slots ? p.items : slots;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = Shared<L>::bytes(p);
  if constexpr (!BACK) {
    return cudaLaunchKernelEx(&cfg, norm_rotate_kernel<T, L>, p);
  } else {
    if (blocks > kBackBlocks) cfg.gridDim = dim3(kBackBlocks);
    const int32_t parts = static_cast<int32_t>(cfg.gridDim.x);
    const size_t sums = sizeof(float) * kWarps * 2 * p.dim;
    if (cfg.dynamicSmemBytes < sums) cfg.dynamicSmemBytes = sums;
    const cudaError_t err =
        cudaLaunchKernelEx(&cfg, norm_rotate_backward_kernel<T, L>, p);
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3((2 * p.dim + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, norm_rotate_sums_kernel, p, parts);
  }
}

// Whole and full rows have forms of their own.
template <typename T, int LPR, int S, bool INTER, bool BACK>
cudaError_t full(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return p.rotary == p.dim ? launch<T, Lane<4, LPR, S, INTER, kWhole>, BACK>(p, num_sms, stream)
                           : launch<T, Lane<4, LPR, S, INTER, kFull>, BACK>(p, num_sms, stream);
}
template <typename T, int LPR, int S, bool INTER, bool BACK>
cudaError_t chunked(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return p.dim == 8 * LPR * S ? full<T, LPR, S, INTER, BACK>(p, num_sms, stream)
                              : launch<T, Lane<4, LPR, S, INTER, kAny>, BACK>(p, num_sms, stream);
}

// Chunks of four channels where every array allows them, else single ones.  A lane
// holds two slots forward (what a row costs beside its values is shared by more of
// them), one in the gradient, which holds five values a channel; more where a
// row has more slots than that in a warp.
template <typename T, bool INTER, bool BACK>
cudaError_t by_shape(const RotateParams& p, int num_sms, cudaStream_t stream) {
  const int n = p.chunks ? p.dim / 8 : (p.dim + 1) / 2;
  if (p.chunks) {
    if (n > 32) return chunked<T, 32, 2, INTER, BACK>(p, num_sms, stream);
    constexpr int S = BACK ? 1 : 2;
    if constexpr (!BACK) {
      // heads of 96 and 192 channels fill lanes of three slots (16384 tokens x 40 heads
      // of 96: 61 -> 48 us)
      if (n == 12) return full<T, 4, 3, INTER, BACK>(p, num_sms, stream);
      if (n == 24) return full<T, 8, 3, INTER, BACK>(p, num_sms, stream);
    }
    if (n > 16) return chunked<T, 32 / S, S, INTER, BACK>(p, num_sms, stream);
    if (n > 8) return chunked<T, 16 / S, S, INTER, BACK>(p, num_sms, stream);
    return chunked<T, 8 / S, S, INTER, BACK>(p, num_sms, stream);
  }
  if (n <= 8) return launch<T, Lane<1, 8, 1, INTER, kAny>, BACK>(p, num_sms, stream);
  if (n <= 16) return launch<T, Lane<1, 16, 1, INTER, kAny>, BACK>(p, num_sms, stream);
  if (n <= 32) return launch<T, Lane<1, 32, 1, INTER, kAny>, BACK>(p, num_sms, stream);
  if (n <= 64) return launch<T, Lane<1, 32, 2, INTER, kAny>, BACK>(p, num_sms, stream);
  if (n <= 128) return launch<T, Lane<1, 32, 4, INTER, kAny>, BACK>(p, num_sms, stream);
  return launch<T, Lane<1, 32, 8, INTER, kAny>, BACK>(p, num_sms, stream);
}

template <typename T, bool BACK>
cudaError_t by_layout(const RotateParams& p, int num_sms, cudaStream_t stream) {
  return p.interleaved ? by_shape<T, true, BACK>(p, num_sms, stream)
                       : by_shape<T, false, BACK>(p, num_sms, stream);
}

}  // namespace
}  // namespace mx
