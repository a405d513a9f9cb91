// route.cu -- the experts of every token from the router's logits, what the
// grouped products need of them, the balance loss, and its and the weights'
// gradient.  For z = logits [tokens, experts]:
//
//   p = softmax(z);  the top_k largest z win (equal ones: the lowest index first);
//   w = p of the winners, divided by their sum when renormalized
//   counts_e = how many of the n tokens that count chose e
//   balance  = experts sum_e counts_e / (n top_k) sum_t p_te / n
//   offsets, order: the (token, place) pairs sorted by expert, in order of tokens
//   dz = p (g - sum p g + d_lse),  g = d_balance experts counts / (n^2 top_k) + d p of the
//   winners,  lse = log sum exp z
//
// Two kernels.  The first finds the winners and counts them per block: of few tokens
// each has a warp, which holds its logits in registers and takes the winners one
// after the other (a maximum over the warp, then the lowest lane and place that hold
// it); of many each has a lane (route_tile_kernel).  The second gives every pair its
// place: a block adds up the counts of the blocks before it, and the tokens before the
// pair's own with the same expert, as bits of words (Pairs); one block more writes what
// is left, the sums over all blocks.  Counts are integers and the sums of p run in a
// fixed order, so the same inputs give the same bits.  Up to kOneBlock tokens, one block
// does all of it in one launch.  The gradient is one kernel, with a group of lanes a token.
//
// 65536 tokens over 64 experts, top 8, FP32 (one GB300; 42 MB in all, 6.2 us of copy
// bandwidth): 16.6 us forward, most of it the first kernel, whose loads come before its
// instructions (14 warps an SM, one round; two lanes a token and 28 warps: 21.6 against
// 20.8), then the second's chain of latencies (with lanes matched by expert and two
// blocks an SM in both kernels 27; 1048576 tokens 179); 10.6 us the gradient, bound by
// instructions.  One token: 4.4 us in a graph, 6.6 called.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "pairs.cuh"
#include "ptx.cuh"
#include "softmax.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kOrderThreads = 1024;  // of the second kernel at most
constexpr int kBackThreads = 256;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kMaxBlocks = 304;
// of route_tile_kernel: one an SM, less one for the second kernel's last block (68096
// tokens, 152 blocks and one more: 22.1 us against 18.2)
constexpr int kTileBlocks = 151;
constexpr int kMasks = 4096;      // words of 32 tokens' choices
constexpr int kOneBlock = 64;
// Tokens from which on (also 128 an expert), and experts and winners up to which, a token
// is a lane's.  (A token a lane against a token a warp, top 8, both kernels: 64 experts
// 4096 tokens 13.7 and 12.1 us, 8192 13.3 and 15.4, 32768 15.6 and 35.2; 128 experts 8192
// 18.3 and 16.9, 16384 18.1 and 22.4.)
constexpr int kTileTokens = 8192;
constexpr int kTileExperts = 128;
constexpr int kTileTopK = 8;
constexpr int kTileWarps = 27;  // of its blocks at most (64 experts: as shared memory holds)
constexpr int kTileBytes = 222 * 1024;  // shared memory of a block's rows at most

// Unsigned keys in the order of the logits: NaN below everything, 0 taken.
__device__ __forceinline__ uint32_t key_of(float z) {
  if (z != z) return 1u;
  const uint32_t b = __float_as_uint(z + 0.f);  // (-0 equals 0)
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }

// V consecutive logits from column c on; NaN-free padding is the caller's.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int32_t c, int32_t n, bool vec,
                                            float (&z)[V]) {
  if (V > 1 && vec) {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      if (c + v >= n) continue;
      if constexpr (V == 2 && sizeof(T) == 4) {
        const float2 q = *reinterpret_cast<const float2*>(row + c);
        z[0] = q.x, z[1] = q.y;
      } else if constexpr (V == 2) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(row + c);
        z[0] = __uint_as_float(q << 16), z[1] = __uint_as_float(q & 0xFFFF0000u);
      } else if constexpr (V < 2) {
      } else if constexpr (sizeof(T) == 4) {
        const float4 q = *reinterpret_cast<const float4*>(row + c + v);
        z[v] = q.x, z[v + 1] = q.y, z[v + 2] = q.z, z[v + 3] = q.w;
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(row + c + v);
        z[v] = __uint_as_float(q.x << 16), z[v + 1] = __uint_as_float(q.x & 0xFFFF0000u);
        z[v + 2] = __uint_as_float(q.y << 16), z[v + 3] = __uint_as_float(q.y & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c + v < n) z[v] = to_float(row[c + v]);
  }
}

// exp(x) for x <= 0, the distance of a logit from its row's largest (or lse): 2^-22
// of the result and, from rounding the argument, |x| 2^-24.
__device__ __forceinline__ float exp_below(float x) { return exp2_fast(x * kLog2e); }

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Counts of a block in the workspace, rows of whole 16 bytes: pairs, pairs that
// count, sums of p; and the tokens that count.
struct Parts {
  int32_t row;       // experts, rounded up to four
  int32_t* pairs;    // [blocks][row]
  int32_t* counted;  // [blocks][row]
  float* p;          // [blocks][row]
  int32_t* tokens;   // [blocks]
  __device__ __forceinline__ Parts(const RouteParams& r) {
    row = (r.experts + 3) & ~3;
    pairs = r.workspace;
    counted = pairs + r.blocks * row;
    p = reinterpret_cast<float*>(counted + r.blocks * row);
    tokens = reinterpret_cast<int32_t*>(p + r.blocks * row);
  }
};

struct RouteShared {
  int32_t pairs[kMaxExperts];
  int32_t counted[kMaxExperts];
  int32_t base[kMaxExperts];
  int32_t tokens;
  float sums[32];
  union {
    int2 win[kWarps][kMaxTopK];            // winners of the tokens under way: expert, key
    float p[kWarps][kMaxExperts];
    struct {
      uint32_t mask[kMasks];               // [32 tokens][expert]: which of them chose it
      int32_t before[kMasks];              // its first place for these
    };
    int4 part[2][kOrderThreads];           // a thread's sums over blocks
  };
};

// Exclusive sums over the experts of `total`, added to s.base and, with their
// total, in `offsets`.
__device__ __forceinline__ void scan_experts(RouteShared& s, int32_t experts, const int32_t* total,
                                             int32_t* offsets) {
  // one warp, 16 experts a lane at most
  if (warp_id() == 0) {
    const int32_t per = (experts + 31) / 32, lo = lane_id() * per;
    int32_t sum = 0;
    for (int32_t i = 0; i < per; ++i)
      if (lo + i < experts) sum += total[lo + i];
    int32_t before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, before, d);
      if (lane_id() >= static_cast<uint32_t>(d)) before += v;
    }
    before -= sum;
    for (int32_t i = 0; i < per; ++i)
      if (lo + i < experts) {
        s.base[lo + i] += before;
        if (offsets) offsets[lo + i] = before;
        before += total[lo + i];
      }
    if (offsets && lane_id() == 31) offsets[experts] = before;
  }
  __syncthreads();
}

// Places of the pairs of tokens [t0, t1), some tokens at a time.  Of each 32 of these and
// expert a word tells which of the tokens chose it: a pair's place is what the words
// before its own hold, and the bits before its own.  Marking the words needs nothing of
// the counts, placing needs s.base, each expert's first place.
struct Pairs {
  static constexpr int kKept = 4;  // pairs of a thread that stay in registers
  const RouteParams& r;
  RouteShared& s;
  int32_t t0, t1, most, words, n, threads;
  uint32_t inverse;     // of top_k, in units of 2^-32 (exact below 2^27 pairs)
  int32_t kept[kKept];  // token * 512 + expert, or -1
  __device__ __forceinline__ Pairs(const RouteParams& r_, RouteShared& s_, int32_t a, int32_t b)
      : r(r_), s(s_), t0(a), t1(b), most(kMasks / r_.experts * 32), threads(blockDim.x),
        inverse(0xFFFFFFFFu / static_cast<uint32_t>(r_.top_k) + 1u) {}
  __device__ __forceinline__ int32_t packed(int32_t i) const {
    const int32_t t = r.top_k == 1 ? i : static_cast<int32_t>(__umulhi(i, inverse));
    return t * kMaxExperts + r.ids[t0 * r.top_k + i];
  }
  __device__ __forceinline__ int32_t word(int32_t pair) const {
    return pair / (32 * kMaxExperts) * r.experts + pair % kMaxExperts;
  }
  __device__ __forceinline__ static uint32_t bit(int32_t pair) {
    return 1u << (pair / kMaxExperts % 32);
  }
  // Clears the words; their marking is a barrier away.
  __device__ __forceinline__ void clear() {
    const int32_t tokens = min(most, t1 - t0);
    n = tokens * r.top_k;
    words = (tokens + 31) / 32;
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
      const int32_t i = int32_t(threadIdx.x) + k * threads;
      kept[k] = i < n ? packed(i) : -1;
    }
    for (int32_t i = threadIdx.x; i < words * r.experts; i += threads) s.mask[i] = 0u;
  }
  __device__ __forceinline__ void mark() {
#pragma unroll
    for (int k = 0; k < kKept; ++k)
      if (kept[k] >= 0) atomicOr(&s.mask[word(kept[k])], bit(kept[k]));
    for (int32_t i = int32_t(threadIdx.x) + kKept * threads; i < n; i += threads) {
      const int32_t pair = packed(i);
      atomicOr(&s.mask[word(pair)], bit(pair));
    }
  }
  __device__ __forceinline__ void place_one(int32_t i, int32_t pair) const {
    const int32_t at = word(pair);
    r.order[s.before[at] + __popc(s.mask[at] & (bit(pair) - 1u))] = t0 * r.top_k + i;
  }
  // After a barrier behind the marks and s.base.
  __device__ __forceinline__ void place() {
    while (true) {
      for (int32_t e = threadIdx.x; e < r.experts; e += threads) {
        int32_t at = s.base[e];
#pragma unroll 8
        for (int32_t w = 0; w < words; ++w) {
          s.before[w * r.experts + e] = at;
          at += __popc(s.mask[w * r.experts + e]);
        }
        s.base[e] = at;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kKept; ++k)
        if (kept[k] >= 0) place_one(int32_t(threadIdx.x) + k * threads, kept[k]);
      for (int32_t i = int32_t(threadIdx.x) + kKept * threads; i < n; i += threads)
        place_one(i, packed(i));
      if (t1 - t0 <= most) return;
      t0 += most;
      __syncthreads();
      clear();
      __syncthreads();
      mark();
      __syncthreads();
    }
  }
};

// The balance loss from each thread's share of sum counts_e sum p_te.
__device__ __forceinline__ void write_balance(const RouteParams& r, RouteShared& s, float share,
                                              int32_t tokens) {
  share = group_sum<32>(share);
  if (lane_id() == 0) s.sums[warp_id()] = share;
  __syncthreads();
  if (threadIdx.x == 0) {
    float all = 0.f;
    for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) all += s.sums[w];
    const float n = static_cast<float>(tokens);
    *r.balance = tokens ? all / n / n * (static_cast<float>(r.experts) / static_cast<float>(r.top_k))
                        : 0.f;
  }
}

template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteParams r) {
  __shared__ RouteShared s;
  const int32_t warp = warp_id();
  const int32_t lane = lane_id();
  for (int32_t e = threadIdx.x; e < r.experts; e += kThreads) s.pairs[e] = s.counted[e] = 0;
  if (threadIdx.x == 0) s.tokens = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int32_t t0 = blockIdx.x * r.tokens_per_block;
  const int32_t t1 = min(r.tokens, t0 + r.tokens_per_block);
  const int32_t c0 = lane * V;
  float acc[V], z[V], ahead[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = z[v] = ahead[v] = 0.f;
  int2* win = s.win[warp];
  const T* logits = static_cast<const T*>(r.logits);
  int32_t t = t0 + warp;
  if (t < t1) load_logits<T, V>(logits + t * r.ld, c0, r.experts, r.vec, z);
  for (; t < t1; t += kWarps) {
    const bool valid = !r.mask || r.mask[t] != 0;
    if (t + kWarps < t1)
      load_logits<T, V>(logits + (t + kWarps) * r.ld, c0, r.experts, r.vec, ahead);
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = c0 + v < r.experts ? key_of(z[v]) : 0u;
    float top = 0.f;
    for (int32_t j = 0; j < r.top_k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = max(best, key[v]);
      const uint32_t most = __reduce_max_sync(0xffffffffu, best);
      const uint32_t who = __ballot_sync(0xffffffffu, best == most);
      if (j == 0) top = logit_of(most);
      if (lane == __ffs(who) - 1) {
        int32_t at = 0;
        bool found = false;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (!found && key[v] == most) found = true, at = v, key[v] = 0u;
        win[j] = make_int2(c0 + at, static_cast<int32_t>(most));
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[v] = c0 + v < r.experts ? exp_below(z[v] - top) : 0.f;
      sum += z[v];
    }
    sum = group_sum<32>(sum);
    const float inv = 1.f / sum;
    if (valid) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(z[v], inv, acc[v]);
      if (lane == 0) atomicAdd(&s.tokens, 1);
    }
    __syncwarp();
    // the winners side by side
    float picked = 0.f;
    for (int32_t j = lane; j < r.top_k; j += 32) {
      const int2 w = win[j];
      const float e = exp_below(logit_of(static_cast<uint32_t>(w.y)) - top);
      picked += e;
      r.ids[t * r.top_k + j] = w.x;
      atomicAdd(&s.pairs[w.x], 1);
      if (valid) atomicAdd(&s.counted[w.x], 1);
      if (!r.renormalize) r.weights[t * r.top_k + j] = e * inv;
      win[j].y = __float_as_int(e);
    }
    if (r.renormalize) {
      // p / sum of p, so that a softmax that is NaN stays so
      picked = group_sum<32>(picked);
      const float scale = inv / (picked * inv);
      for (int32_t j = lane; j < r.top_k; j += 32)
        r.weights[t * r.top_k + j] = __int_as_float(win[j].y) * scale;
    }
    if (lane == 0) r.lse[t] = top + logf(sum);
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = ahead[v];
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (c0 + v < r.experts) s.p[warp][c0 + v] = acc[v];
  __syncthreads();
  const Parts parts(r);
  float share = 0.f;
  for (int32_t e = threadIdx.x; e < (ONE ? r.experts : parts.row); e += kThreads) {
    float a = 0.f;
    if (e < r.experts) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += s.p[w][e];
    }
    if constexpr (ONE) {
      r.counts[e] = s.counted[e];
      share += a * static_cast<float>(s.counted[e]);
      s.base[e] = 0;
    } else {
      const int32_t at = blockIdx.x * parts.row + e;
      parts.pairs[at] = e < r.experts ? s.pairs[e] : 0;
      parts.counted[at] = e < r.experts ? s.counted[e] : 0;
      parts.p[at] = a;
    }
  }
  if constexpr (ONE) {
    write_balance(r, s, share, s.tokens);
    scan_experts(s, r.experts, s.pairs, r.offsets);
    if (t0 >= t1) return;  // (no token)
    Pairs pairs(r, s, t0, t1);
    pairs.clear();
    __syncthreads();
    pairs.mark();
    __syncthreads();
    pairs.place();
  } else {
    if (threadIdx.x == 0) parts.tokens[blockIdx.x] = s.tokens;
  }
}

// The first kernel for many tokens: a warp takes 32 of them at a time, a token a
// lane.  The logits come to shared memory in rows of an odd length.  Every lane
// keeps the largest of each eight of its row in registers; a winner is the largest
// of those, looked up among its eight, which then give their next largest (a NaN
// in its place: the maximum passes over it).  The exponentials take the logits'
// places, and the sums of p go down the columns, an expert a lane.
template <typename T, int EIGHTS>
__global__ void __launch_bounds__(kTileWarps * 32) route_tile_kernel(const RouteParams r) {
  extern __shared__ float tiles[];
  __shared__ int32_t pairs[kTileExperts], counted[kTileExperts], tokens;
  __shared__ __align__(16) float factor[kTileWarps][32];
  const int32_t warp = warp_id(), lane = lane_id(), warps = blockDim.x / 32;
  const int32_t row_size = (r.experts + 7) / 8 * 8 + 1;
  float* tile = tiles + warp * 32 * row_size;
  for (int32_t e = threadIdx.x; e < r.experts; e += blockDim.x) pairs[e] = counted[e] = 0;
  if (threadIdx.x == 0) tokens = 0;
  float* mine = tile + lane * row_size;
  for (int32_t e = r.experts; e < row_size; ++e) mine[e] = NAN;  // (no expert: never chosen)
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int32_t end = min(r.tokens, (static_cast<int32_t>(blockIdx.x) + 1) * r.tokens_per_block);
  float acc[EIGHTS / 4];
#pragma unroll
  for (int i = 0; i < EIGHTS / 4; ++i) acc[i] = 0.f;
  const T* logits = static_cast<const T*>(r.logits);
  // lanes of a row's four-logit runs, a power of two
  const int32_t shift = r.experts <= 32 ? 3 : r.experts <= 64 ? 4 : 5;
  for (int32_t t0 = blockIdx.x * r.tokens_per_block + warp * 32; t0 < end; t0 += warps * 32) {
    const int32_t rows = min(32, end - t0);
    if (r.vec) {
      const int32_t c = (lane & ((1 << shift) - 1)) * 4, step = 32 >> shift;
      if (c < r.experts) {
#pragma unroll 8
        for (int32_t row = lane >> shift; row < rows; row += step) {
          float z[4];
          load_logits<T, 4>(logits + (t0 + row) * r.ld, c, r.experts, true, z);
#pragma unroll
          for (int v = 0; v < 4; ++v) tile[row * row_size + c + v] = z[v];
        }
      }
    } else {
      for (int32_t row = 0; row < rows; ++row)
        for (int32_t c = lane; c < r.experts; c += 32)
          tile[row * row_size + c] = to_float(logits[(t0 + row) * r.ld + c]);
    }
    __syncwarp();
    const int32_t t = t0 + lane;
    bool valid = false;
    if (lane < rows) {
      valid = !r.mask || r.mask[t] != 0;
      float most[EIGHTS];
#pragma unroll
      for (int g = 0; g < EIGHTS; ++g) {
        most[g] = NAN;
        if (g * 8 < r.experts) {
#pragma unroll
          for (int i = 0; i < 8; ++i) most[g] = fmaxf(most[g], mine[g * 8 + i]);
        }
      }
      float w[kTileTopK];
      int32_t id[kTileTopK];
#pragma unroll
      for (int j = 0; j < kTileTopK; ++j) {
        w[j] = 0.f;
        id[j] = 0;
        if (j >= r.top_k) continue;
        float best = most[0];
#pragma unroll
        for (int g = 1; g < EIGHTS; ++g) best = fmaxf(best, most[g]);
        if (best == best) {
          int32_t at = 0;
#pragma unroll
          for (int g = EIGHTS - 1; g >= 0; --g) at = most[g] == best ? g : at;
          float* eight = mine + at * 8;
          float v[8], next = NAN;
          int32_t place = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = eight[i];
#pragma unroll
          for (int i = 7; i >= 0; --i) place = v[i] == best ? i : place;
#pragma unroll
          for (int i = 0; i < 8; ++i) next = i == place ? next : fmaxf(next, v[i]);
#pragma unroll
          for (int g = 0; g < EIGHTS; ++g) most[g] = g == at ? next : most[g];
          w[j] = eight[place];
          eight[place] = NAN;
          id[j] = at * 8 + place;
        } else {
          // nothing but NaN is left: the lowest expert that was not taken
          int32_t e = 0;
          for (bool taken = true; taken; e += taken) {
            taken = false;
#pragma unroll
            for (int i = 0; i < j; ++i) taken = taken || id[i] == e;
          }
          w[j] = NAN;
          id[j] = e;
        }
      }
      const float top = w[0];
#pragma unroll
      for (int j = 0; j < kTileTopK; ++j)
        if (j < r.top_k) mine[id[j]] = w[j];
      // exponentials two at a time, as exp_below has them
      float2 s2[2] = {both(0.f), both(0.f)};
      const int32_t whole = r.experts & ~3;
#pragma unroll 4
      for (int32_t e = 0; e < whole; e += 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 p = make_float2(mine[e + 2 * i], mine[e + 2 * i + 1]);
          p = mul2(add2(p, both(-top)), both(kLog2e));
          p = make_float2(exp2_fast(p.x), exp2_fast(p.y));
          mine[e + 2 * i] = p.x;
          mine[e + 2 * i + 1] = p.y;
          s2[i] = add2(s2[i], p);
        }
      }
      float sum = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
      for (int32_t e = whole; e < r.experts; ++e) sum += mine[e] = exp_below(mine[e] - top);
      const float inv = 1.f / sum;
      r.lse[t] = top + logf(sum);
      float picked = 0.f;
#pragma unroll
      for (int j = 0; j < kTileTopK; ++j)
        if (j < r.top_k) {
          w[j] = mine[id[j]];
          picked += w[j];
          atomicAdd(&pairs[id[j]], 1);
          if (valid) atomicAdd(&counted[id[j]], 1);
        }
      // p / sum of p, so that a softmax that is NaN stays so
      const float scale = r.renormalize ? inv / (picked * inv) : inv;
      const int64_t at = static_cast<int64_t>(t) * r.top_k;
      // eight winners, the most and the usual number, by 16 bytes (65536 tokens over 64
      // experts 16.6 us, one by one 18.2; 262144 47.6 and 52.0; 8192 11.0 and 11.7)
      if (r.top_k == 8 && r.vec_ids) {
        int4* ids = reinterpret_cast<int4*>(r.ids + at);
        float4* ws = reinterpret_cast<float4*>(r.weights + at);
        ids[0] = make_int4(id[0], id[1], id[2], id[3]);
        ids[1] = make_int4(id[4], id[5], id[6], id[7]);
        ws[0] = make_float4(w[0] * scale, w[1] * scale, w[2] * scale, w[3] * scale);
        ws[1] = make_float4(w[4] * scale, w[5] * scale, w[6] * scale, w[7] * scale);
      } else {
#pragma unroll
        for (int j = 0; j < kTileTopK; ++j)
          if (j < r.top_k) {
            r.ids[at + j] = id[j];
            r.weights[at + j] = w[j] * scale;
          }
      }
      factor[warp][lane] = inv;
    }
    const uint32_t count = __ballot_sync(0xffffffffu, valid);
    if (lane == 0) atomicAdd(&tokens, __popc(count));
    __syncwarp();
    auto add = [&](int32_t row, float f) {
#pragma unroll
      for (int i = 0; i < EIGHTS / 4; ++i)
        if (i * 32 + lane < r.experts)
          acc[i] = fmaf(tile[row * row_size + i * 32 + lane], f, acc[i]);
    };
    if (count == 0xffffffffu) {  // (65536 tokens 17.8 -> 16.9 us, with the pairs above)
      for (int32_t row = 0; row < 32; row += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&factor[warp][row]);
        add(row, f.x), add(row + 1, f.y), add(row + 2, f.z), add(row + 3, f.w);
      }
    } else {
      for (uint32_t left = count; left; left &= left - 1) {
        const int32_t row = __ffs(left) - 1;
        add(row, factor[warp][row]);
      }
    }
    __syncwarp();
  }
  // sums of p, warp by warp
#pragma unroll
  for (int i = 0; i < EIGHTS / 4; ++i)
    if (i * 32 + lane < r.experts) tile[i * 32 + lane] = acc[i];
  __syncthreads();
  const Parts parts(r);
  for (int32_t e = threadIdx.x; e < parts.row; e += blockDim.x) {
    float a = 0.f;
    if (e < r.experts)
      for (int32_t w = 0; w < warps; ++w)
        a += tiles[w * 32 * row_size + e];
    const int32_t at = blockIdx.x * parts.row + e;
    parts.pairs[at] = e < r.experts ? pairs[e] : 0;
    parts.counted[at] = e < r.experts ? counted[e] : 0;
    parts.p[at] = a;
  }
  if (threadIdx.x == 0) parts.tokens[blockIdx.x] = tokens;
}

__device__ __forceinline__ void add4(int4& a, const int4& b) {
  a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
}

// Places of the pairs of r.group blocks of the first kernel; the last block: counts,
// offsets and the balance loss.  One block an SM (registers for no more): of blocks that
// start before the first kernel has ended two would share an SM beside empty ones (65536
// tokens 17.8 us, with two an SM 20.5; 8192 over 256 experts, 256 blocks of the first
// kernel, 25.3 in pairs, 31.7 one by one).
__global__ void __launch_bounds__(kOrderThreads, 1) route_order_kernel(const RouteParams r) {
  __shared__ RouteShared s;
  pdl_wait();
  pdl_launch_dependents();
  const Parts parts(r);
  const bool last = blockIdx.x == gridDim.x - 1;
  const int32_t threads = blockDim.x, part0 = blockIdx.x * r.group;
  // four experts a thread, the blocks' rows dealt out to as many threads as there
  // are for each
  const int32_t quads = parts.row / 4, slices = threads / quads;
  const int32_t quad = threadIdx.x % quads, slice = threadIdx.x / quads;
  for (int32_t e = threadIdx.x; e < parts.row; e += threads) s.pairs[e] = s.base[e] = 0;
  const int32_t t0 = part0 * r.tokens_per_block;
  Pairs pairs(r, s, t0, min(r.tokens, t0 + r.group * r.tokens_per_block));
  if (!last) pairs.clear();
  __syncthreads();
  if (!last) pairs.mark();
  if (slice < slices) {
    int4 all = make_int4(0, 0, 0, 0), before = all;
#pragma unroll 8
    for (int32_t b = slice; b < r.blocks; b += slices) {
      const int4 c = *reinterpret_cast<const int4*>(parts.pairs + b * parts.row + quad * 4);
      add4(all, c);
      if (b < part0) add4(before, c);
    }
    const int32_t sums[4] = {all.x, all.y, all.z, all.w};
    const int32_t bases[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      atomicAdd(&s.pairs[quad * 4 + i], sums[i]);
      if (!last) atomicAdd(&s.base[quad * 4 + i], bases[i]);
    }
  }
  __syncthreads();
  scan_experts(s, r.experts, s.pairs, last ? r.offsets : nullptr);
  if (!last) {
    pairs.place();
    return;
  }
  int32_t n = 0;
  for (int32_t b = threadIdx.x; b < r.blocks; b += threads) n += parts.tokens[b];
  if (threadIdx.x == 0) s.tokens = 0;
  int4 counted = make_int4(0, 0, 0, 0);
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
  if (slice < slices) {
#pragma unroll 4
    for (int32_t b = slice; b < r.blocks; b += slices) {
      const int32_t at = b * parts.row + quad * 4;
      add4(counted, *reinterpret_cast<const int4*>(parts.counted + at));
      const float4 q = *reinterpret_cast<const float4*>(parts.p + at);
      p.x += q.x, p.y += q.y, p.z += q.z, p.w += q.w;
    }
    s.part[0][slice * quads + quad] = counted;
    reinterpret_cast<float4*>(s.part[1])[slice * quads + quad] = p;
  }
  __syncthreads();
  atomicAdd(&s.tokens, n);
  float share = 0.f;
  for (int32_t e = threadIdx.x; e < r.experts; e += threads) {
    int32_t c = 0;
    float a = 0.f;
    for (int32_t i = 0; i < slices; ++i) {
      c += reinterpret_cast<const int32_t*>(s.part[0])[i * parts.row + e];
      a += reinterpret_cast<const float*>(s.part[1])[i * parts.row + e];
    }
    r.counts[e] = c;
    share += a * static_cast<float>(c);
  }
  __syncthreads();
  write_balance(r, s, share, s.tokens);
}

template <typename T, int L, int V>
__global__ void __launch_bounds__(kBackThreads) route_backward_kernel(const RouteParams r) {
  constexpr int kGroups = 32 / L;
  constexpr int kWarps = kBackThreads / 32;
  __shared__ float coef[kMaxExperts];
  // the weights' share by expert, of the tokens that a warp has under way
  __shared__ __align__(16) float scatter[kWarps][kGroups][L * V];
  __shared__ int32_t s_pairs;
  const int32_t lane = lane_id() % L, group = lane_id() / L;
  if (threadIdx.x == 0) s_pairs = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  // d balance / d p_te = experts counts_e / (n^2 top_k), n = sum of counts / top_k
  int32_t counted = 0;
  for (int32_t e = threadIdx.x; e < r.experts; e += kBackThreads) counted += r.counts_in[e];
  atomicAdd(&s_pairs, counted);
  __syncthreads();
  const float n = static_cast<float>(s_pairs / r.top_k);
  const float scale = r.d_balance && s_pairs
                          ? *r.d_balance * (static_cast<float>(r.experts) / (n * n * r.top_k))
                          : 0.f;
  for (int32_t e = threadIdx.x; e < r.experts; e += kBackThreads)
    coef[e] = scale * static_cast<float>(r.counts_in[e]);
  __syncthreads();
  const int32_t c0 = lane * V;
  float c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = c0 + v < r.experts ? coef[c0 + v] : 0.f;
  constexpr int kPer = kMaxTopK / L;  // winners of a lane
  float* mine = scatter[warp_id()][group];
  float add[V];
#pragma unroll
  for (int v = 0; v < V; ++v) mine[c0 + v] = add[v] = 0.f;
  __syncwarp();
  // a token's loads, asked for one round ahead
  struct Token {
    float z[V], lse, w[kPer], g[kPer];
    int32_t id[kPer];
    bool here, valid;
  };
  auto load = [&](Token& k, int32_t t) {
    k.here = t < r.tokens;
    k.valid = false;
    k.lse = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) k.z[v] = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) k.id[i] = -1;
    if (!k.here) return;
    load_logits<T, V>(static_cast<const T*>(r.logits) + t * r.ld, c0, r.experts, r.vec, k.z);
    k.lse = r.lse_in[t];
    k.valid = !r.mask || r.mask[t] != 0;
    if (!r.d_weights) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int32_t j = lane + i * L, at = t * r.top_k + j;
      if (j >= r.top_k) continue;
      const int32_t id = r.ids_in[at];
      k.id[i] = static_cast<uint32_t>(id) < static_cast<uint32_t>(r.experts) ? id : -1;
      k.w[i] = r.w_in[at];
      k.g[i] = r.d_weights[at];
    }
  };
  const int32_t step = gridDim.x * kWarps * kGroups;
  int32_t base = (blockIdx.x * kWarps + warp_id()) * kGroups;
  Token ahead;
  load(ahead, base + group);
  for (; base < r.tokens; base += step) {
    const int32_t t = base + group;
    const Token k = ahead;
    if (base + step < r.tokens) load(ahead, t + step);
    const bool here = k.here, valid = k.valid;
    float z[V];
    float dot = 0.f;
    if (r.d_weights) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (k.id[i] >= 0) dot = fmaf(k.w[i], k.g[i], dot);
      dot = group_sum<L>(dot);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (k.id[i] >= 0) mine[k.id[i]] = k.w[i] * (k.g[i] - (r.renormalize ? dot : 0.f));
      __syncwarp();
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const float4 q = *reinterpret_cast<const float4*>(mine + c0 + v);
        add[v] = q.x, add[v + 1] = q.y, add[v + 2] = q.z, add[v + 3] = q.w;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (k.id[i] >= 0) mine[k.id[i]] = 0.f;
      __syncwarp();
    }
    float inner = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[v] = c0 + v < r.experts ? exp_below(k.z[v] - k.lse) : 0.f;
      if (valid) inner = fmaf(z[v], c[v], inner);
    }
    inner = group_sum<L>(inner);
    if (!r.renormalize) inner += dot;
    if (here && r.d_lse) inner -= r.d_lse[t];
    if (!here) continue;
    T* out = static_cast<T*>(r.d_logits) + static_cast<int64_t>(t) * r.experts;
#pragma unroll
    for (int v = 0; v < V; ++v)
      z[v] = fmaf(z[v], (valid ? c[v] : 0.f) - inner, add[v]);
    if (r.vec_out) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        if (c0 + v >= r.experts) continue;
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(out + c0 + v) =
              make_float4(z[v], z[v + 1], z[v + 2], z[v + 3]);
        else
          *reinterpret_cast<uint2*>(out + c0 + v) =
              make_uint2(pack_bf16x2(z[v], z[v + 1]), pack_bf16x2(z[v + 2], z[v + 3]));
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (c0 + v >= r.experts) continue;
        if constexpr (sizeof(T) == 4) out[c0 + v] = z[v];
        else out[c0 + v] = __float2bfloat16_rn(z[v]);
      }
    }
  }
}

template <typename F>
cudaError_t launch_pdl(F* kern, int blocks, int threads, const RouteParams& r,
                       cudaStream_t stream, size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, r);
}

bool tiled(int64_t tokens, int32_t experts, int32_t top_k) {
  return tokens >= kTileTokens && tokens >= 128 * experts && experts <= kTileExperts && top_k <= kTileTopK;
}

template <typename T, int EIGHTS>
cudaError_t tile_forward(const RouteParams& r, cudaStream_t stream) {
  auto kern = route_tile_kernel<T, EIGHTS>;
  static PerDeviceOnce setup;
  const cudaError_t err = setup.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytes);
  });
  if (err != cudaSuccess) return err;
  // as few rounds of as few warps as shared memory allows
  const int32_t bytes = 32 * ((r.experts + 7) / 8 * 8 + 1) * 4, runs = (r.tokens_per_block + 31) / 32;
  const int32_t most = kTileBytes / bytes < kTileWarps ? kTileBytes / bytes : kTileWarps;
  const int32_t rounds = (runs + most - 1) / most, warps = (runs + rounds - 1) / rounds;
  return launch_pdl(kern, r.blocks, warps * 32, r, stream, warps * bytes);
}

template <typename T, int V>
cudaError_t forward(const RouteParams& r, cudaStream_t stream) {
  if (r.blocks == 1) return launch_pdl(route_kernel<T, V, true>, 1, kThreads, r, stream);
  const cudaError_t err =
      !tiled(r.tokens, r.experts, r.top_k)
          ? launch_pdl(route_kernel<T, V, false>, r.blocks, kThreads, r, stream)
          : r.experts <= 64 ? tile_forward<T, 8>(r, stream) : tile_forward<T, 16>(r, stream);
  if (err != cudaSuccess) return err;
  // Loads and pairs of a thread, if it is one of 512, that make it one of 1024 (65536
  // tokens 19.9 us with 512 threads, 17.8 with 1024; 512 over 128 experts 10.9 and 12.6).
  const int32_t loads = r.blocks * ((r.experts + 3) / 4) / 512;
  const int32_t pairs = r.group * r.tokens_per_block * r.top_k / 512;
  return launch_pdl(route_order_kernel, (r.blocks + r.group - 1) / r.group + 1,
                    loads > 4 || pairs > 4 ? kOrderThreads : kOrderThreads / 2, r, stream);
}

template <typename T, int L, int V>
cudaError_t backward(const RouteParams& r, int num_sms, cudaStream_t stream) {
  constexpr int kTokens = kBackThreads / L;  // of a block at a time
  // Blocks an SM: as many as run side by side where a row takes less than a warp (65536
  // tokens over 64 experts 10.4 us, with 8 blocks 11.4; 262144 34.5 and 38), else more
  // (256 experts 31 us with 8, 35 with 3).
  constexpr int kBlocks = L == 32 ? 8 : V == 8 ? 3 : 6;
  const int64_t need = (static_cast<int64_t>(r.tokens) + kTokens - 1) / kTokens;
  return launch_pdl(route_backward_kernel<T, L, V>,
                    static_cast<int>(need < kBlocks * num_sms ? need : kBlocks * num_sms),
                    kBackThreads, r, stream);
}

// Logits of a lane: a token has a warp forward, and in the gradient as many lanes as
// give each eight, or four for few experts, up to a warp (262144 tokens over 64 experts
// with eight 37.8 us, with four 42.4; 65536 over 256 with sixteen 43, with eight 31).
template <typename T>
cudaError_t by_experts(const RouteParams& r, bool back, int num_sms, cudaStream_t stream) {
  if (r.experts <= 32)
    return back ? backward<T, 8, 4>(r, num_sms, stream) : forward<T, 1>(r, stream);
  if (r.experts <= 64)
    return back ? backward<T, 8, 8>(r, num_sms, stream) : forward<T, 2>(r, stream);
  if (r.experts <= 128)
    return back ? backward<T, 16, 8>(r, num_sms, stream) : forward<T, 4>(r, stream);
  if (r.experts <= 256)
    return back ? backward<T, 32, 8>(r, num_sms, stream) : forward<T, 8>(r, stream);
  return back ? backward<T, 32, 16>(r, num_sms, stream) : forward<T, 16>(r, stream);
}

// Blocks of the two kernels: one up to kOneBlock tokens, then of 32 tokens at
// least.
void split(int64_t tokens, int32_t most, int32_t* blocks, int32_t* per) {
  if (tokens <= kOneBlock) {
    *blocks = 1;
    *per = static_cast<int32_t>(tokens);
    return;
  }
  int64_t b = (tokens + 31) / 32;
  if (b > most) b = most;
  *per = static_cast<int32_t>((tokens + b - 1) / b + 31) / 32 * 32;
  *blocks = static_cast<int32_t>((tokens + *per - 1) / *per);
}

}  // namespace

// For the most blocks that `tokens` or fewer have, in either first kernel (their number
// itself falls where a block's tokens step up: 304 blocks for 9728, 153 for 9729).
size_t route_workspace(int64_t tokens, int32_t experts) {
  if (tokens <= kOneBlock) return 0;
  const int64_t most = (tokens + 31) / 32, blocks = most < kMaxBlocks ? most : kMaxBlocks;
  const size_t row = (experts + 3) / 4 * 4;
  return sizeof(int32_t) * (blocks * row * 3 + blocks);
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  RouteParams r = p;
  r.vec_ids = ((reinterpret_cast<uintptr_t>(r.ids) | reinterpret_cast<uintptr_t>(r.weights)) & 15u) == 0;
  split(r.tokens, tiled(r.tokens, r.experts, r.top_k) ? kTileBlocks : kMaxBlocks, &r.blocks,
        &r.tokens_per_block);
  r.group = r.blocks > kTileBlocks ? 2 : 1;
  return r.logits_fp32 ? by_experts<float>(r, false, 0, stream)
                       : by_experts<bf16>(r, false, 0, stream);
}

cudaError_t launch_route_backward(const RouteParams& p, int num_sms, cudaStream_t stream) {
  return p.logits_fp32 ? by_experts<float>(p, true, num_sms, stream)
                       : by_experts<bf16>(p, true, num_sms, stream);
}

}  // namespace mx
