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
// Two kernels.  The first gives every token to a group of lanes, which hold its
// logits in registers, finds the winners one after the other (a maximum over the
// group, then the lowest lane and place that hold it) and counts them per block.
// The second gives every pair its place: a block adds up the counts of the blocks
// before it, its warps' counts, and the lanes before it with the same expert; one
// block more writes what is left, the sums over all blocks.  Counts are integers
// and the sums of p run in a fixed order, so the same inputs give the same bits.
// Up to kOneBlock tokens, one block does all of it in one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBackThreads = 256;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kMaxBlocks = 304;
constexpr int kOneBlock = 64;

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
  if (vec) {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      if (c + v >= n) continue;
      if constexpr (sizeof(T) == 4) {
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

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The lanes of this thread's group, as a mask of the warp.
template <int L>
__device__ __forceinline__ uint32_t group_mask() {
  return (L == 32 ? 0xffffffffu : (1u << (L % 32)) - 1u) << (lane_id() / L * L);
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
  float sums[kWarps];
  union {
    int2 win[kWarps][4][kMaxTopK];         // winners of the tokens under way: expert, key
    float p[kWarps][kMaxExperts];
    int32_t next[kWarps][kMaxExperts];     // a warp's next place for each expert
    int4 part[2][kThreads];                // a thread's sums over blocks
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

// Places of the pairs of tokens [t0, t1): s.base holds each expert's first.
__device__ __forceinline__ void place_pairs(const RouteParams& r, RouteShared& s, int32_t t0,
                                            int32_t t1) {
  const int32_t warp = warp_id(), lane = lane_id();
  const int32_t lo = t0 * r.top_k, n = (t1 - t0) * r.top_k;
  const int32_t per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int32_t a = lo + min(n, warp * per), b = lo + min(n, (warp + 1) * per);
  int32_t* next = s.next[warp];
  for (int32_t e = lane; e < r.experts; e += 32) next[e] = 0;
  __syncwarp();
  for (int32_t i = a + lane; i < b; i += 32) atomicAdd(&next[r.ids[i]], 1);
  __syncthreads();
  for (int32_t e = threadIdx.x; e < r.experts; e += kThreads) {
    int32_t at = s.base[e];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int32_t c = s.next[w][e];
      s.next[w][e] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int32_t i = a; i < b; i += 32) {
    const bool here = i + lane < b;
    const int32_t e = here ? r.ids[i + lane] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int32_t rank = __popc(same & ((1u << lane) - 1u));
    int32_t at = 0;
    if (here) at = next[e] + rank;
    __syncwarp();
    if (here) {
      r.order[at] = i + lane;
      if (rank == 0) next[e] = at + __popc(same);
    }
    __syncwarp();
  }
}

// The balance loss from each thread's share of sum counts_e sum p_te.
__device__ __forceinline__ void write_balance(const RouteParams& r, RouteShared& s, float share,
                                              int32_t tokens) {
  share = group_sum<32>(share);
  if (lane_id() == 0) s.sums[warp_id()] = share;
  __syncthreads();
  if (threadIdx.x == 0) {
    float all = 0.f;
    for (int w = 0; w < kWarps; ++w) all += s.sums[w];
    const float n = static_cast<float>(tokens);
    *r.balance = tokens ? all / n / n * (static_cast<float>(r.experts) / static_cast<float>(r.top_k))
                        : 0.f;
  }
}

template <typename T, int L, int V, bool ONE>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteParams r) {
  constexpr int kGroups = 32 / L;  // tokens of a warp at a time
  __shared__ RouteShared s;
  const int32_t warp = warp_id();
  const int32_t lane = lane_id() % L, group = lane_id() / L;
  const uint32_t mask = group_mask<L>();
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
  int2* win = s.win[warp][group];
  const T* logits = static_cast<const T*>(r.logits);
  int32_t base = t0 + warp * kGroups;
  if (base + group < t1) load_logits<T, V>(logits + (base + group) * r.ld, c0, r.experts, r.vec, z);
  for (; base < t1; base += kWarps * kGroups) {
    const int32_t t = base + group;
    const bool here = t < t1;
    const bool valid = here && (!r.mask || r.mask[t] != 0);
    if (t + kWarps * kGroups < t1)
      load_logits<T, V>(logits + (t + kWarps * kGroups) * r.ld, c0, r.experts, r.vec, ahead);
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = c0 + v < r.experts ? key_of(z[v]) : 0u;
    float top = 0.f;
    for (int32_t j = 0; j < r.top_k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = max(best, key[v]);
      const uint32_t most = __reduce_max_sync(mask, best);
      const uint32_t who = __ballot_sync(0xffffffffu, best == most) & mask;
      if (j == 0) top = logit_of(most);
      if (static_cast<int32_t>(lane_id()) == __ffs(who) - 1) {
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
      z[v] = c0 + v < r.experts ? expf(z[v] - top) : 0.f;
      sum += z[v];
    }
    sum = group_sum<L>(sum);
    const float inv = 1.f / sum;
    if (valid) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(z[v], inv, acc[v]);
      if (lane == 0) atomicAdd(&s.tokens, 1);
    }
    __syncwarp();
    // the winners side by side
    float picked = 0.f;
    for (int32_t j = lane; j < r.top_k; j += L) {
      const int2 w = win[j];
      const float e = expf(logit_of(static_cast<uint32_t>(w.y)) - top);
      picked += e;
      if (here) {
        r.ids[t * r.top_k + j] = w.x;
        atomicAdd(&s.pairs[w.x], 1);
        if (valid) atomicAdd(&s.counted[w.x], 1);
        if (!r.renormalize) r.weights[t * r.top_k + j] = e * inv;
        win[j].y = __float_as_int(e);
      }
    }
    if (r.renormalize) {
      // p / sum of p, so that a softmax that is NaN stays so
      picked = group_sum<L>(picked);
      const float scale = inv / (picked * inv);
      if (here)
        for (int32_t j = lane; j < r.top_k; j += L)
          r.weights[t * r.top_k + j] = __int_as_float(win[j].y) * scale;
    }
    if (here && lane == 0) r.lse[t] = top + logf(sum);
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = ahead[v];
  }
  // sums of p: groups of a warp, then warps
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a = acc[v];
#pragma unroll
    for (int d = L; d < 32; d <<= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
    if (group == 0 && c0 + v < r.experts) s.p[warp][c0 + v] = a;
  }
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
    place_pairs(r, s, t0, t1);
  } else {
    if (threadIdx.x == 0) parts.tokens[blockIdx.x] = s.tokens;
  }
}

__device__ __forceinline__ void add4(int4& a, const int4& b) {
  a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
}

// Block b < blocks: places of that block's pairs; the last block: counts, offsets
// and the balance loss.
__global__ void __launch_bounds__(kThreads) route_order_kernel(const RouteParams r) {
  __shared__ RouteShared s;
  pdl_wait();
  pdl_launch_dependents();
  const Parts parts(r);
  const int32_t block = blockIdx.x;
  const bool last = block == r.blocks;
  // four experts a thread, the blocks' rows dealt out to as many threads as there
  // are for each
  const int32_t quads = parts.row / 4, slices = kThreads / quads;
  const int32_t quad = threadIdx.x % quads, slice = threadIdx.x / quads;
  int4 all = make_int4(0, 0, 0, 0), before = all;
  if (slice < slices) {
#pragma unroll 4
    for (int32_t b = slice; b < r.blocks; b += slices) {
      const int4 c = *reinterpret_cast<const int4*>(parts.pairs + b * parts.row + quad * 4);
      add4(all, c);
      if (b < block) add4(before, c);
    }
    s.part[0][slice * quads + quad] = all;
    s.part[1][slice * quads + quad] = before;
  }
  __syncthreads();
  for (int32_t e = threadIdx.x; e < r.experts; e += kThreads) {
    int32_t a = 0, b = 0;
    for (int32_t i = 0; i < slices; ++i) {
      a += reinterpret_cast<const int32_t*>(s.part[0])[i * parts.row + e];
      b += reinterpret_cast<const int32_t*>(s.part[1])[i * parts.row + e];
    }
    s.pairs[e] = a;
    s.base[e] = last ? 0 : b;
  }
  __syncthreads();
  scan_experts(s, r.experts, s.pairs, last ? r.offsets : nullptr);
  if (!last) {
    const int32_t t0 = block * r.tokens_per_block;
    place_pairs(r, s, t0, min(r.tokens, t0 + r.tokens_per_block));
    return;
  }
  int32_t n = 0;
  for (int32_t b = threadIdx.x; b < r.blocks; b += kThreads) n += parts.tokens[b];
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
  for (int32_t e = threadIdx.x; e < r.experts; e += kThreads) {
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
  const int32_t step = gridDim.x * kWarps * kGroups;
  for (int32_t base = (blockIdx.x * kWarps + warp_id()) * kGroups; base < r.tokens; base += step) {
    const int32_t t = base + group;
    const bool here = t < r.tokens;
    float z[V];
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = 0.f;
    float lse = 0.f;
    bool valid = false;
    if (here) {
      load_logits<T, V>(static_cast<const T*>(r.logits) + t * r.ld, c0, r.experts, r.vec, z);
      lse = r.lse_in[t];
      valid = !r.mask || r.mask[t] != 0;
    }
    float dot = 0.f;
    if (r.d_weights) {
      float w[kPer], g[kPer];
      int32_t id[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int32_t j = lane + i * L;
        id[i] = -1;
        if (here && j < r.top_k) {
          const int32_t at = t * r.top_k + j;
          id[i] = r.ids_in[at];
          w[i] = r.w_in[at];
          g[i] = r.d_weights[at];
          dot = fmaf(w[i], g[i], dot);
        }
      }
      dot = group_sum<L>(dot);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (id[i] >= 0) mine[id[i]] = w[i] * (g[i] - (r.renormalize ? dot : 0.f));
      __syncwarp();
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const float4 q = *reinterpret_cast<const float4*>(mine + c0 + v);
        add[v] = q.x, add[v + 1] = q.y, add[v + 2] = q.z, add[v + 3] = q.w;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (id[i] >= 0) mine[id[i]] = 0.f;
    }
    float inner = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[v] = c0 + v < r.experts ? expf(z[v] - lse) : 0.f;
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
                       cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, r);
}

template <typename T, int L, int V>
cudaError_t forward(const RouteParams& r, cudaStream_t stream) {
  if (r.blocks == 1) return launch_pdl(route_kernel<T, L, V, true>, 1, kThreads, r, stream);
  const cudaError_t err =
      launch_pdl(route_kernel<T, L, V, false>, r.blocks, kThreads, r, stream);
  return err != cudaSuccess ? err
                            : launch_pdl(route_order_kernel, r.blocks + 1, kThreads, r, stream);
}

template <typename T, int L, int V>
cudaError_t backward(const RouteParams& r, int num_sms, cudaStream_t stream) {
  constexpr int kTokens = kBackThreads / L;  // of a block at a time
  const int64_t need = (static_cast<int64_t>(r.tokens) + kTokens - 1) / kTokens;
  return launch_pdl(route_backward_kernel<T, L, V>,
                    static_cast<int>(need < 8 * num_sms ? need : 8 * num_sms), kBackThreads, r,
                    stream);
}

// Lanes of a token: four logits each where that is at most a warp.
template <typename T>
cudaError_t by_experts(const RouteParams& r, bool back, int num_sms, cudaStream_t stream) {
  if (r.experts <= 32)
    return back ? backward<T, 8, 4>(r, num_sms, stream) : forward<T, 8, 4>(r, stream);
  if (r.experts <= 64)
    return back ? backward<T, 16, 4>(r, num_sms, stream) : forward<T, 16, 4>(r, stream);
  if (r.experts <= 128)
    return back ? backward<T, 32, 4>(r, num_sms, stream) : forward<T, 32, 4>(r, stream);
  if (r.experts <= 256)
    return back ? backward<T, 32, 8>(r, num_sms, stream) : forward<T, 32, 8>(r, stream);
  return back ? backward<T, 32, 16>(r, num_sms, stream) : forward<T, 32, 16>(r, stream);
}

// Blocks of the two kernels: one up to kOneBlock tokens, then of 32 tokens at
// least.
void split(int64_t tokens, int32_t* blocks, int32_t* per) {
  if (tokens <= kOneBlock) {
    *blocks = 1;
    *per = static_cast<int32_t>(tokens);
    return;
  }
  int64_t b = (tokens + 31) / 32;
  if (b > kMaxBlocks) b = kMaxBlocks;
  *per = static_cast<int32_t>((tokens + b - 1) / b);
  *blocks = static_cast<int32_t>((tokens + *per - 1) / *per);
}

}  // namespace

size_t route_workspace(int64_t tokens, int32_t experts) {
  int32_t blocks, per;
  split(tokens, &blocks, &per);
  const size_t row = (experts + 3) / 4 * 4;
  return blocks == 1 ? 0 : sizeof(int32_t) * (blocks * row * 3 + blocks);
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  RouteParams r = p;
  split(r.tokens, &r.blocks, &r.tokens_per_block);
  return r.logits_fp32 ? by_experts<float>(r, false, 0, stream)
                       : by_experts<bf16>(r, false, 0, stream);
}

cudaError_t launch_route_backward(const RouteParams& p, int num_sms, cudaStream_t stream) {
  return p.logits_fp32 ? by_experts<float>(p, true, num_sms, stream)
                       : by_experts<bf16>(p, true, num_sms, stream);
}

}  // namespace mx
