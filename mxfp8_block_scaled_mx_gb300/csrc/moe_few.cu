// moe_few.cu -- a whole mixture-of-experts layer for 1 to 64 tokens.
//
//   z = x router^T, the top_k largest per token win, w = softmax share;
//   y = sum over the winners e of w_e down_e (silu(gate_e x) * (up_e x))
//
// What bounds it is reading the chosen experts' weights once.  Weights are
// the A operand of the tensor cores (128 rows a tile, straight from their MX
// storage, block scales applied by the MMA), tokens the B operand (N = twice
// the token count rounded up to 16), so that nothing is decoded in registers
// and a token more costs nothing until N outgrows the weights' transfer.
//
// Activations keep their precision on FP8 tensor cores as a sum of two E4M3
// terms per value: hi = E4M3(v / S), lo = E4M3((v / S - hi) * 32), with S the
// power of two that brings the 32-element block's largest value into
// [128, 256).  hi has 4 significant bits, the remainder at most 1/16 of v, so
// hi + lo / 32 holds 8 significant bits: a bf16 exactly (down to 2^-14 of its
// block's largest, below that to within 2^-22 of it), and the FP32 activation
// rounded once as bf16 would be (or to within 2^-22 of its block's largest).
// The terms are rows of one B operand (N = 2 x the padded token count, one MMA
// per 32 of K: an MMA this narrow costs what reading its A tile costs), and
// the epilogue adds their two accumulator columns.
//
// Two launches.  moe_router_kernel forms the logits and x's B operand.
// moe_experts_kernel (one block per SM, cooperative) lets every block choose
// the winners for itself (identical arithmetic), then works through
//   phase 1  gate and up: items of 128 channels of one active expert, K = hidden
//   phase 2  down: items of 128 channels of y, K = all active experts'
//            channels one after the other; the routing weights are in the
//            activations, so one accumulator sums over experts.
// Either phase's 128 x 128 tiles are dealt out as one sequence, evenly and in
// order.  An item whose tiles fall to several blocks is the last of its first
// block's share and the first of every other's, so the others leave their
// part (FP32) and go on, and the first, when it gets there, adds the parts in
// block order to its own: same inputs, same bits, and nobody waits long.  Parts
// start as a NaN that no sum is written as (the router kernel sets them), so
// a value is there once it is not that: no flag to wait for, which cost a
// fence and two more trips to L2.
// Between the phases blocks wait for all activations, with their rings
// already full of down tiles.
//
// Measured on one GB300 (FP8 weights, part of the time that the measured copy
// bandwidth takes for the chosen experts' weights):
//   16 tokens, hidden 7168, 56 of 64 experts of 2048:       384 us, 1.00 (403 on
//       the slowest of several GPUs)
//   64 tokens, hidden 4096, 64 experts of 1536:             223 us, 0.84 (the
//       router kernel's 8 us, SMs that differ by 5 % in speed, and the last join)
//   1 token, hidden 2048, 8 of 128 experts of 768:          18.2 us, 0.32 (a chain
//       of latencies: logits 4, routing 2, first tiles, two joins of 2.5 each)
//   1 token, hidden 7168, 8 experts of 2048, 4-bit weights: 45.6 us, 0.62 (about 8
//       of it that chain; 4-bit tiles alone, without MMAs, tokens and scales, take
//       41: they come at 0.85 of the copy bandwidth, 64 bytes of a row each)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "status.cuh"

namespace mx {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kMaxBlocks = 192;     // workspaces are sized for this many SMs
constexpr int kTile = 128;          // rows and K of a weight tile
constexpr int kTileBytes = kTile * kTile;
constexpr int kSfBytes = 512;       // scales of a tile, and of a B record
constexpr int kTerms = 2;
constexpr int kMaxStages = 9;

__host__ __device__ constexpr int pad_tokens(int t) { return (t + 15) / 16 * 16; }
__host__ __device__ constexpr int64_t tiles(int64_t n) { return (n + kTile - 1) / kTile; }

// One K tile of the B operand as the ring holds it: 2 * pad rows of 128 codes
// (128-byte swizzle; row t is token t's hi, row pad + t its lo), then one tile
// of scales for those rows.
__host__ __device__ constexpr int64_t code_bytes(int pad) { return int64_t(kTerms) * pad * kTile; }
__host__ __device__ constexpr int64_t record_bytes(int pad) { return code_bytes(pad) + kSfBytes; }
static_assert(kTerms * kMaxTokens <= kTile, "the scales of all rows in one tile");
static_assert(2 * 192 + kMaxStages * 8 <= 512, "tensor memory: two sets and the scales");

// Workspace: the count of finished activation items (its first word), logits,
// x's records, the activations' records, parts.  A block's part: gates and ups of
// one item of phase 1, then one item of phase 2.
__host__ __device__ constexpr int64_t part_floats(int tokens) { return int64_t(3) * tokens * kTile; }
struct Layout {
  int64_t logits, x, h, parts, bytes;
};
__host__ __device__ inline Layout layout(int tokens, int64_t hidden, int64_t inter, int experts,
                                         int top_k) {
  const int pad = pad_tokens(tokens);
  const int64_t active = experts < tokens * top_k ? experts : tokens * top_k;
  Layout l;
  l.logits = 4096;
  l.x = l.logits + (int64_t(tokens) * experts * 4 + 255) / 256 * 256;
  l.h = l.x + tiles(hidden) * record_bytes(pad);
  l.parts = l.h + active * tiles(inter) * record_bytes(pad);
  l.bytes = l.parts + kMaxBlocks * part_floats(tokens) * 4;
  return l;
}

// What a part's word holds before its sum: a NaN that put_sum never writes.
constexpr uint32_t kNoSum = 0xFFFFFFFFu;
__device__ __forceinline__ void put_sum(float* p, float v) {
  const uint32_t bits = v != v ? 0x7FC00000u : __float_as_uint(v);
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(bits) : "memory");
}
__device__ __forceinline__ uint32_t get_sum(const float* p) {
  uint32_t bits;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(bits) : "l"(p) : "memory");
  return bits;
}

// Byte of code k (0..127) of row t of a record.
__device__ __forceinline__ uint32_t code_at(uint32_t t, uint32_t k) {
  return t * 128 + (((k >> 4) ^ (t & 7)) << 4) + (k & 15);
}
// Byte of the scale of block j (0..3) of row t in a record's scale tile.
__device__ __forceinline__ uint32_t scale_at(uint32_t t, uint32_t j) {
  return (t & 31) * 16 + (t >> 5) * 4 + j;
}

__device__ __forceinline__ uint32_t e4m3_pair(float hi, float lo) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(code)));
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h2));
  return f;
}

// A warp writes its 32 values (one block, one per lane) of row t, block j of a
// record as two E4M3 terms.
__device__ __forceinline__ void write_block(uint8_t* record, int pad, uint32_t t, uint32_t j,
                                            float v) {
  const uint32_t lane = lane_id();
  const uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu);
  // the exponent of S; not below -122, so that lo's scale, S / 32, exists
  int e = static_cast<int>(amax >> 23) - 127 - 7;
  e = e < -122 ? -122 : e;
  uint32_t hi, lo;
  if (amax >= 0x7F800000u) {  // NaN or Inf in the block
    hi = lo = 0x7Fu;
    e = 0;
  } else {
    const float s = v * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    hi = e4m3_pair(0.f, s) & 0xFFu;
    lo = e4m3_pair(0.f, (s - e4m3_value(hi)) * 32.f) & 0xFFu;
  }
  const uint32_t at = code_at(t, j * 32 + lane);
  record[at] = static_cast<uint8_t>(hi);
  record[pad * kTile + at] = static_cast<uint8_t>(lo);  // pad % 8 == 0: the same swizzle
  if (lane == 0) {
    uint8_t* sf = record + code_bytes(pad);
    sf[scale_at(t, j)] = static_cast<uint8_t>(e + 127);
    sf[scale_at(pad + t, j)] = static_cast<uint8_t>(e + 127 - 5);
  }
}

// ------------------------------------------------------------------ router and x

constexpr int kRouterThreads = 256;
constexpr uint32_t kClearUnits = 16 * kRouterThreads;  // of 16 bytes, per block
constexpr int kRouterWarps = kRouterThreads / 32;  // a block's, shared by one or two experts
constexpr int kRouterTokens = 8;    // per block: the router's rows are read tokens / 8 times

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Logits of expert e for tokens t0 .. t0 + nt - 1 (nt <= T), the part of the row
// of this warp of PARTS, complete in every lane.
template <int T, int PARTS>
__device__ __forceinline__ void dot_tokens(const MoeFewParams& p, int e, int t0, int nt,
                                           float (&sum)[kRouterTokens]) {
  const __nv_bfloat16* x[T];
#pragma unroll
  for (int i = 0; i < T; ++i)  // (past the last token: that token again, not used)
    x[i] = static_cast<const __nv_bfloat16*>(p.x) + (t0 + (i < nt ? i : nt - 1)) * p.ldx;
  const int64_t row = static_cast<int64_t>(e) * p.hidden;
#pragma unroll 2
  for (int c = static_cast<int>((warp_id() & (PARTS - 1)) * 32 + lane_id()) * 8; c < p.hidden;
       c += PARTS * 32 * 8) {
    uint4 raw[T];
#pragma unroll
    for (int i = 0; i < T; ++i) raw[i] = *reinterpret_cast<const uint4*>(x[i] + c);
    float w[8];
    if (p.router_fp32) {
      const float4* r = reinterpret_cast<const float4*>(static_cast<const float*>(p.router) + row + c);
      const float4 a = r[0], b = r[1];
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.router) + row + c), w);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
      float v[8];
      unpack8(raw[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[i] += w[j] * v[j];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < T; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
}

// The router's part is latency: 128 experts x 2048 for one token 3 us, of which
// the launch takes half; rows of x and router are read in 16-byte pieces, and
// tokens beyond one share the router's (one token alone: layer 18.9 us, by the
// form for eight 19.8).  The parts are set by blocks of their own: by the blocks
// that form logits the layer took 1 to 4 us longer.
// Blocks [0, logit_blocks): logits of EACH experts for eight tokens.  The next
// record_blocks: x's records, a warp per token and K tile.  The rest: parts of
// part_units 16-byte units in all set to kNoSum.  Block 0 also clears the counter.
template <int EACH>
__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeFewParams p,
                                                                    int logit_blocks,
                                                                    int record_blocks,
                                                                    uint32_t part_units) {
  __shared__ float part[kRouterThreads / 32][kRouterTokens];
  pdl_wait();
  pdl_launch_dependents();
  const Layout l = layout(p.tokens, p.hidden, p.inter, p.experts, p.top_k);
  const uint32_t warp = warp_id(), lane = lane_id();
  if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<uint32_t*>(p.workspace) = 0;
  if (static_cast<int>(blockIdx.x) >= logit_blocks + record_blocks) {
    uint4* parts = reinterpret_cast<uint4*>(p.workspace + l.parts);
    const uint4 none = make_uint4(kNoSum, kNoSum, kNoSum, kNoSum);
    uint32_t i = (blockIdx.x - logit_blocks - record_blocks) * kClearUnits + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kClearUnits / kRouterThreads; ++j, i += kRouterThreads)
      if (i < part_units) parts[i] = none;
    return;
  }
  if (static_cast<int>(blockIdx.x) >= logit_blocks) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
    const int kt_count = static_cast<int>(tiles(p.hidden));
    const int w = (static_cast<int>(blockIdx.x) - logit_blocks) * (kRouterThreads / 32) + static_cast<int>(warp);
    const int t = w / kt_count, kt = w % kt_count;
    if (t >= p.tokens) return;
    const int pad = pad_tokens(p.tokens);
    uint8_t* record = p.workspace + l.x + kt * record_bytes(pad);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = kt * kTile + j * 32 + static_cast<int>(lane);
      v[j] = c < p.hidden ? __bfloat162float(x[t * p.ldx + c]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) write_block(record, pad, t, j, v[j]);
    return;
  }
  constexpr int kParts = kRouterWarps / EACH;
  const int groups = (p.experts + EACH - 1) / EACH;
  const int e = static_cast<int>(blockIdx.x) % groups * EACH + static_cast<int>(warp) / kParts;
  const int t0 = static_cast<int>(blockIdx.x) / groups * kRouterTokens;
  const int nt = p.tokens - t0 < kRouterTokens ? p.tokens - t0 : kRouterTokens;
  float sum[kRouterTokens];
#pragma unroll
  for (int i = 0; i < kRouterTokens; ++i) sum[i] = 0.f;
  if (e < p.experts) {
    if (nt == 1)
      dot_tokens<1, kParts>(p, e, t0, nt, sum);
    else if (nt <= 4)
      dot_tokens<4, kParts>(p, e, t0, nt, sum);
    else
      dot_tokens<kRouterTokens, kParts>(p, e, t0, nt, sum);
  }
#pragma unroll
  for (int i = 0; i < kRouterTokens; ++i)
    if (lane == 0) part[warp][i] = sum[i];
  __syncthreads();
  if ((warp & (kParts - 1)) == 0 && e < p.experts && static_cast<int>(lane) < nt) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) s += part[warp + i][lane];
    reinterpret_cast<float*>(p.workspace + l.logits)[static_cast<int64_t>(t0 + lane) * p.experts + e] = s;
  }
}

// ------------------------------------------------------------------ experts

constexpr int kEpiWarps = 8;
constexpr int kPartsAtOnce = 4;     // parts of an item that are read at a time,
constexpr int kTokensAtOnce = 4;    // and tokens in phase 1
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr uint32_t kTmemCols = 512;

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2], mma_done;
  uint32_t tmem, abort;
  int32_t active;                           // number of active experts
  uint32_t chosen[kMaxExperts / 32];        // bit per expert
  uint16_t expert[kMaxExperts];             // active experts, ascending
  // the tokens that chose an item's expert, ascending, and their weights:
  // written for one item while the item before may still be read
  uint32_t routed[2][kMaxTokens / 32];      // bit per token
  uint16_t token[2][kMaxTokens];
  float share[2][kMaxTokens];
  uint16_t id[kMaxTokens * kMaxTopK];       // [tokens][top_k]
  float weight[kMaxTokens * kMaxTopK];
};

// Order-preserving key of a logit: equal zeros alike, NaN below everything,
// never 0.
__device__ __forceinline__ uint32_t logit_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return z != z ? 1u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// A warp chooses the winners of token t (N logits a lane): largest logit
// first, the lowest expert among equal ones.
template <int N>
__device__ __forceinline__ void select_experts(const MoeFewParams& p, const float* logits, int t,
                                               Shared* sh) {
  const uint32_t lane = lane_id();
  float z[N];
  uint32_t key[N], top = 0u;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = j * 32 + static_cast<int>(lane);
    z[j] = e < p.experts ? logits[t * p.experts + e] : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    key[j] = j * 32 + static_cast<int>(lane) < p.experts ? logit_key(z[j]) : 0u;
    top = key[j] > top ? key[j] : top;
  }
  const float z0 = key_logit(__reduce_max_sync(0xffffffffu, top));
  float sum = 0.f, chosen = 0.f, my_w = 0.f;
  uint32_t my_e = 0u;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    z[j] = key[j] ? expf(z[j] - z0) : 0.f;
    sum += z[j];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  for (int k = 0; k < p.top_k; ++k) {
    uint32_t best = 0u, at = 0xFFFFFFFFu;
    float w = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j * 32 + lane;
        w = z[j];
      }
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == m ? at : 0xFFFFFFFFu);
    w = __shfl_sync(0xffffffffu, w, e & 31u);
    chosen += w;
    if (lane == static_cast<uint32_t>(k)) {
      my_e = e;
      my_w = w;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (e == j * 32 + lane) key[j] = 0u;
  }
  if (static_cast<int>(lane) < p.top_k) {
    sh->id[t * p.top_k + lane] = static_cast<uint16_t>(my_e);
    // (a NaN anywhere among the logits is one of the whole softmax)
    sh->weight[t * p.top_k + lane] = my_w / (p.renormalize && sum == sum ? chosen : sum);
    atomicOr(&sh->chosen[my_e >> 5], 1u << (my_e & 31u));
  }
}

// A block's run of tiles of one item.
struct Segment {
  int32_t item, k0, k1;   // tiles [k0, k1) of the item's K
};

// One phase's tiles, `per` of each of `items` items in sequence (2^27 at most,
// from the limits on sizes), dealt to the first n blocks: q each, the first r
// blocks one more.
struct Share {
  uint32_t per, total, n, q, r, lo, hi;   // this block's: [lo, hi)
  __device__ __forceinline__ Share(uint32_t items, uint32_t per_item)
      : per(per_item), total(items * per_item) {
    n = total < gridDim.x ? total : gridDim.x;
    q = total / n;
    r = total - q * n;
    lo = blockIdx.x < n ? start(blockIdx.x) : total;
    hi = blockIdx.x < n ? start(blockIdx.x + 1) : total;
  }
  __device__ __forceinline__ uint32_t start(uint32_t b) const { return b * q + (b < r ? b : r); }
  __device__ __forceinline__ uint32_t block_of(uint32_t u) const {
    const uint32_t t = r * (q + 1);
    return u < t ? u / (q + 1) : r + (u - t) / q;
  }
  // the segment that starts at tile u (an empty one at the end of all)
  __device__ __forceinline__ Segment at(uint32_t u) const {
    Segment s;
    s.item = static_cast<int32_t>(u / per);
    s.k0 = static_cast<int32_t>(u - s.item * per);
    const uint32_t end = s.k0 + (hi - u);
    s.k1 = static_cast<int32_t>(end < per ? end : per);
    return s;
  }
};

__device__ __forceinline__ void epi_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
}

// Adds one to *word after everything that this thread has seen done (its
// block's writes before a barrier among it).
__device__ __forceinline__ void add_release(uint32_t* word) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(word) : "memory");
}

// Waits until *word reaches `want`.
__device__ __forceinline__ bool wait_count(const uint32_t* word, uint32_t want,
                                           volatile uint32_t* abort_flag, uint32_t* status,
                                           uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  uint32_t spins = 0;
  while (true) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
    if (v >= want) return true;
    if ((++spins & 15u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > limit_ns) {
        record_device_status(status, MX_DEV_TIMEOUT);
        *abort_flag = 1u;
        return false;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    moe_experts_kernel(const __grid_constant__ CUtensorMap tmap_gate,
                       const __grid_constant__ CUtensorMap tmap_up,
                       const __grid_constant__ CUtensorMap tmap_down, const MoeFewParams p,
                       int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int pad = pad_tokens(p.tokens);
  const uint32_t b_bytes = static_cast<uint32_t>(code_bytes(pad));
  uint8_t* sA = smem;                                 // [stages][16 KB]
  uint8_t* sB = sA + stages * kTileBytes;             // [stages][record, A's scales]
  const uint32_t b_step = b_bytes + 2 * kSfBytes;
  Shared* sh = reinterpret_cast<Shared*>(sB + stages * b_step);
  volatile uint32_t* s_abort = &sh->abort;
  const uint32_t warp = warp_id(), lane = lane_id();
  const Layout l = layout(p.tokens, p.hidden, p.inter, p.experts, p.top_k);
  uint32_t* done_items = reinterpret_cast<uint32_t*>(p.workspace);

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->acc_full[i], 1);
      mbar_init(&sh->acc_empty[i], kEpiWarps);
    }
    mbar_init(&sh->mma_done, 1);
    sh->abort = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmap_gate);
    tma_prefetch_desc(&tmap_up);
    tma_prefetch_desc(&tmap_down);
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem, kTmemCols);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += kThreads) sh->chosen[i] = 0u;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh->tmem;
  pdl_wait();
  pdl_launch_dependents();

  // Routing: every block for itself, block 0 reports it.
  const float* logits = reinterpret_cast<const float*>(p.workspace + l.logits);
  // (four logits a lane where they hold all: one token of 128 experts 18.2 us a
  // layer, with sixteen 19.6)
  for (int t = static_cast<int>(warp); t < p.tokens; t += kThreads / 32) {
    if (p.experts <= 128)
      select_experts<4>(p, logits, t, sh);
    else
      select_experts<kMaxExperts / 32>(p, logits, t, sh);
  }
  __syncthreads();
  if (warp == 2) {
    uint32_t before = 0;
    for (int i = 0; i * 32 < p.experts; ++i) {
      const uint32_t bits = sh->chosen[i];
      if (bits >> lane & 1u)
        sh->expert[before + __popc(bits & ((1u << lane) - 1u))] = static_cast<uint16_t>(i * 32 + lane);
      before += __popc(bits);
    }
    if (lane == 0) sh->active = static_cast<int32_t>(before);
  }
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.tokens * p.top_k; i += kThreads) {
      p.ids[i] = sh->id[i];
      p.weights[i] = sh->weight[i];
    }
  __syncthreads();

  const int32_t it_count = static_cast<int32_t>(tiles(p.inter));
  const int32_t ht_count = static_cast<int32_t>(tiles(p.hidden));
  const int32_t items1 = sh->active * it_count;       // (expert, 128 channels)
  const Share share1(items1, ht_count);               // each tile: gate and up
  const Share share2(ht_count, items1);
  const uint32_t b_record = b_bytes + kSfBytes;
  // accumulators: two columns per padded token, for gate and up; a second
  // set where tensor memory holds it next to the scales (16 tokens of 4096, 64
  // experts of 1024: 136.7 us, with one set 137.5; one token of 2048 18.2 and 18.6)
  const uint32_t acc_cols = 2u * kTerms * pad;
  const uint32_t acc_sets = acc_cols <= 192u ? 2u : 1u;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (in both this role and the next the whole warp computes the operands and
    // one elected lane issues: computed in a one-lane branch they cost more
    // than the tile's transfer)
    const uint32_t tx_gu = kTileBytes * p.bits_gu / 8 + kSfBytes;
    const uint32_t tx_d = kTileBytes * p.bits_d / 8 + kSfBytes;
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    auto next = [&] {
      ++issued;
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    auto wait_empty = [&] {
      return mbar_wait_warp(&sh->empty[stage], phase ^ 1u, s_abort, p.status, p.wait_limit_ns);
    };
    // phase 1: gate tile with x's record, then the up tile (same record)
    const int64_t mat1 = static_cast<int64_t>(it_count) * ht_count * kSfBytes;
    for (uint32_t u = share1.lo; u < share1.hi && ok;) {
      const Segment g = share1.at(u);
      const int32_t a = g.item / it_count;
      const int32_t e = sh->expert[a], tile = g.item - a * it_count;
      const int32_t y = e * p.inter + tile * kTile;
      const int64_t sf0 = e * mat1 + (static_cast<int64_t>(tile) * ht_count + g.k0) * kSfBytes;
      const uint8_t* gate_sf = p.gate_scales + sf0;
      const uint8_t* up_sf = p.up_scales + sf0;
      const uint8_t* record = p.workspace + l.x + g.k0 * record_bytes(pad);
      int32_t x = g.k0 * kTile;
      for (int32_t k = g.k0; k < g.k1; ++k) {
        if (!(ok = wait_empty())) break;
        {
          uint64_t* bar = &sh->full[stage];
          uint8_t *a_dst = sA + stage * kTileBytes, *b_dst = sB + stage * b_step;
          uint8_t* sf_dst = b_dst + b_record;
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, tx_gu + b_record);
            tma_load_2d(a_dst, &tmap_gate, bar, x, y);
            bulk_load(sf_dst, gate_sf, kSfBytes, bar);
            bulk_load(b_dst, record, b_record, bar);
          }
          __syncwarp();
        }
        next();
        if (!(ok = wait_empty())) break;
        {
          uint64_t* bar = &sh->full[stage];
          uint8_t *a_dst = sA + stage * kTileBytes, *sf_dst = sB + stage * b_step + b_record;
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, tx_gu);
            tma_load_2d(a_dst, &tmap_up, bar, x, y);
            bulk_load(sf_dst, up_sf, kSfBytes, bar);
          }
          __syncwarp();
        }
        next();
        gate_sf += kSfBytes;
        up_sf += kSfBytes;
        record += record_bytes(pad);
        x += kTile;
      }
      u += g.k1 - g.k0;
    }
    // phase 2.  The tile at the front: item, k and k's expert (its place among
    // the active) and tile.
    const int64_t mat2 = static_cast<int64_t>(ht_count) * it_count * kSfBytes;
    Segment w = share2.at(share2.lo);  // (a block without a share has nothing at the front)
    int32_t a = w.k0 / it_count, kt = w.k0 - a * it_count;
    int32_t e = share2.lo < share2.hi ? sh->expert[a] : 0;
    auto step = [&] {
      if (++w.k0 == static_cast<int32_t>(share2.per)) {
        w.k0 = kt = a = 0;
        ++w.item;
        e = sh->expert[0];
      } else if (++kt == it_count) {
        kt = 0;
        e = sh->expert[++a];
      }
    };
    auto load_tile = [&](bool with_record) {
      uint64_t* bar = &sh->full[stage];
      uint8_t *a_dst = sA + stage * kTileBytes, *b_dst = sB + stage * b_step;
      uint8_t* sf_dst = b_dst + b_record;
      const uint8_t* sf = p.down_scales + e * mat2 + (static_cast<int64_t>(w.item) * it_count + kt) * kSfBytes;
      const uint8_t* record = p.workspace + l.h + w.k0 * record_bytes(pad);
      const int32_t x = kt * kTile, y = e * p.hidden + w.item * kTile;
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, tx_d + b_record);
        tma_load_2d(a_dst, &tmap_down, bar, x, y);
        bulk_load(sf_dst, sf, kSfBytes, bar);
        if (with_record) bulk_load(b_dst, record, b_record, bar);
      }
      __syncwarp();
    };
    // The weights of the first tiles may come before the activations are
    // complete; their records follow.
    uint32_t u = share2.lo;
    const int first = stage;
    const int32_t first_k = w.k0;
    int ahead = 0;
    for (; ok && ahead < stages && u < share2.hi; ++ahead, ++u) {
      if (!(ok = wait_empty())) break;
      load_tile(false);
      next();
      step();
    }
    if (ahead > 0) {
      const bool ready = wait_count(done_items, items1, s_abort, p.status, p.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ready) && ok;
      fence_proxy_async_global();
      // (also after a wait gave up: every stage begun is completed)
      for (int i = 0; i < ahead; ++i) {
        const int s = first + i < stages ? first + i : first + i - stages;
        const uint8_t* record =
            p.workspace + l.h + (first_k + i) % static_cast<int32_t>(share2.per) * record_bytes(pad);
        uint64_t* bar = &sh->full[s];
        uint8_t* b_dst = sB + s * b_step;
        if (elect_one()) bulk_load(b_dst, record, b_record, bar);
        __syncwarp();
      }
    }
    for (; ok && u < share2.hi; ++u) {
      if (!(ok = wait_empty())) break;
      load_tile(true);
      next();
      step();
    }
    // every copy has landed before the block may end
    for (int s = 0; s < stages; ++s) {
      const int64_t fills = issued > s ? (issued - s + stages - 1) / stages : 0;
      if (fills)
        mbar_wait_warp(&sh->full[s], static_cast<uint32_t>((fills - 1) & 1), s_abort, p.status,
                       p.wait_limit_ns, true);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t kHiOperand = smem_desc_hi(1024, 2);
    constexpr uint32_t kHiScale = smem_desc_hi(128, 0);
    const uint32_t a_lo0 = smem_desc_lo(smem_u32(sA), 16);
    const uint32_t b_lo0 = smem_desc_lo(smem_u32(sB), 16);
    const uint32_t sf_lo0 = smem_desc_lo(smem_u32(sB + b_bytes), 0);  // B's, then A's
    const uint32_t sf_col0 = tmem + acc_sets * acc_cols;
    int stage = 0;
    uint32_t phase = 0, acc = 0, acc_phase = 0;
    bool ok = true;
    auto wait_full = [&] {
      const bool got =
          mbar_wait_warp(&sh->full[stage], phase, s_abort, p.status, p.wait_limit_ns);
      tc_fence_after_sync();
      return got;
    };
    auto next = [&] {
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    auto begin_item = [&] {
      const bool got = mbar_wait_warp(&sh->acc_empty[acc], acc_phase ^ 1u, s_abort, p.status,
                                      p.wait_limit_ns);
      tc_fence_after_sync();
      return got;
    };
    auto end_item = [&] {
      uint64_t* bar = &sh->acc_full[acc];
      if (elect_one()) tc_commit(bar);
      __syncwarp();
      if (++acc == acc_sets) {
        acc = 0;
        acc_phase ^= 1u;
      }
    };
    // the elected lane's part: the tile's blocks times the record's
    auto multiply = [&](uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sfa,
                        uint32_t sfb, uint32_t blocks, uint32_t add) {
#pragma unroll
      for (uint32_t kb = 0; kb < 4; ++kb)
        if (kb < blocks)
          tc_mma_mxf8(d, a_lo + 2u * kb, kHiOperand, b_lo + 2u * kb, kHiOperand,
                      idesc | kb << 4 | kb << 29, sfa, sfb, kb > 0 ? 1u : add);
    };
    {
      const uint32_t idesc = mxf8_idesc(p.type_gu, 0, kTile, kTerms * pad, 0, 0);
      const uint32_t k_blocks = (p.hidden + 31) / 32;
      for (uint32_t u = share1.lo; u < share1.hi && ok;) {
        const Segment g = share1.at(u);
        if (!(ok = begin_item())) break;
        const uint32_t d = tmem + acc * acc_cols, d_up = d + kTerms * pad;
        uint32_t add = 0;
        for (int32_t k = g.k0; k < g.k1; ++k, add = 1) {
          const uint32_t left = k_blocks - k * 4, blocks = left < 4 ? left : 4;
          if (!(ok = wait_full())) break;
          const int gate_stage = stage;
          const uint32_t sfa = sf_col0 + stage * 8u, sfb = sfa + 4u;
          const uint32_t sf_lo = sf_lo0 + stage * (b_step >> 4);
          const uint32_t a_lo = a_lo0 + stage * (kTileBytes >> 4);
          const uint32_t b_lo = b_lo0 + stage * (b_step >> 4);
          if (elect_one()) {
            tc_cp_32x128b_warpx4(sfa, sf_lo + (kSfBytes >> 4), kHiScale);
            tc_cp_32x128b_warpx4(sfb, sf_lo, kHiScale);
            multiply(d, a_lo, b_lo, idesc, sfa, sfb, blocks, add);
          }
          __syncwarp();
          next();
          if (!(ok = wait_full())) break;
          const uint32_t up_sfa = sf_col0 + stage * 8u;
          const uint32_t up_sf_lo = sf_lo0 + stage * (b_step >> 4) + (kSfBytes >> 4);
          const uint32_t up_lo = a_lo0 + stage * (kTileBytes >> 4);
          uint64_t *empty0 = &sh->empty[gate_stage], *empty1 = &sh->empty[stage];
          if (elect_one()) {
            tc_cp_32x128b_warpx4(up_sfa, up_sf_lo, kHiScale);
            multiply(d_up, up_lo, b_lo, idesc, up_sfa, sfb, blocks, add);
            tc_commit(empty0);
            tc_commit(empty1);
          }
          __syncwarp();
          next();
        }
        if (!ok) break;
        end_item();
        u += g.k1 - g.k0;
      }
    }
    {
      const uint32_t idesc = mxf8_idesc(p.type_d, 0, kTile, kTerms * pad, 0, 0);
      const uint32_t k_blocks = (p.inter + 31) / 32;
      int32_t kt = share2.lo < share2.hi ? share2.at(share2.lo).k0 % it_count : 0;
      for (uint32_t u = share2.lo; u < share2.hi && ok;) {
        const Segment g = share2.at(u);
        if (!(ok = begin_item())) break;
        const uint32_t d = tmem + acc * acc_cols;
        uint32_t add = 0;
        for (int32_t k = g.k0; k < g.k1; ++k, add = 1) {
          const uint32_t left = k_blocks - kt * 4, blocks = left < 4 ? left : 4;
          if (!(ok = wait_full())) break;
          const uint32_t sfa = sf_col0 + stage * 8u, sfb = sfa + 4u;
          const uint32_t sf_lo = sf_lo0 + stage * (b_step >> 4);
          const uint32_t a_lo = a_lo0 + stage * (kTileBytes >> 4);
          const uint32_t b_lo = b_lo0 + stage * (b_step >> 4);
          uint64_t* empty = &sh->empty[stage];
          if (elect_one()) {
            tc_cp_32x128b_warpx4(sfa, sf_lo + (kSfBytes >> 4), kHiScale);
            tc_cp_32x128b_warpx4(sfb, sf_lo, kHiScale);
            multiply(d, a_lo, b_lo, idesc, sfa, sfb, blocks, add);
            tc_commit(empty);
          }
          __syncwarp();
          next();
          if (++kt == it_count) kt = 0;
        }
        if (!ok) break;
        end_item();
        u += g.k1 - g.k0;
      }
    }
    if (elect_one()) {
      tc_commit(&sh->mma_done);
      mbar_wait(&sh->mma_done, 0, s_abort, p.status, p.wait_limit_ns, true);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // (after a wait gave up every item is still gone through, without work,
    // so that all epilogue warps meet at every barrier)
    const uint32_t q = warp & 3u;                     // tensor-memory lanes 32 q ..+31
    const int half = static_cast<int>(warp - 2) >> 2; // of an item's tokens
    const int row = static_cast<int>(q * 32 + lane);  // of the tile
    const int tid = static_cast<int>(threadIdx.x) - 64;
    const int64_t part_size = part_floats(p.tokens);
    float* parts1 = reinterpret_cast<float*>(p.workspace + l.parts) + row;
    float* parts2 = parts1 + 2 * p.tokens * kTile;
    const uint32_t t_lane = tmem + (q * 32u << 16);
    uint32_t acc = 0, acc_phase = 0;
    bool ok = true;
    auto wait_acc = [&] {
      const bool got =
          mbar_wait(&sh->acc_full[acc], acc_phase, s_abort, p.status, p.wait_limit_ns);
      if (!__all_sync(0xffffffffu, got)) ok = false;
      tc_fence_after_sync();
    };
    auto release_acc = [&] {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->acc_empty[acc]);
      if (++acc == acc_sets) {
        acc = 0;
        acc_phase ^= 1u;
      }
    };
    // Sum of the parts of blocks c0 + 1 .. c1, in that order, of N values, the
    // i-th `at(i)` floats into a part and wanted where want(i); waits for them
    // to be there.
    auto add_parts = [&](const float* parts, uint32_t c0, uint32_t c1, auto& v,
                         auto want, auto at) {
      constexpr int N = sizeof(v) / sizeof(float);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.f;
      for (uint32_t c = c0 + 1; c <= c1; c += kPartsAtOnce) {
        uint32_t r[kPartsAtOnce][N];
        uint64_t begun = 0;
        for (uint32_t spins = 0;; ++spins) {
          bool missing = false;
#pragma unroll
          for (int b = 0; b < kPartsAtOnce; ++b)
#pragma unroll
            for (int i = 0; i < N; ++i)
              r[b][i] = c + b <= c1 && want(i) ? get_sum(parts + (c + b) * part_size + at(i)) : 0u;
#pragma unroll
          for (int b = 0; b < kPartsAtOnce; ++b)
#pragma unroll
            for (int i = 0; i < N; ++i) missing |= r[b][i] == kNoSum;
          if (!__any_sync(0xffffffffu, missing)) break;
          if (spins == 0) begun = global_timer_ns();
          bool late = *s_abort != 0;
          if (global_timer_ns() - begun > p.wait_limit_ns) {
            record_device_status(p.status, MX_DEV_TIMEOUT);
            *s_abort = 1u;
            late = true;
          }
          if (__any_sync(0xffffffffu, late)) {
            ok = false;
            break;
          }
        }
#pragma unroll
        for (int b = 0; b < kPartsAtOnce; ++b)
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] += __uint_as_float(r[b][i]);
      }
    };

    // phase 1: activations of 128 channels of one expert, for its tokens
    int buf = 0;
    for (uint32_t u = share1.lo; u < share1.hi; buf ^= 1) {
      const Segment g = share1.at(u);
      u += g.k1 - g.k0;
      const uint32_t u0 = g.item * share1.per;
      const uint32_t c0 = share1.block_of(u0), c1 = share1.block_of(u0 + share1.per - 1);
      const bool owner = g.k0 == 0;
      const int32_t a = g.item / it_count, tile = g.item % it_count;
      if (tid < kMaxTokens) {
        const int e = sh->expert[a];
        float w = -1.f;
        if (tid < p.tokens)
          for (int k = 0; k < p.top_k; ++k)
            if (sh->id[tid * p.top_k + k] == e) w = sh->weight[tid * p.top_k + k];
        const bool in = !(w < 0.f);
        const uint32_t bits = __ballot_sync(0xffffffffu, in);
        if (lane == 0) sh->routed[buf][tid >> 5] = bits;
        if (in) {
          // (a second warp's come from the back; the order among tokens has no effect)
          const int at = __popc(bits & ((1u << lane) - 1u));
          const int place = tid < 32 ? at : kMaxTokens - 1 - at;
          sh->token[buf][place] = static_cast<uint16_t>(tid);
          sh->share[buf][place] = w;
        }
      }
      epi_sync();
      const uint32_t low = __popc(sh->routed[buf][0]);
      const int count = static_cast<int>(low + __popc(sh->routed[buf][1]));
      const int i_begin = half == 0 ? 0 : (count + 1) / 2;
      const int i_end = half == 0 ? (count + 1) / 2 : count;
      auto place = [&](int i) { return i < static_cast<int>(low) ? i : kMaxTokens - 1 - (i - static_cast<int>(low)); };
      uint8_t* record = p.workspace + l.h + g.item * record_bytes(pad);
      if (owner && ok) {
        // a token that did not choose this expert has zeros: a lane each
        const int t = half * 32 + static_cast<int>(lane);
        if (t < p.tokens && !(sh->routed[buf][half] >> lane & 1u)) {
#pragma unroll
          for (int term = 0; term < kTerms; ++term) {
            const int r = term * pad + t;
            *reinterpret_cast<uint4*>(record + code_at(r, q * 32)) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(record + code_at(r, q * 32 + 16)) = make_uint4(0, 0, 0, 0);
            record[code_bytes(pad) + scale_at(r, q)] = 127;
          }
        }
      }
      bool held = false;                              // the accumulator is there
      for (int i0 = i_begin; i0 < i_end; i0 += kTokensAtOnce) {
        float v[2 * kTokensAtOnce];                   // gates, then ups
        auto want = [&](int i) { return i0 + i % kTokensAtOnce < i_end; };
        auto at = [&](int i) { return (i / kTokensAtOnce * p.tokens + i0 + i % kTokensAtOnce) * kTile; };
        if (owner && ok) add_parts(parts1, c0, c1, v, want, at);
        if (!held) wait_acc();
        held = true;
        if (!ok) break;
        const uint32_t d = t_lane + acc * acc_cols;
        uint32_t hi[2 * kTokensAtOnce] = {}, lo[2 * kTokensAtOnce] = {};
#pragma unroll
        for (int i = 0; i < 2 * kTokensAtOnce; ++i)
          if (want(i)) {
            const uint32_t col = d + i / kTokensAtOnce * kTerms * pad +
                                 sh->token[buf][place(i0 + i % kTokensAtOnce)];
            tmem_ld_32x32b_x1(col, hi[i]);
            tmem_ld_32x32b_x1(col + pad, lo[i]);
          }
        tmem_ld_wait_for(hi, lo);
        if (!owner) {
#pragma unroll
          for (int i = 0; i < 2 * kTokensAtOnce; ++i)
            if (want(i))
              put_sum(parts1 + blockIdx.x * part_size + at(i), __uint_as_float(hi[i]) + __uint_as_float(lo[i]));
          continue;
        }
#pragma unroll
        for (int i = 0; i < kTokensAtOnce; ++i) {
          if (!want(i)) break;
          const int j = i + kTokensAtOnce, pl = place(i0 + i);
          const float gate = v[i] + (__uint_as_float(hi[i]) + __uint_as_float(lo[i]));
          const float up = v[j] + (__uint_as_float(hi[j]) + __uint_as_float(lo[j]));
          const float act = gate / (1.f + expf(-gate)) * up;
          write_block(record, pad, sh->token[buf][pl], q,
                      tile * kTile + row < p.inter ? act * sh->share[buf][pl] : 0.f);
        }
      }
      if (!held) wait_acc();
      release_acc();
      if (owner) {
        // its records are for every block's copies
        fence_proxy_async_global();
        epi_sync();
        if (tid == 0) add_release(done_items);
      }
    }

    // phase 2: 128 channels of y, for all tokens
    const int t_begin = half * (pad / 2);
    const int t_end = t_begin + pad / 2 < p.tokens ? t_begin + pad / 2 : p.tokens;
    for (uint32_t u = share2.lo; u < share2.hi;) {
      const Segment g = share2.at(u);
      u += g.k1 - g.k0;
      const uint32_t u0 = g.item * share2.per;
      const uint32_t c0 = share2.block_of(u0), c1 = share2.block_of(u0 + share2.per - 1);
      const bool owner = g.k0 == 0;
      bool held = false;
      for (int t = t_begin; t < t_end; t += 8) {
        float v[8];
        auto want = [&](int i) { return t + i < t_end; };
        auto at = [&](int i) { return (t + i) * kTile; };
        if (owner && ok) add_parts(parts2, c0, c1, v, want, at);
        if (!held) wait_acc();
        held = true;
        if (!ok) break;
        const uint32_t d = t_lane + acc * acc_cols + t;
        uint32_t hi[8], lo[8];
        tmem_ld_32x32b_x8(d, hi);
        tmem_ld_32x32b_x8(d + pad, lo);
        tmem_ld_wait_for(hi, lo);
        const int c = g.item * kTile + row;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!want(i)) break;
          const float own = __uint_as_float(hi[i]) + __uint_as_float(lo[i]);
          if (!owner)
            put_sum(parts2 + blockIdx.x * part_size + at(i), own);
          else if (c < p.hidden)
            static_cast<__nv_bfloat16*>(p.y)[(t + i) * p.ldy + c] = __float2bfloat16_rn(v[i] + own);
        }
      }
      if (!held) wait_acc();
      release_acc();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr size_t kSmemMax = 227 * 1024;

}  // namespace

size_t moe_few_workspace(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                         int32_t top_k) {
  return static_cast<size_t>(layout(tokens, hidden, inter, experts, top_k).bytes);
}

cudaError_t launch_moe_few(const MoeFewParams& p, const CUtensorMap& tmap_gate,
                           const CUtensorMap& tmap_up, const CUtensorMap& tmap_down, int num_sms,
                           cudaStream_t stream) {
  static PerDeviceOnce setup;
  cudaError_t err = setup.run([&]() -> cudaError_t {
    return cudaFuncSetAttribute(moe_experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemMax));
  });
  if (err != cudaSuccess) return err;
  const int blocks = num_sms < kMaxBlocks ? num_sms : kMaxBlocks;
  {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    // An expert a block while that makes two blocks an SM at most (one token
    // of 2048, 128 experts: layer 18.1 us, with two experts a block 18.7; 4-bit
    // token of 7168 45.4 and 46.8; but 64 tokens of 64 experts 225.5 and 223.8,
    // 4 tokens of 512 experts 24.9 and 24.2).
    const int token_groups = (p.tokens + kRouterTokens - 1) / kRouterTokens;
    const int each = static_cast<int64_t>(p.experts) * token_groups <= 2 * num_sms ? 1 : 2;
    const int logit_blocks = (p.experts + each - 1) / each * token_groups;
    const int record_blocks = static_cast<int>(
        (p.tokens * tiles(p.hidden) + kRouterThreads / 32 - 1) / (kRouterThreads / 32));
    const uint32_t units = static_cast<uint32_t>(blocks * part_floats(p.tokens) / 4);
    cfg.gridDim = dim3(static_cast<unsigned>(logit_blocks + record_blocks) +
                       (units + kClearUnits - 1) / kClearUnits);
    cfg.blockDim = dim3(kRouterThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, each == 1 ? moe_router_kernel<1> : moe_router_kernel<2>, p, logit_blocks,
                             record_blocks, units);
    if (err != cudaSuccess) return err;
  }
  const int pad = pad_tokens(p.tokens);
  const size_t stage = kTileBytes + code_bytes(pad) + 2 * kSfBytes;
  size_t stages = (kSmemMax - 1024 - sizeof(Shared)) / stage;
  if (stages > kMaxStages) stages = kMaxStages;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;  // the blocks wait for one another
  attr[0].val.cooperative = 1;
  attr[1] = pdl_attribute();
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = stages * stage + sizeof(Shared) + 1024;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_experts_kernel, tmap_gate, tmap_up, tmap_down, p,
                            static_cast<int>(stages));
}

}  // namespace mx
