// vocab_loss.cu -- softmax cross entropy over a vocabulary, with the product
// that gives the logits, without keeping them:
//
//   z = x W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,label
//   dz = (d_loss + d_lse) exp(z - lse) - d_loss [v = label],  dx = dz W,  dW = dz^T x
//
// All four products run on block pairs (tcgen05 cta_group::2, bf16 operands,
// FP32 accumulators): 256 x 256 tiles, 64 elements of the contraction a stage,
// six stages, two accumulators in tensor memory so that the epilogue of a tile
// runs beside the MMAs of the next.  The gradient goes through the vocabulary in
// pieces: dz of a piece is computed again from x and W, rounded to bf16 (it is
// an operand of bf16 MMAs; its 8 significant bits are those that x and W have), in
// units of the largest |d_loss|, and read by the two products, which share a launch: where the tiles of one do not
// fill the device's last round, those of the other do.  Operands that are
// contiguous along M or N (dz and x in dW, W in dx) are read as they lie: the
// tensor core transposes.
//
//   warp 0 (both blocks)  tensor copies of A and of this block's half of B
//   warp 1                tensor memory; in block 0 the MMAs of the pair
//   warps 2..9 (both)     epilogue, 32 rows x 128 columns of the tile each
// All waits are bounded.
//
// Bound by the tensor cores.  Measured on one GB300 in a burst and, behind the slash,
// after seconds of such work, at the power cap (1560 to 1680 MHz; cuBLAS bf16 1884 /
// 1692 TFLOP/s): losses of 4096 tokens over 131072 x 7168 3.9 / 4.3 ms, 1950 / 1780
// TFLOP/s; losses and gradients (four products, one of them z again) 17.1 / 18.5 ms, 1800
// / 1670 TFLOP/s; 2048 tokens over 32768 x 2048 575 / 670 us; 777 over 50257 x 2048 112 /
// 128 us for losses (1430 / 1250; 1880 / 1650 on its 1024 rows of tiles); 333 over
// 18433 x 1000 78 us, latencies of six launches and two rounds of tiles.
// Six stages: with five and a second staging buffer in the gradients' epilogue 12.97
// -> 13.07 ms at the largest, 64.3 -> 62.8 us at the smallest of these.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "status.cuh"
#include "vocab.cuh"

namespace mx {
namespace {

constexpr int kTile = 256;        // rows and columns of a pair's tile
constexpr int kHalf = 128;        // of one block (rows of A, rows of B)
constexpr int kStep = 64;         // contraction elements of a stage (128 bytes)
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalf * kStep * 2;  // 16 KB of A, as many of B
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kStoreBytes = 32 * 128;             // a warp's staging: 32 rows of 128 bytes
constexpr int kOffB = kStages * kOperandBytes;
constexpr int kOffStore = 2 * kOffB;
constexpr int kOffBar = kOffStore + kEpiWarps * kStoreBytes;
constexpr int kNumBars = 2 * kStages + 5;
constexpr int kOffMost = kOffBar + kNumBars * 8 + 16;  // a float a warp of the epilogue
constexpr int kSmemBytes = kOffMost + kEpiWarps * 4 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
constexpr uint32_t kTmemCols = 512;
constexpr uint16_t kBoth = 0x3;
// Tiles are walked in bands of this many rows of tiles, columns outer inside a
// band: the band's part of A (59 MB at hidden 7168) stays in L2 while B goes by once.
constexpr int kBand = 16;
// Tile of a unit of work.
struct Unit {
  int32_t m, n, step0, steps, part;
};

__device__ __forceinline__ Unit unit_of(const VocabParams& p, int32_t u) {
  const int32_t m_units = (p.m + kTile - 1) / kTile, n_tiles = (p.n + kTile - 1) / kTile;
  Unit t;
  const int32_t tiles = m_units * n_tiles;
  t.part = u / tiles;
  const int32_t r = u - t.part * tiles;
  const int32_t band = r / (kBand * n_tiles);
  const int32_t rows = min(kBand, m_units - band * kBand);
  const int32_t w = r - band * kBand * n_tiles;
  t.n = w / rows;
  t.m = band * kBand + (w - t.n * rows);
  t.step0 = t.part * p.steps;
  t.steps = min(p.steps, (p.k + kStep - 1) / kStep - t.step0);
  return t;
}

__host__ __device__ __forceinline__ int64_t units_of(const VocabParams& p) {
  return static_cast<int64_t>((p.m + kTile - 1) / kTile) * ((p.n + kTile - 1) / kTile) * p.splits;
}

// What dz is held in units of: the largest |d_loss| of the tokens that count.  A mean's
// d_loss is the same for all of them, and so would be its rounding in every label's entry:
// the gradient would be off by up to 2^-8 in one direction (255 tokens).  In these units the
// entry is -1 and the label's probability.  (1 where that is nothing, not finite, or so far
// from 1 that dz could leave the type's range.)  Of all epilogue threads of a block.
__device__ __forceinline__ float dz_unit(const VocabParams& p, float* most_of_warp) {
  const int32_t first = static_cast<int32_t>(threadIdx.x) - 64;
  float most = 0.f;
  if (p.d_loss) {
#pragma unroll 4
    for (int32_t t = first; t < p.tokens; t += kEpiWarps * 32)
      if (counts(p, label_of(p, t))) most = fmaxf(most, fabsf(p.d_loss[t]));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
  if (lane_id() == 0) most_of_warp[first / 32] = most;
  asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
#pragma unroll
  for (int i = 0; i < kEpiWarps; ++i) most = fmaxf(most, most_of_warp[i]);
  return most >= 0x1p-100f && most <= 0x1p100f ? most : 1.f;
}

// A product and the maps of its operands and output.
struct Product {
  CUtensorMap a, b, y;
  VocabParams p;
};
// What a kernel computes: the logits' product alone, or dx and dW, one after the other
// (units of the second follow those of the first).
template <bool GRADIENTS>
struct Work {
  Product first, second;
};
template <>
struct Work<false> {
  Product first;
};

// W: kStats, kGrad, or kDx for both gradients.  RUNS: the contraction is taken in runs
// (kStats: one or more; kGrad: more than one).
template <VocabProduct W, bool RUNS>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_product_kernel(const __grid_constant__ Work<W == VocabProduct::kDx> work) {
  constexpr bool kGradients = W == VocabProduct::kDx;
  const VocabParams& p = work.first.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kOffB;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // one per accumulator
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* s_abort = s_tmem + 1;

  const uint32_t warp = warp_id();
  const uint32_t lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int32_t cluster = blockIdx.x / 2;
  const int32_t clusters = gridDim.x / 2;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *s_abort = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&work.first.a);
    tma_prefetch_desc(&work.first.b);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(s_tmem, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync();  // barriers of both blocks exist before any use from the other
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;
  pdl_wait();
  pdl_launch_dependents();

  const int32_t units0 = static_cast<int32_t>(units_of(p));
  int32_t units = units0;
  if constexpr (kGradients) units += static_cast<int32_t>(units_of(work.second.p));
  // the product that a unit belongs to
  auto second = [&](int32_t u) { return kGradients && u >= units0; };
  auto product = [&](int32_t u) -> const Product& {
    if constexpr (kGradients) return u >= units0 ? work.second : work.first;
    else return work.first;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t full_leader0 = cluster_map(&full[0], 0);
    uint32_t stage = 0, phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int32_t u = cluster; u < units && ok; u += clusters) {
      const Product& w = product(u);
      const bool dw = second(u);
      const Unit t = unit_of(w.p, dw ? u - units0 : u);
      const int32_t a0 = t.m * kTile + static_cast<int32_t>(rank) * kHalf;
      const int32_t b0 = t.n * kTile + static_cast<int32_t>(rank) * kHalf;
      for (int32_t i = 0; i < t.steps; ++i) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, s_abort, p.status, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        int32_t k0 = (t.step0 + i) * kStep, kb = k0;
        if (kGradients && w.p.low_row) k0 = i * w.p.low_row, kb = 0;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], 4u * kOperandBytes);
          const uint32_t bar = full_leader0 + stage * 8u;
          uint8_t* a = sA + stage * kOperandBytes;
          uint8_t* b = sB + stage * kOperandBytes;
          if (dw) {
            tma_load_2d_pair(a, &w.a, bar, a0, k0);
            tma_load_2d_pair(a + kOperandBytes / 2, &w.a, bar, a0 + 64, k0);
          } else {
            tma_load_2d_pair(a, &w.a, bar, k0, a0);
          }
          if constexpr (kGradients) {
            tma_load_2d_pair(b, &w.b, bar, b0, kb);
            tma_load_2d_pair(b + kOperandBytes / 2, &w.b, bar, b0 + 64, kb);
          } else {
            tma_load_2d_pair(b, &w.b, bar, kb, b0);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // until block 0 has consumed every fill, copies into this block's ring and
    // arrivals on its barriers are pending
    for (int s = 0; s < kStages; ++s) {
      const int64_t fills = issued > s ? (issued - s + kStages - 1) / kStages : 0;
      if (fills)
        mbar_wait_warp(&empty[s], static_cast<uint32_t>((fills - 1) & 1), s_abort, p.status,
                       p.wait_limit_ns, true);
    }
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------ MMA issuer
    // An operand contiguous along K: rows of 128 bytes, eight of them 1024 bytes;
    // 16 elements on are 32 bytes.  Contiguous along M or N: 64 of them are a row
    // of 128 bytes, rows follow along K, the next 64 lie 8 KB on; 16 elements of K on
    // are 2 KB.
    constexpr uint32_t kHi = smem_desc_hi(1024, 2);
    constexpr uint32_t kMnLbo = kOperandBytes / 2, kMnNext = 2048 >> 4, kKNext = 32 >> 4;
    constexpr uint32_t kNextB = kGradients ? kMnNext : kKNext;
    const uint32_t b_lo0 = smem_desc_lo(smem_u32(sB), kGradients ? kMnLbo : 16);
    uint32_t stage = 0, phase = 0, buf = 0, acc_phase = 0;
    bool ok = true;
    for (int32_t u = cluster; u < units && ok; u += clusters) {
      const Product& w = product(u);
      const bool dw = second(u);
      const Unit t = unit_of(w.p, dw ? u - units0 : u);
      const uint32_t a_lo0 = smem_desc_lo(smem_u32(sA), dw ? kMnLbo : 16);
      const uint32_t next_a = dw ? kMnNext : kKNext;
      const uint32_t idesc = bf16_idesc(kTile, kTile, dw, kGradients);
      const Runs runs(t.steps, RUNS);
      for (int32_t i0 = 0; i0 < t.steps && ok; i0 += runs.steps) {
        if (!mbar_wait_warp(&acc_empty[buf], acc_phase ^ 1u, s_abort, p.status, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t acc = tmem_base + buf * kTile;
        const int32_t end = min(t.steps, i0 + runs.steps);
        for (int32_t i = i0; i < end; ++i) {
          if (!mbar_wait_warp(&full[stage], phase, s_abort, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_lo = a_lo0 + stage * (kOperandBytes >> 4);
          const uint32_t b_lo = b_lo0 + stage * (kOperandBytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (uint32_t j = 0; j < kStep / 16; ++j)
              tc_mma_pair_f16(acc, a_lo + j * next_a, kHi, b_lo + j * kNextB, kHi, idesc,
                              (i > i0 || j > 0) ? 1u : 0u);
            tc_commit_pair_multicast(&empty[stage], kBoth);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_multicast(&acc_full[buf], kBoth);
        __syncwarp();
        buf ^= 1u;
        if (buf == 0) acc_phase ^= 1u;
      }
    }
    if (elect_one()) {
      tc_commit_pair_multicast(mma_done, 0x1);
      mbar_wait(mma_done, 0, s_abort, p.status, p.wait_limit_ns, true);
    }
    __syncwarp();
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const uint32_t q = warp & 3u;            // lanes of tensor memory: rows 32 q .. 32 q + 31
    const uint32_t half = (warp - 2) >> 2;   // columns 128 half .. + 127
    uint8_t* store = smem + kOffStore + (warp - 2) * kStoreBytes;
    const uint32_t empty_leader0 = cluster_map(&acc_empty[0], 0);
    float unit = 1.f;  // of dz
    if constexpr (W == VocabProduct::kGrad) {
      unit = dz_unit(p, reinterpret_cast<float*>(smem + kOffMost));
      if (blockIdx.x == 0 && threadIdx.x == 64) *p.scale = unit;
    } else if constexpr (kGradients) {
      if (p.scale) unit = *p.scale;
    }
    uint32_t buf = 0, acc_phase = 0;
    for (int32_t u = cluster; u < units; u += clusters) {
      const Product& w = product(u);
      const bool dw = second(u);
      const Unit t = unit_of(w.p, dw ? u - units0 : u);
      const int32_t row0 = t.m * kTile + static_cast<int32_t>(rank * kHalf + q * 32);
      const int32_t row = row0 + static_cast<int32_t>(lane);
      const int32_t col0 = t.n * kTile + static_cast<int32_t>(half) * kHalf;
      // what the row needs of global memory, asked for ahead of the wait
      float lse2 = 0.f, both = 0.f, once = 0.f;
      int32_t label = -1;  // the label's column of this tile half
      if constexpr (W == VocabProduct::kStats || W == VocabProduct::kGrad) {
        if (row < p.m) {
          const int64_t l = label_of(p, row);
          const bool valid = counts(p, l);
          if (valid) {
            const int64_t at = l - p.col0 - col0;
            label = at >= 0 && at < kHalf ? static_cast<int32_t>(at) : -1;
          }
          if constexpr (W == VocabProduct::kGrad) {
            lse2 = p.lse[row] * kLog2e;
            once = valid && p.d_loss ? p.d_loss[row] : 0.f;
            both = (once + (p.d_lse ? p.d_lse[row] : 0.f)) / unit;
            once /= unit;
          }
        }
      }
      auto release = [&] {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_cluster(empty_leader0 + buf * 8u);
      };
      auto wait = [&] {
        const bool got = mbar_wait(&acc_full[buf], acc_phase, s_abort, p.status, p.wait_limit_ns);
        return __all_sync(0xffffffffu, got);
      };
      const uint32_t taddr0 = tmem_base + ((q * 32u) << 16) + half * kHalf;
      // the runs' sums, each accumulator released as soon as it is read
      float z[RUNS ? kHalf : 1];
      if constexpr (RUNS) {
        const Runs runs(t.steps, true);
        bool got = true;
        for (int32_t run = 0; run < runs.count; ++run) {
          if (!(got = wait())) break;
          tc_fence_after_sync();
#pragma unroll
          for (int c = 0; c < kHalf; c += 16) {
            uint32_t a[8], b[8];
            tmem_ld_32x32b_x8(taddr0 + buf * kTile + c, a);
            tmem_ld_32x32b_x8(taddr0 + buf * kTile + c + 8, b);
            tmem_ld_wait_for(a, b);
            if (c + 16 == kHalf) release();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              z[c + j] = __uint_as_float(a[j]) + (run == 0 ? 0.f : z[c + j]);
              z[c + 8 + j] = __uint_as_float(b[j]) + (run == 0 ? 0.f : z[c + 8 + j]);
            }
          }
          buf ^= 1u;
          if (buf == 0) acc_phase ^= 1u;
        }
        if (!got) break;
      }
      if constexpr (W == VocabProduct::kStats) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int32_t left = p.n - (col0 + c * 32);  // columns of the matrix from here on
          if (left < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j >= left) z[c * 32 + j] = -INFINITY;
          }
          const int32_t at = label - c * 32;
          if (__any_sync(0xffffffffu, label >= 0 && at >= 0 && at < 32)) {
            float chosen = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j == at) chosen = z[c * 32 + j];
            if (label >= 0 && at >= 0 && at < 32) p.z_label[row] = chosen;
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], z[c * 32 + j]);
          // the reference that both the sum and its later uses take: a value of
          // float, in log2 units
          const float next =
              fmaxf(top, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * kLog2e);
          const float ref = next == -INFINITY ? 0.f : next;
          float s4[4] = {sum * exp2_fast(top - ref), 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) s4[j & 3] += exp2_fast(fmaf(z[c * 32 + j], kLog2e, -ref));
          sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          top = next;
        }
        if (row < p.m)
          p.partial[static_cast<int64_t>(row) * p.slots + t.n * 2 + half] = make_float2(top, sum);
      } else if constexpr (RUNS) {
        // dz, rounded to bf16, straight from the logits' registers to the staging rows
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 128 bytes a row
          const int32_t at = label - c * 64;
          const bool mine = label >= 0 && at >= 0 && at < 64;
          float chosen = 0.f;
          const bool any = __any_sync(0xffffffffu, mine);
          if (any) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (j == at) chosen = z[c * 64 + j];
          }
          auto softmax = [&](float v) { return both * exp2_fast(fmaf(v, kLog2e, -lse2)); };
          if (lane == 0) bulk_wait_read<0>();  // the copy before has left the staging rows
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = pack_bf16x2(softmax(z[c * 64 + j * 8 + 2 * i]),
                                 softmax(z[c * 64 + j * 8 + 2 * i + 1]));
            *reinterpret_cast<uint4*>(store + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
          if (any && mine)
            *reinterpret_cast<__nv_bfloat16*>(store + lane * 128 + (((at >> 3) ^ (lane & 7)) * 16) +
                                              (at & 7) * 2) =
                __float2bfloat16_rn(softmax(chosen) - once);
          fence_proxy_async_shared();
          __syncwarp();
          const int32_t col = col0 + c * 64;
          if (lane == 0 && row0 < p.m && col < p.n) {
            tma_store_3d(&work.first.y, store, col, row0, 0);
            bulk_commit();
          }
        }
      } else {
        if (!wait()) break;
        tc_fence_after_sync();
        const uint32_t taddr = taddr0 + buf * kTile;
        const bool f32 = W != VocabProduct::kGrad && w.p.y_fp32 != 0;
        const int32_t rounds = f32 ? 4 : 2;  // of 128 bytes a row
        for (int32_t c = 0; c < rounds; ++c) {
          const int32_t width = f32 ? 32 : 64;
          uint32_t v[64];
          tmem_ld_32x32b_x32(taddr + c * width, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          if (!f32)
            tmem_ld_32x32b_x32(taddr + c * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          tmem_ld_wait();
          if (c == rounds - 1) release();
          if constexpr (W == VocabProduct::kGrad) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              v[j] = __float_as_uint(
                  both * exp2_fast(fmaf(__uint_as_float(v[j]), kLog2e, -lse2)));
            const int32_t at = label - c * 64;
            if (__any_sync(0xffffffffu, label >= 0 && at >= 0 && at < 64)) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (label >= 0 && j == at) v[j] = __float_as_uint(__uint_as_float(v[j]) - once);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * unit);
            if (!f32) {
#pragma unroll
              for (int j = 32; j < 64; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * unit);
            }
          }
          if (!f32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
          }
          if (lane == 0) bulk_wait_read<0>();  // the copy before has left the staging rows
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(store + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          fence_proxy_async_shared();
          __syncwarp();
          const int32_t col = col0 + c * width;
          if (lane == 0 && row0 < w.p.m && col < w.p.n) {
            if (kGradients && w.p.add)
              tma_add_3d(&w.y, store, col, row0, t.part);
            else
              tma_store_3d(&w.y, store, col, row0, t.part);
            bulk_commit();
          }
        }
        buf ^= 1u;
        if (buf == 0) acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the partner no longer touches this block's memory
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <VocabProduct W, bool RUNS>
cudaError_t launch(const Work<W == VocabProduct::kDx>& work, int64_t units, int num_sms,
                   cudaStream_t stream) {
  auto kern = vocab_product_kernel<W, RUNS>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  // Pairs of blocks that fit the device at once, asked of the runtime the first time
  // (the query takes longer than a launch) and kept as the set-up flag's companion.
  static PerDeviceOnce setup;
  static std::atomic<int> fit[64];
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  std::atomic<int>& clusters = fit[device < 64 ? device : 63];
  err = setup.run([&]() -> cudaError_t {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;  // the query sees the cluster shape only
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms / 2 * 2));
    int active = 0;
    if (cudaOccupancyMaxActiveClusters(&active, kern, &cfg) != cudaSuccess || active < 1)
      active = num_sms / 2;
    clusters.store(active < num_sms / 2 ? active : num_sms / 2);
    return cudaSuccess;
  });
  if (err != cudaSuccess) return err;
  const int max_clusters = clusters.load();
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < max_clusters ? units : max_clusters)));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, work);
}

// One warp per row joins the row's parts.
__global__ void vocab_finish_kernel(const VocabParams p, float* loss, float* lse) {
  pdl_wait();
  pdl_launch_dependents();
  const int32_t row = blockIdx.x * (blockDim.x / 32) + warp_id();
  if (row >= p.tokens) return;
  const float2* part = p.partial + static_cast<int64_t>(row) * p.slots;
  float top = -INFINITY, sum = 0.f;
  for (int32_t i = lane_id(); i < p.slots; i += 32) {
    const float2 v = part[i];
    const float next = fmaxf(top, v.x);
    const float ref = next == -INFINITY ? 0.f : next;
    sum = sum * exp2_fast(top - ref) + v.y * exp2_fast(v.x - ref);
    top = next;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, top, d);
    const float s = __shfl_xor_sync(0xffffffffu, sum, d);
    const float next = fmaxf(top, t);
    const float ref = next == -INFINITY ? 0.f : next;
    sum = sum * exp2_fast(top - ref) + s * exp2_fast(t - ref);
    top = next;
  }
  if (lane_id() == 0) {
    const float l = fmaf(top, kLn2, logf(sum));
    const int64_t label = label_of(p, row);
    lse[row] = l;
    if (counts(p, label)) {
      loss[row] = l - p.z_label[row];
    } else if (label == p.ignore_index) {
      loss[row] = 0.f;
    } else {
      loss[row] = NAN;
      record_device_status(p.status, MX_DEV_BAD_LABEL);
    }
  }
}

__global__ void vocab_join_kernel(const float* __restrict__ parts, int32_t splits, int64_t n,
                                  uint4* __restrict__ y) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n / 8;
       i += step) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
    for (int32_t s = 0; s < splits; ++s) {
      const float4* src = reinterpret_cast<const float4*>(parts + s * n) + 2 * i;
      const float4 u = src[0], v = src[1];
      a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
      b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
    }
    y[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                      pack_bf16x2(b.z, b.w));
  }
}

}  // namespace

cudaError_t launch_vocab_logits(VocabProduct which, const VocabParams& p, const CUtensorMap& tmap_a,
                                const CUtensorMap& tmap_b, const CUtensorMap& tmap_y, int num_sms,
                                cudaStream_t stream) {
  const Work<false> work = {{tmap_a, tmap_b, tmap_y, p}};
  if (which == VocabProduct::kStats)
    return launch<VocabProduct::kStats, true>(work, units_of(p), num_sms, stream);
  // (a single run's logits go to dz from the accumulator, by halves: 4096 tokens x 512 over
  // 65536 columns 586 us, through the registers that several runs take 650; 2048 x 2048
  // over 32768, two runs, 437 us either way)
  return p.steps > kRunSteps ? launch<VocabProduct::kGrad, true>(work, units_of(p), num_sms, stream)
                             : launch<VocabProduct::kGrad, false>(work, units_of(p), num_sms, stream);
}

cudaError_t launch_vocab_gradients(const VocabGradient* dx, const VocabGradient* dw, int num_sms,
                                   cudaStream_t stream) {
  if (!dx && !dw) return cudaSuccess;
  Work<true> work;
  const VocabGradient& any = dx ? *dx : *dw;
  work.first = {*any.a, *any.b, *any.y, *any.p};
  work.second = work.first;
  if (!dx) work.first.p.m = 0;  // (no units)
  if (!dw) work.second.p.m = 0;
  if (dx && dw) work.second = {*dw->a, *dw->b, *dw->y, *dw->p};
  return launch<VocabProduct::kDx, false>(work, units_of(work.first.p) + units_of(work.second.p), num_sms,
                                   stream);
}

cudaError_t launch_vocab_finish(const VocabParams& p, float* loss, float* lse,
                                cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.gridDim = dim3(static_cast<unsigned>((p.tokens + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, vocab_finish_kernel, p, loss, lse);
}

cudaError_t launch_vocab_join(const float* parts, int32_t splits, int64_t n, void* y, int num_sms,
                              cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = pdl_attribute();
  const int64_t blocks = (n / 8 + 255) / 256;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < num_sms * 8 ? blocks : num_sms * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, vocab_join_kernel, parts, splits, n, static_cast<uint4*>(y));
}

}  // namespace mx
