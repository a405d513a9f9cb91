// vocab_few.cu -- the vocabulary loss for up to 64 tokens, where reading the weights
// bounds every product: the operands change places.
//
//   z^T = W x^T      rows of W are the 128 rows of a tile, tokens its columns
//   dx^T = W^T dz^T  hidden channels are the rows; W is read as it lies (contiguous
//                    along the rows of the tile), the tensor core transposes
//
// dz is held here as two bf16 terms, high and low (16 significant bits): one rounding
// of a label's entry would be most of the gradient's error where few tokens share it,
// and the second term costs MMAs that have nothing else to do.  dx takes both as
// columns of one tile, dW (vocab_loss.cu) as two steps of its contraction.
//
// An MMA then does no work for tokens that are not there, and a stage of the ring
// holds 16 KB of weights and 2 to 16 KB of tokens, so that up to 208 KB of weights
// are on their way to an SM.  One block per SM:
//   warp 0       tensor copies          warp 1   tensor memory, MMAs
//   warps 2..5   epilogue, 32 rows of the tile each
// The softmax runs over rows here, so over lanes: a warp's share of z goes through
// shared memory, token by token, and every lane keeps the running maximum and sum
// of its tokens over all tiles of the block.  All waits are bounded.
//
// Bound by memory.  Measured on one GB300 over 131072 x 4096 weights (1.07 GB, 158 us
// at the measured copy bandwidth): losses of 1 token 168 us, 0.94, of 64 tokens 159;
// losses' gradients of 64 tokens 519 us (weights read twice, their gradient written:
// 475; with one term of dz 527).  The tiles of vocab_loss.cu take 291 us for one token, 181 for 65.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "status.cuh"
#include "vocab.cuh"

namespace mx {
namespace {

constexpr int kRows = 128;        // of a tile
constexpr int kStep = 64;         // contraction elements of a stage (128 bytes)
constexpr int kABytes = kRows * kStep * 2;
constexpr int kEpiWarps = 4;
constexpr int kThreads = (2 + kEpiWarps) * 32;

// N columns of a tile: tokens, or (kDx) both terms of dz of half as many.
template <int N>
struct Few {
  static constexpr int kBBytes = N * kStep * 2;
  static constexpr int kStages = N == 16 ? 12 : N == 32 ? 10 : N == 64 ? 8 : 6;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffZ = kOffB + kStages * kBBytes;
  static constexpr int kShare = N < 32 ? N : 32;
  static constexpr int kZBytes = kShare * 33 * 4;  // 32 rows of z of a warp, up to 32 tokens
  static constexpr int kOffRow = kOffZ + kEpiWarps * kZBytes;
  static constexpr int kOffBar = kOffRow + (N < 64 ? N : 64) * 16;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16 + 1024;  // + alignment slack
  static constexpr uint32_t kTmemCols = 2 * N;  // two accumulators
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(kBBytes % 1024 == 0, "whole swizzle units");
};

// N consecutive 32-bit columns of this warp's 32 tensor-memory lanes.
template <int N>
__device__ __forceinline__ void load_accumulator(uint32_t taddr, uint32_t (&v)[N]) {
  if constexpr (N >= 32) {
#pragma unroll
    for (int c = 0; c < N; c += 32)
      tmem_ld_32x32b_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 8)
      tmem_ld_32x32b_x8(taddr + c, *reinterpret_cast<uint32_t(*)[8]>(&v[c]));
  }
  tmem_ld_wait();
}

template <VocabProduct W, int N>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_few_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_b, const VocabParams p) {
  using C = Few<N>;
  constexpr int kStages = C::kStages;
  constexpr bool kAMn = W == VocabProduct::kDx;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::kOffB;
  // per token: lse in log2 units, d_loss + d_lse, d_loss, label (kGrad)
  float4* s_row = reinterpret_cast<float4*>(smem + C::kOffRow);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // one per accumulator
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* s_abort = s_tmem + 1;
  const uint32_t warp = warp_id();
  const uint32_t lane = lane_id();
  const int32_t block = blockIdx.x, blocks = gridDim.x;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *s_abort = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_b);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;
  pdl_wait();
  pdl_launch_dependents();

  const int32_t tiles = (p.m + kRows - 1) / kRows;
  const int32_t units = tiles * p.splits;
  const int32_t all_steps = (p.k + kStep - 1) / kStep;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t stage = 0, phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int32_t u = block; u < units && ok; u += blocks) {
      const int32_t part = u / tiles, row0 = (u - part * tiles) * kRows;
      const int32_t step0 = part * p.steps, steps = min(p.steps, all_steps - step0);
      for (int32_t i = 0; i < steps; ++i) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, s_abort, p.status, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        const int32_t k0 = (step0 + i) * kStep;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], kABytes + C::kBBytes);
          uint8_t* a = sA + stage * kABytes;
          if constexpr (kAMn) {
            tma_load_2d(a, &tmap_a, &full[stage], row0, k0);
            tma_load_2d(a + kABytes / 2, &tmap_a, &full[stage], row0 + 64, k0);
          } else {
            tma_load_2d(a, &tmap_a, &full[stage], k0, row0);
          }
          uint8_t* b = sB + stage * C::kBBytes;
          tma_load_2d(b, &tmap_b, &full[stage], k0, 0);
          // the low terms' rows follow the high ones' (what a box takes of them with the
          // high ones lands in columns that nobody reads)
          if constexpr (W == VocabProduct::kDx)
            tma_load_2d(b + C::kBBytes / 2, &tmap_b, &full[stage], k0, p.tokens);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // copies and arrivals are pending until every fill has been consumed
    for (int s = 0; s < kStages; ++s) {
      const int64_t fills = issued > s ? (issued - s + kStages - 1) / kStages : 0;
      if (fills)
        mbar_wait_warp(&empty[s], static_cast<uint32_t>((fills - 1) & 1), s_abort, p.status,
                       p.wait_limit_ns, true);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t kHi = smem_desc_hi(1024, 2);
    constexpr uint32_t kNextA = (kAMn ? 2048 : 32) >> 4, kNextB = 32 >> 4;
    constexpr uint32_t kIdesc = bf16_idesc(kRows, N, kAMn, 0);
    const uint32_t a_lo0 = smem_desc_lo(smem_u32(sA), kAMn ? kABytes / 2 : 16);
    const uint32_t b_lo0 = smem_desc_lo(smem_u32(sB), 16);
    uint32_t stage = 0, phase = 0, buf = 0, acc_phase = 0;
    bool ok = true;
    for (int32_t u = block; u < units && ok; u += blocks) {
      const int32_t step0 = u / tiles * p.steps, steps = min(p.steps, all_steps - step0);
      const Runs runs(steps, W != VocabProduct::kDx);
      for (int32_t i0 = 0; i0 < steps && ok; i0 += runs.steps) {
        if (!mbar_wait_warp(&acc_empty[buf], acc_phase ^ 1u, s_abort, p.status, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int32_t end = min(steps, i0 + runs.steps);
        for (int32_t i = i0; i < end; ++i) {
          if (!mbar_wait_warp(&full[stage], phase, s_abort, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_lo = a_lo0 + stage * (kABytes >> 4);
          const uint32_t b_lo = b_lo0 + stage * (C::kBBytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (uint32_t j = 0; j < kStep / 16; ++j)
              tc_mma_f16(tmem_base + buf * N, a_lo + j * kNextA, kHi, b_lo + j * kNextB, kHi,
                         kIdesc, (i > i0 || j > 0) ? 1u : 0u);
            tc_commit(&empty[stage]);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) tc_commit(&acc_full[buf]);
        __syncwarp();
        buf ^= 1u;
        if (buf == 0) acc_phase ^= 1u;
      }
    }
    if (elect_one()) {
      tc_commit(mma_done);
      mbar_wait(mma_done, 0, s_abort, p.status, p.wait_limit_ns, true);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t q = warp & 3u;  // lanes of tensor memory: rows 32 q .. 32 q + 31 of the tile
    float* z = reinterpret_cast<float*>(smem + C::kOffZ + (warp - 2) * C::kZBytes);
    constexpr int kOwn = (N + 31) / 32;  // tokens of a lane
    float top[kOwn], sum[kOwn];
    int64_t label[kOwn];
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      top[o] = -INFINITY;
      sum[o] = 0.f;
      const int32_t t = static_cast<int32_t>(lane) + o * 32;
      label[o] = -1;
      if (W != VocabProduct::kDx && t < p.tokens) {
        const int64_t l = label_of(p, t);
        if (counts(p, l)) label[o] = l - p.col0;
      }
      if constexpr (W == VocabProduct::kGrad) {
        if (warp == 2 && t < N) {
          float4 r = make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
          if (t < p.tokens) {
            const bool valid = counts(p, label_of(p, t));
            r.x = p.lse[t] * kLog2e;
            r.z = valid && p.d_loss ? p.d_loss[t] : 0.f;
            r.y = r.z + (p.d_lse ? p.d_lse[t] : 0.f);
            // (labels of other pieces of the vocabulary match no row)
            r.w = __int_as_float(label[o] >= 0 && label[o] < p.m ? static_cast<int32_t>(label[o]) : -1);
          }
          s_row[t] = r;
        }
      }
    }
    if constexpr (W == VocabProduct::kGrad)
      asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");  // the epilogue warps
    uint32_t buf = 0, acc_phase = 0;
    for (int32_t u = block; u < units; u += blocks) {
      const int32_t part = u / tiles;
      const int32_t row0 = (u - part * tiles) * kRows + static_cast<int32_t>(q * 32);
      const int32_t row = row0 + static_cast<int32_t>(lane);
      auto wait = [&] {
        const bool got = mbar_wait(&acc_full[buf], acc_phase, s_abort, p.status, p.wait_limit_ns);
        return __all_sync(0xffffffffu, got);
      };
      auto release = [&] {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      };
      if constexpr (W == VocabProduct::kDx) {
        // the high and the low terms' sums of 16 tokens at a time
        if (!wait()) break;
        tc_fence_after_sync();
        const uint32_t taddr = tmem_base + ((q * 32u) << 16) + buf * N;
        float* y = static_cast<float*>(p.out) +
                   (static_cast<int64_t>(part) * p.tokens) * p.ld_out + row;
#pragma unroll
        for (int c = 0; c < N / 2; c += 16) {
          uint32_t high[16], low[16];
          load_accumulator<16>(taddr + c, high);
          load_accumulator<16>(taddr + N / 2 + c, low);
          if (c + 16 == N / 2) release();
          if (row < p.m) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (c + j >= p.tokens) break;
              float* at = y + (c + j) * p.ld_out;
              const float sum = __uint_as_float(high[j]) + __uint_as_float(low[j]);
              *at = p.add ? *at + sum : sum;
            }
          }
        }
        buf ^= 1u;
        if (buf == 0) acc_phase ^= 1u;
        continue;
      }
      float v[N];
      const Runs runs(min(p.steps, all_steps - part * p.steps), true);
      bool got = true;
      for (int32_t run = 0; run < runs.count; ++run) {
        if (!(got = wait())) break;
        tc_fence_after_sync();
        uint32_t w[N];
        load_accumulator<N>(tmem_base + ((q * 32u) << 16) + buf * N, w);
        release();
#pragma unroll
        for (int j = 0; j < N; ++j)
          v[j] = run == 0 ? __uint_as_float(w[j]) : v[j] + __uint_as_float(w[j]);
        buf ^= 1u;
        if (buf == 0) acc_phase ^= 1u;
      }
      if (!got) break;
      if constexpr (W == VocabProduct::kStats) {
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
#pragma unroll
          for (int j = 0; j < C::kShare; ++j)
            z[j * 33 + lane] = row < p.m ? v[o * 32 + j] : -INFINITY;
          __syncwarp();
          const int32_t t = static_cast<int32_t>(lane) + o * 32;
          if (t < p.tokens && row0 < p.m) {
            const float* mine = z + lane * 33;
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], mine[j]);
            const float next =
                fmaxf(top[o], fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * kLog2e);
            const float ref = next == -INFINITY ? 0.f : next;
            float s4[4] = {sum[o] * exp2_fast(top[o] - ref), 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 32; ++j) s4[j & 3] += exp2_fast(fmaf(mine[j], kLog2e, -ref));
            sum[o] = (s4[0] + s4[1]) + (s4[2] + s4[3]);
            top[o] = next;
            const int64_t at = label[o] - row0;
            if (label[o] >= 0 && at >= 0 && at < 32) p.z_label[t] = mine[at];
          }
          __syncwarp();
        }
      } else {
        __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(p.out) + row;
        if (row < p.m) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            if (j >= p.tokens) break;
            const float4 r = s_row[j];
            float d = r.y * exp2_fast(fmaf(v[j], kLog2e, -r.x));
            if (__float_as_int(r.w) == row) d -= r.z;
            const __nv_bfloat16 high = __float2bfloat16_rn(d);
            dz[j * p.ld_out] = high;
            dz[(p.tokens + j) * p.ld_out] = __float2bfloat16_rn(d - __bfloat162float(high));
          }
        }
      }
    }
    if constexpr (W == VocabProduct::kStats) {
#pragma unroll
      for (int o = 0; o < kOwn; ++o) {
        const int32_t t = static_cast<int32_t>(lane) + o * 32;
        if (t < p.tokens)
          p.partial[static_cast<int64_t>(t) * p.slots + block * kEpiWarps + q] =
              make_float2(top[o], sum[o]);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <VocabProduct W, int N>
cudaError_t launch(const VocabParams& p, const CUtensorMap& ta, const CUtensorMap& tb, int blocks,
                   cudaStream_t stream) {
  auto kern = vocab_few_kernel<W, N>;
  static PerDeviceOnce setup;
  const cudaError_t err = setup.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Few<N>::kSmemBytes);
  });
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Few<N>::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, p);
}

template <VocabProduct W>
cudaError_t by_tokens(const VocabParams& p, const CUtensorMap& ta, const CUtensorMap& tb,
                      int blocks, cudaStream_t stream) {
  constexpr int kTerms = W == VocabProduct::kDx ? 2 : 1;
  switch (vocab_few_box(p.tokens)) {
    case 16: return launch<W, 16 * kTerms>(p, ta, tb, blocks, stream);
    case 32: return launch<W, 32 * kTerms>(p, ta, tb, blocks, stream);
    default: return launch<W, 64 * kTerms>(p, ta, tb, blocks, stream);
  }
}

}  // namespace

int vocab_few_blocks(int64_t rows, int splits) {
  const int64_t units = (rows + kRows - 1) / kRows * splits;
  return static_cast<int>(units < kVocabFewBlocks ? units : kVocabFewBlocks);
}

cudaError_t launch_vocab_few(VocabProduct which, const VocabParams& p, const CUtensorMap& tmap_a,
                             const CUtensorMap& tmap_b, cudaStream_t stream) {
  const int blocks = vocab_few_blocks(p.m, p.splits);
  switch (which) {
    case VocabProduct::kStats:
      return by_tokens<VocabProduct::kStats>(p, tmap_a, tmap_b, blocks, stream);
    case VocabProduct::kGrad:
      return by_tokens<VocabProduct::kGrad>(p, tmap_a, tmap_b, blocks, stream);
    case VocabProduct::kDx:
      return by_tokens<VocabProduct::kDx>(p, tmap_a, tmap_b, blocks, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace mx
