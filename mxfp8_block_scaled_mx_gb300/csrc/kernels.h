// kernels.h -- launch interface between the C-ABI layer (mx_api.cu) and the
// CUDA kernels (quantize.cu and quantize_f32.cu, which instantiate
// quantize_kernel.cuh; gemm_pair.cu; norm.cu, norm_mixed.cu and norm_f32.cu,
// which instantiate norm_kernel.cuh; moe_few.cu; rotate.cu,
// rotate_f32.cu, rotate_back.cu and rotate_back_f32.cu, which instantiate
// rotate_kernel.cuh; route.cu; vocab_loss.cu; vocab_few.cu;
// status.cu).  Not part of the public
// ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace mx {

// Launch attribute of every kernel of the library: programmatic stream
// serialization (the kernels wait for their predecessor with griddepcontrol
// before touching global memory).
inline cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// One-time set-up of a kernel per device (its dynamic shared-memory limit):
// `fn` runs until it first succeeds on the current device.  The flags are
// guarded by a mutex, so concurrent first calls from several host threads
// are safe.
class PerDeviceOnce {
 public:
  template <typename Fn>
  cudaError_t run(Fn&& fn) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kMaxDev) return fn();
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev]) return cudaSuccess;
    err = fn();
    if (err == cudaSuccess) done_[dev] = true;
    return err;
  }

 private:
  static constexpr int kMaxDev = 64;
  std::mutex mu_;
  bool done_[kMaxDev] = {};
};

struct QuantizeParams {
  const void* x;       // bf16 or FP32 elements, [rows, cols], leading dimension ldx
                       // (the kernels read x through its tensor map)
  int64_t rows;
  int64_t cols;
  int64_t ldx;
  uint8_t* q_row;      // [rows, cols] codes or nullptr
  uint8_t* s_row;      // swizzled scales of the [rows, cols] operand
  uint8_t* q_col;      // [cols, rows] codes or nullptr
  uint8_t* s_col;      // swizzled scales of the [cols, rows] operand
  int32_t fmt;         // element format: 0 E4M3, 1 E5M2, 2 E2M3, 3 E3M2, 4 E2M1; 5-7 the
                       // last three in packed storage
  int32_t rule;        // 0 = floor, 1 = ceil
  const int32_t* offsets;  // grouped only: device int32[groups + 1]
  int32_t groups;
  uint32_t* status;    // device status word
  uint64_t wait_limit_ns;
  int64_t ldq_col;     // columns of the q_col matrix (dense: rows; grouped: the
                       // 128-padded token capacity, a multiple of 128)
};

// tmap_x: 2-D bf16 tensor map over x (box 64 columns x 128 rows, 128-byte
// swizzle); tmap_r: the same over the 16-bit random integers for stochastic
// rounding, or nullptr for round-to-nearest-even.
cudaError_t launch_quantize(const QuantizeParams& p, const CUtensorMap& tmap_x,
                            const CUtensorMap* tmap_r, int num_sms, cudaStream_t stream);
// Grouped: rowwise (q_row) and/or columnwise (q_col, per-group padded
// segments of 128 columns) quantization of token groups.
cudaError_t launch_quantize_grouped(const QuantizeParams& p, const CUtensorMap& tmap_x,
                                    int num_sms, cudaStream_t stream);
// The same for FP32 x: tmap_x is a 2-D FP32 tensor map (box 32 columns x 128
// rows, 128-byte swizzle); tmap_r as above.
cudaError_t launch_quantize_f32(const QuantizeParams& p, const CUtensorMap& tmap_x,
                                const CUtensorMap* tmap_r, int num_sms, cudaStream_t stream);
cudaError_t launch_quantize_grouped_f32(const QuantizeParams& p, const CUtensorMap& tmap_x,
                                        int num_sms, cudaStream_t stream);

// GEMM modes: dense; grouped by rows of A (each expert owns a range of A
// rows and its own B); grouped along K (each expert owns a 128-aligned
// range of the K columns of A and B and its own output matrix).
constexpr int kModeDense = 0;
constexpr int kModeGroupM = 1;
constexpr int kModeGroupK = 2;

struct GemmParams {
  int64_t m;           // rows of A and Y (grouped by rows: total rows; grouped
                       // along K: rows of A and of each output matrix)
  int64_t n;           // rows of each B (columns of Y)
  int64_t k;           // contraction length, a multiple of 16 (a final block of
                       // 16 is zero-filled past K; grouped along K: unused,
                       // each group's length comes from the offsets)
  int64_t lda;         // columns of the A code matrix (K-contiguous)
  int64_t ldb;         // columns of the B code matrix
  int32_t b_concat;    // grouped by rows: 1 = B is one [n, ldb] matrix with
                       // expert g's operand in columns [g*k, (g+1)*k)
  const uint8_t* sa;   // swizzled scales of A (grouped: per-group padded)
  const uint8_t* sb;   // swizzled scales of B (grouped: one matrix per group)
  void* y;
  int64_t ldy;         // elements
  int32_t y_fp32;      // 1: FP32 output, 0: BF16 output
  int32_t fa;          // tensor-core operand type code (E4M3 0, E5M2 1, E2M3 3, E3M2 4, E2M1 5)
  int32_t fb;
  const int32_t* offsets;  // grouped only: device int32[groups + 1]
  int32_t groups;          // 0 for the dense GEMM
  int32_t mode;            // kModeDense, kModeGroupM or kModeGroupK
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t band_m;          // m-tiles per raster band (dense), a multiple of 2
  const float* bias;       // fused epilogue: FP32 bias per output column, or nullptr
  int32_t act;             // fused epilogue: 0 none, 1 SiLU
  int32_t a_bits;          // bits of global storage per A / B code: 8, or 4 / 6 when
  int32_t b_bits;          // packed (the tensor copy counts the global bytes it reads)
};

// Block-pair GEMM (cta_group::2, 256 x 256 pair tiles), all three modes.
// tmap_a / tmap_b: codes, box 128 rows; tmap_sa / tmap_sb: the swizzled
// scale buffers viewed as uint32 [row_tiles][k_tiles][128], boxes of one
// (A) and two (B) 512-byte units.
cudaError_t launch_gemm_pair(const GemmParams& p, const CUtensorMap& tmap_a,
                             const CUtensorMap& tmap_b, const CUtensorMap& tmap_sa,
                             const CUtensorMap& tmap_sb, int num_sms, cudaStream_t stream);

struct NormParams {
  const void* block;     // [rows, cols] of the blocks' type, leading dimension ldb
  const void* residual;  // [rows, cols] of the stream's type, ldr
  const void* w_post;    // [cols] or nullptr
  const void* w_pre;     // [cols]
  const void* gate;      // [gates, cols] or nullptr
  void* res_out;         // stream's type, ldo
  void* y;               // blocks' type, ldy
  int64_t rows, cols, gates;
  int64_t ldb, ldr, ldo, ldy;
  int32_t c_fp32, s_fp32, w_fp32;  // 1: FP32, 0: BF16 (blocks, stream, weights and gate)
  float alpha, eps;
};

struct NormBackParams {
  const void* d_res;    // [rows, cols] of the stream's type, ldd, or nullptr
  const void* dy;       // blocks' type, lddy
  const void* block;    // blocks' type, ldb
  const void* res_out;  // stream's type, ldr
  const void* w_post;   // [cols] or nullptr
  const void* w_pre;    // [cols]
  const void* gate;     // [gates, cols] or nullptr
  void* d_block;        // blocks' type, lddb
  void* d_residual;     // stream's type, lddr
  float* d_w_post;      // [cols] or nullptr
  float* d_w_pre;       // [cols]
  float* d_gate;        // [gates, cols] or nullptr
  float* workspace;
  uint32_t* status;     // device status word
  uint64_t wait_limit_ns;
  int64_t rows, cols, gates;
  int64_t ldd, lddy, ldb, ldr, lddb, lddr;
  int32_t c_fp32, s_fp32, w_fp32;
  float alpha, eps;
};

size_t norm_backward_workspace(int64_t rows, int64_t cols, int64_t gates);
cudaError_t launch_norm_residual(const NormParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_residual_backward(const NormBackParams& p, int num_sms,
                                          cudaStream_t stream);

struct MoeFewParams {
  const void* x;         // bf16 [tokens, hidden], ldx
  const void* router;    // [experts, hidden]
  const uint8_t* gate_scales;
  const uint8_t* up_scales;
  const uint8_t* down_scales;
  void* y;               // bf16 [tokens, hidden], ldy
  int32_t* ids;          // [tokens, top_k]
  float* weights;        // [tokens, top_k]
  uint8_t* workspace;
  int64_t ldx, ldy;
  int32_t hidden, inter;
  int32_t tokens, experts, top_k, renormalize;
  int32_t router_fp32;
  int32_t type_gu, type_d;  // tensor-core operand type codes
  int32_t bits_gu, bits_d;  // bits of storage per code
  uint32_t* status;         // device status word
  uint64_t wait_limit_ns;
};

size_t moe_few_workspace(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                         int32_t top_k);
// tmap_gate, tmap_up: codes [experts * inter, hidden]; tmap_down: codes
// [experts * hidden, inter]; boxes of 128 elements x 128 rows.
cudaError_t launch_moe_few(const MoeFewParams& p, const CUtensorMap& tmap_gate,
                           const CUtensorMap& tmap_up, const CUtensorMap& tmap_down, int num_sms,
                           cudaStream_t stream);

// ------------------------------------------------------------------ heads' norms with rotation

struct RotateParams {
  const void* q;       // [tokens, q_heads, dim], strides of tokens and heads in elements
  const void* k;       // [tokens, k_heads, dim]
  const void* d_q;     // gradient: those of the outputs
  const void* d_k;
  const void* w_q;     // [dim]
  const void* w_k;
  const void* positions;      // int32 or int64 [tokens]
  const double* frequencies;  // [rotary / 2], radians per position
  void* out_q;         // outputs, or the gradients of q and k
  void* out_k;
  float* dw_q;         // gradient: [dim]
  float* dw_k;
  float* workspace;
  int64_t q_st, q_sh, k_st, k_sh, dq_st, dq_sh, dk_st, dk_sh, oq_st, oq_sh, ok_st, ok_sh;
  int32_t tokens, q_heads, k_heads, dim, rotary;
  int32_t interleaved, x_fp32, w_fp32, positions_64;
  int32_t chunks;      // every row of every array can be read in chunks of four channels
  // items of work, set by the launch
  int32_t tokens_per_item, heads_per_item, chunks_of_heads, items;
  float scale, eps;
};

size_t norm_rotate_backward_workspace(int64_t tokens, int64_t dim);
cudaError_t launch_norm_rotate(const RotateParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_rotate_backward(const RotateParams& p, int num_sms, cudaStream_t stream);
// (FP32 heads; called by the two above)
cudaError_t launch_norm_rotate_f32(const RotateParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_rotate_backward_f32(const RotateParams& p, int num_sms,
                                            cudaStream_t stream);

// ------------------------------------------------------------------ routing

struct RouteParams {
  const void* logits;        // [tokens, experts], ld
  const uint8_t* mask;       // [tokens] or nullptr: 0 = does not count
  int64_t ld;
  int32_t tokens, experts, top_k, renormalize, logits_fp32;
  int32_t vec;               // rows allow accesses of four logits
  int32_t* ids;              // [tokens, top_k]
  float* weights;            // [tokens, top_k]
  float* lse;                // [tokens]
  int32_t* counts;           // [experts]
  int32_t* offsets;          // [experts + 1]
  int32_t* order;            // [tokens * top_k]
  float* balance;            // [1]
  int32_t* workspace;
  int32_t blocks, tokens_per_block, vec_ids;  // set by the launch
  int32_t group;             // blocks whose pairs a block of the second kernel places
  // gradient
  const float* d_weights;    // [tokens, top_k] or nullptr
  const float* d_balance;    // [1] or nullptr
  const float* d_lse;        // [tokens] or nullptr
  const float* w_in;         // weights, ids, counts and lse of the forward pass
  const int32_t* ids_in;
  const int32_t* counts_in;
  const float* lse_in;
  void* d_logits;            // [tokens, experts] contiguous
  int32_t vec_out;
};

size_t route_workspace(int64_t tokens, int32_t experts);
cudaError_t launch_route(const RouteParams& p, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteParams& p, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------------ vocabulary loss

// The products of the vocabulary loss (vocab_loss.cu):
//   kStats   z = x W^T; per row and half tile of columns the running maximum
//            and sum of the softmax, and the label's logit
//   kGrad    dz = (d_loss + d_lse) exp(z - lse) - d_loss [label] of a piece of the
//            vocabulary, bf16 in units of the largest d_loss (few tokens: two terms)
//   kDx      dx = dz W of the piece, over `splits` parts of its columns
//   kDw      dW = dz^T x of the piece
enum class VocabProduct { kStats, kGrad, kDx, kDw };

struct VocabParams {
  int32_t m, n, k;         // rows and columns of the product, contraction length
  int32_t splits;          // parts of the contraction (kDx; else 1)
  int32_t steps;           // 64-element steps of a part
  int32_t tokens;
  const void* labels;      // int32 or int64 [tokens]
  int32_t labels_64;
  int64_t ignore_index;
  int32_t vocab;
  int32_t col0;            // kGrad: the piece's first column of the vocabulary
  float2* partial;         // kStats: [tokens][slots] (maximum in log2 units, sum)
  int32_t slots;
  float* z_label;          // kStats: [tokens]
  const float* lse;        // kGrad: [tokens]
  const float* d_loss;     // [tokens] or nullptr (zero)
  const float* d_lse;      // [tokens] or nullptr
  float* scale;            // what dz is held in units of, written by kGrad, read by kDx and
                           // kDw; nullptr (few tokens): 1
  int32_t y_fp32;          // kDx, kDw: type of the output
  int32_t add;             // kDx: 1 adds to the output (FP32)
  int32_t low_row;         // kDw of few tokens: first row of dz's low terms (else 0);
                           // the contraction's second step is theirs, with x again
  void* out;               // few tokens, kGrad, kDx: the output, ld_out elements a row
  int64_t ld_out;
  uint32_t* status;
  uint64_t wait_limit_ns;
};

// kStats or kGrad.  Boxes of the tensor maps of A and B: 64 elements x 128 rows; of
// the output (3-D: columns, rows, parts): 128 bytes x 32 rows; all with the 128-byte
// swizzle.
cudaError_t launch_vocab_logits(VocabProduct which, const VocabParams& p, const CUtensorMap& tmap_a,
                                const CUtensorMap& tmap_b, const CUtensorMap& tmap_y, int num_sms,
                                cudaStream_t stream);
// kDx and kDw of a piece in one launch; either may be absent.  Boxes: A of kDx 64
// elements x 128 rows, all other operands 64 x 64.
struct VocabGradient {
  const VocabParams* p;
  const CUtensorMap *a, *b, *y;
};
cudaError_t launch_vocab_gradients(const VocabGradient* dx, const VocabGradient* dw, int num_sms,
                                   cudaStream_t stream);
// kStats, kGrad and kDx for few tokens (vocab_few.cu), with rows of W (kDx: hidden
// channels) as the m rows of the product and tokens as its columns.  Boxes: A 64
// elements x 128 rows (kDx 64 x 64), B 64 elements x vocab_few_box(tokens) rows.
// p.m = vocabulary, columns of the piece, or hidden; slots = 4 vocab_few_blocks.  dz
// has two bf16 terms: rows [0, tokens) the high ones, [tokens, 2 tokens) the low ones.
constexpr int kVocabFewTokens = 64;
constexpr int kVocabFewBlocks = 152;  // one an SM
constexpr int vocab_few_box(int64_t tokens) { return tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64; }
int vocab_few_blocks(int64_t rows, int splits);
cudaError_t launch_vocab_few(VocabProduct which, const VocabParams& p, const CUtensorMap& tmap_a,
                             const CUtensorMap& tmap_b, cudaStream_t stream);
// loss and lse from the parts of every row.
cudaError_t launch_vocab_finish(const VocabParams& p, float* loss, float* lse, cudaStream_t stream);
// bf16 y[i] = sum over parts of parts[s][i], n elements (a multiple of 8).
cudaError_t launch_vocab_join(const float* parts, int32_t splits, int64_t n, void* y, int num_sms,
                              cudaStream_t stream);

// Clears the bits `bits` of the device status word (atomically, so bits
// set meanwhile by kernels on other streams survive).
cudaError_t launch_status_clear(uint32_t* status, uint32_t bits, cudaStream_t stream);

cudaError_t launch_wait_selftest(uint32_t* status, uint64_t limit_ns, cudaStream_t stream);

}  // namespace mx
