// mx_api.cu -- the C ABI (include/mx.h): argument validation, TMA tensor
// map encoding through the driver entry point, device status word, and
// kernel launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "kernels.h"
#include "mx.h"

namespace {

// The device status word (one per device, in this module's device memory).
__device__ uint32_t g_status_word;

constexpr int kMaxDevices = 64;
constexpr uint64_t kDefaultWaitNs = 2000000000ull;

struct DeviceState {
  bool ready = false;
  int device = 0;
  int num_sms = 0;
  uint32_t* status = nullptr;  // device address of g_status_word on this device
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::atomic<uint64_t> g_wait_ns{kDefaultWaitNs};
// Dense GEMMs walk their output tiles in bands of this many 128-row tiles
// (n-tiles outer inside a band), so a band of A stays in L2 while B streams.
constexpr int32_t kBandM = 32;

mx_status device_state(DeviceState** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MX_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState& st = g_dev[dev];
  if (!st.ready) {
    if (cudaDeviceGetAttribute(&st.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return MX_ERR_CUDA;
    void* addr = nullptr;
    if (cudaGetSymbolAddress(&addr, g_status_word) != cudaSuccess) return MX_ERR_CUDA;
    st.status = static_cast<uint32_t*>(addr);
    if (cudaMemset(st.status, 0, sizeof(uint32_t)) != cudaSuccess) return MX_ERR_CUDA;
    st.device = dev;
    st.ready = true;
  }
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return MX_ERR_CUDA;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  *out = &st;
  return MX_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every non-null pointer of the list points into device memory of device
// `dev` (memory of cudaMalloc or a memory pool on that device).  Host memory
// (pinned, mapped or unregistered), managed memory and the memory of other
// devices -- all reachable through unified addressing -- are refused, so
// the kernels and their tensor copies only ever read this GPU's own memory.
bool all_on_device(int dev, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs) {
    if (p == nullptr) continue;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
      (void)cudaGetLastError();  // clear the (non-sticky) error of the query
      return false;
    }
    if (a.type != cudaMemoryTypeDevice || a.device != dev) return false;
  }
  return true;
}

bool valid_fmt(mx_fmt f) { return f == MX_E4M3 || f == MX_E5M2; }

// GEMM operand formats: FP8 and the MXFP6 / MXFP4 element formats, the
// latter in container or packed storage.
bool valid_gemm_fmt(mx_fmt f) { return f >= MX_E4M3 && f <= MX_E2M1_PACKED; }

bool is_packed(mx_fmt f) { return f >= MX_E2M3_PACKED; }

// Code width in bits.
int code_bits(mx_fmt f) {
  switch (f) {
    case MX_E2M3: case MX_E3M2: case MX_E2M3_PACKED: case MX_E3M2_PACKED: return 6;
    case MX_E2M1: case MX_E2M1_PACKED: return 4;
    default: return 8;
  }
}

// Operand type code of tcgen05.mma.kind::mxf8f6f4 (instruction descriptor
// bits 7-9 / 10-12): E4M3 0, E5M2 1, E2M3 3, E3M2 4, E2M1 5 (either storage).
int32_t mma_type_code(mx_fmt f) {
  switch (f) {
    case MX_E5M2: return 1;
    case MX_E2M3: case MX_E2M3_PACKED: return 3;
    case MX_E3M2: case MX_E3M2_PACKED: return 4;
    case MX_E2M1: case MX_E2M1_PACKED: return 5;
    default: return 0;
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 2-D uint8 tensor map over a [rows, inner] row-major matrix with row stride
// `stride` bytes, tile box {128 bytes, box_rows}, 128-byte swizzle, zero
// fill outside the matrix.
mx_status encode_codes_map(CUtensorMap* map, const void* base, int64_t inner, int64_t rows,
                           int64_t stride, uint32_t box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  cuuint32_t box[2] = {128u, box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// 2-D bf16 tensor map over x[rows, cols] (leading dimension ldx elements),
// box 64 columns x 128 rows (128-byte rows, two boxes per 128 x 128 tile),
// 128-byte swizzle, zero fill outside the matrix.
mx_status encode_bf16_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                          int64_t ldx) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldx * 2)};
  cuuint32_t box[2] = {64u, 128u};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// 2-D tensor map over an FP32 [rows, cols] matrix with leading dimension
// ldx: box 32 columns x 128 rows (128-byte rows, two boxes per 128 x 64
// tile), 128-byte swizzle, zero fill outside the matrix.
mx_status encode_f32_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                         int64_t ldx) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldx * 4)};
  cuuint32_t box[2] = {32u, 128u};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// 2-D tensor map over packed 6- or 4-bit codes [rows, inner elements] with
// row stride `stride` bytes, read with the unpacking element type: each run
// of 16 codes lands in 16 bytes of shared memory (the container layout the
// MMA reads), so the shared-memory tile equals that of a container-layout
// operand.  Box {128 elements, box_rows}, 128-byte swizzle, zero fill.
mx_status encode_packed_map(CUtensorMap* map, const void* base, int64_t inner, int64_t rows,
                            int64_t stride, uint32_t box_rows, int bits) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  cuuint32_t box[2] = {128u, box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapDataType type =
      bits == 4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_16U6_ALIGN16B;
  CUresult r = g_encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// Tensor map of a GEMM code operand [rows, ld elements] in its storage.
mx_status encode_operand_map(CUtensorMap* map, const void* base, mx_fmt f, int64_t ld,
                             int64_t rows) {
  if (is_packed(f))
    return encode_packed_map(map, base, ld, rows, ld * code_bits(f) / 8, 128, code_bits(f));
  return encode_codes_map(map, base, ld, rows, ld, 128);
}

// The swizzled scale buffer of a [rows, k] operand viewed as uint32
// [ceil(rows/128)][ceil(k/128)][128] (one 512-byte unit per 128-row x
// 128-K tile); box of `units` consecutive row tiles at one K tile.
mx_status encode_scale_map(CUtensorMap* map, const void* base, int64_t rows, int64_t k,
                           uint32_t units) {
  const int64_t row_tiles = ceil_div(rows, 128);
  const int64_t k_tiles = ceil_div(k, 128);
  cuuint64_t dims[3] = {128u, static_cast<cuuint64_t>(k_tiles),
                        static_cast<cuuint64_t>(row_tiles)};
  cuuint64_t strides[2] = {512u, static_cast<cuuint64_t>(512 * k_tiles)};
  cuuint32_t box[3] = {128u, 1u, units};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// Operand geometry of one GEMM launch: A codes [m, lda] (grouped along K:
// [m, lda] shared by all groups), B codes [b_rows, ldb]; scales swizzled
// over the same shapes.
struct GemmShape {
  int64_t m, n, k;
  int64_t lda, ldb, b_rows;
  int32_t groups = 0;
  const int32_t* d_offsets = nullptr;
  int32_t mode = mx::kModeDense;
  int32_t b_concat = 0;
};

mx_status gemm_common(const GemmShape& g, const uint8_t* a, const uint8_t* sa, mx_fmt fa,
                      const uint8_t* b, const uint8_t* sb, mx_fmt fb, void* y, mx_dtype y_dtype,
                      int64_t ldy, cudaStream_t stream, const float* bias = nullptr,
                      int32_t act = 0) {
  const int64_t m = g.m, n = g.n, k = g.k;
  if (!a || !sa || !b || !sb || !y) return MX_ERR_INVALID_ARG;
  if (m < 0 || n <= 0 || k < 0 || n % 8 != 0 || ldy < n) return MX_ERR_INVALID_ARG;
  // grouped along K, k is the token total that the offsets split; else
  // whole 16-element runs (a final partial block of 16 is zero-padded)
  if (g.mode != mx::kModeGroupK && (k < 16 || k % 16 != 0)) return MX_ERR_INVALID_ARG;
  if (!valid_gemm_fmt(fa) || !valid_gemm_fmt(fb)) return MX_ERR_INVALID_ARG;
  if (y_dtype != MX_BF16 && y_dtype != MX_FP32) return MX_ERR_INVALID_ARG;
  if (m > INT32_MAX || g.b_rows > INT32_MAX || k > INT32_MAX || g.lda > INT32_MAX ||
      g.ldb > INT32_MAX)
    return MX_ERR_UNSUPPORTED;
  // the kernels index their 256x256 work units in 32 bits
  {
    const int64_t m_tiles = ceil_div(m, 128);
    int64_t units = g.mode == mx::kModeGroupM ? (m_tiles + g.groups + 1) / 2 + g.groups
                                              : (m_tiles + 1) / 2;
    units *= ceil_div(n, 256);
    if (g.mode == mx::kModeGroupK) units *= g.groups;
    if (units > INT32_MAX) return MX_ERR_UNSUPPORTED;
  }
  const int64_t elt = y_dtype == MX_FP32 ? 4 : 2;
  if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(y) ||
      (ldy * elt) % 16 != 0 || g.lda % 16 != 0 || g.ldb % 16 != 0)
    return MX_ERR_MISALIGNED;
  // packed operands: whole 128-element K tiles (the unpacking tensor copy
  // reads rows of a multiple of 128 elements) and 32-byte aligned rows
  if ((is_packed(fa) && (g.lda % 128 != 0 || (g.mode != mx::kModeGroupK && k % 128 != 0))) ||
      (is_packed(fb) && (g.ldb % 128 != 0 || (g.mode != mx::kModeGroupK && k % 128 != 0))))
    return MX_ERR_INVALID_ARG;
  if ((is_packed(fa) && (reinterpret_cast<uintptr_t>(a) & 31u) != 0) ||
      (is_packed(fb) && (reinterpret_cast<uintptr_t>(b) & 31u) != 0))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  mx_status s = device_state(&st);
  if (s != MX_OK) return s;
  if (m == 0) return MX_OK;
  if (!all_on_device(st->device, {a, sa, b, sb, y, bias, g.d_offsets})) return MX_ERR_INVALID_ARG;

  mx::GemmParams p{};
  p.m = m;
  p.n = n;
  p.k = k;
  p.lda = g.lda;
  p.ldb = g.ldb;
  p.b_concat = g.b_concat;
  p.sa = sa;
  p.sb = sb;
  p.y = y;
  p.ldy = ldy;
  p.y_fp32 = y_dtype == MX_FP32 ? 1 : 0;
  p.fa = mma_type_code(fa);
  p.fb = mma_type_code(fb);
  p.offsets = g.d_offsets;
  p.groups = g.groups;
  p.mode = g.mode;
  p.status = st->status;
  p.wait_limit_ns = g_wait_ns.load(std::memory_order_relaxed);
  p.bias = bias;
  p.act = act;
  p.band_m = kBandM;
  p.a_bits = is_packed(fa) ? code_bits(fa) : 8;
  p.b_bits = is_packed(fb) ? code_bits(fb) : 8;

  // Block pairs (cta_group::2, 256x256 pair tiles): each block loads 128
  // rows of A and 128 of the 256 rows of the B tile; the scale buffers are
  // viewed as grids of 512-byte units, A's with the per-group padded row
  // bound when grouped by rows.
  CUtensorMap ta, tb, tsa, tsb;
  const int64_t a_scale_rows = g.mode == mx::kModeGroupM ? (ceil_div(m, 128) + g.groups) * 128 : m;
  if ((s = encode_operand_map(&ta, a, fa, g.lda, m)) != MX_OK) return s;
  if ((s = encode_operand_map(&tb, b, fb, g.ldb, g.b_rows)) != MX_OK) return s;
  if ((s = encode_scale_map(&tsa, sa, a_scale_rows, g.lda, 1)) != MX_OK) return s;
  if ((s = encode_scale_map(&tsb, sb, g.b_rows, g.ldb, 2)) != MX_OK) return s;
  const cudaError_t err = mx::launch_gemm_pair(p, ta, tb, tsa, tsb, st->num_sms, stream);
  if (err == cudaErrorNotSupported) return MX_ERR_UNSUPPORTED;
  return err == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

GemmShape dense_shape(int64_t m, int64_t n, int64_t k) {
  GemmShape g;
  g.m = m;
  g.n = n;
  g.k = k;
  g.lda = k;
  g.ldb = k;
  g.b_rows = n;
  return g;
}

}  // namespace

extern "C" {

size_t mx_scale_bytes(int64_t rows, int64_t k) {
  if (rows < 0 || k < 0 || k % 16 != 0) return 0;
  return static_cast<size_t>(ceil_div(rows, 128) * 128 * ceil_div(ceil_div(k, 32), 4) * 4);
}

size_t mx_grouped_scale_bytes(int64_t total_rows, int32_t groups, int64_t k) {
  if (total_rows < 0 || groups < 0 || k < 0 || k % 16 != 0) return 0;
  return static_cast<size_t>((ceil_div(total_rows, 128) + groups) * 128 * ceil_div(k, 128) * 4);
}

}  // extern "C"

namespace {

mx_status quantize_common(const void* x, mx_dtype x_dtype, int64_t rows, int64_t cols,
                          int64_t ldx, const uint16_t* rbits, int64_t ldr, mx_fmt fmt,
                          mx_axis axis, mx_scale_rule rule, uint8_t* q_row, uint8_t* s_row,
                          uint8_t* q_col, uint8_t* s_col, cudaStream_t stream) {
  if (x_dtype != MX_BF16 && x_dtype != MX_FP32) return MX_ERR_INVALID_ARG;
  const bool f32 = x_dtype == MX_FP32;
  if (!valid_gemm_fmt(fmt) || (rule != MX_SCALE_FLOOR && rule != MX_SCALE_CEIL))
    return MX_ERR_INVALID_ARG;
  if (axis != MX_ROWWISE && axis != MX_COLWISE && axis != MX_BOTH) return MX_ERR_INVALID_ARG;
  const bool row = axis & MX_ROWWISE;
  const bool col = axis & MX_COLWISE;
  if (!x || (row && (!q_row || !s_row)) || (col && (!q_col || !s_col))) return MX_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0 || ldx < cols || cols % 8 != 0) return MX_ERR_INVALID_ARG;
  if (rbits && ldr < cols) return MX_ERR_INVALID_ARG;
  // the blocked axis: whole 16-element runs (16-byte code rows; a final
  // partial block of 16 is zero-padded), whole blocks in packed storage
  const int64_t k_unit = is_packed(fmt) ? 32 : 16;
  if (row && cols % k_unit != 0) return MX_ERR_INVALID_ARG;
  if (col && rows % k_unit != 0) return MX_ERR_INVALID_ARG;
  if (ceil_div(cols, 128) > 65535) return MX_ERR_UNSUPPORTED;
  // the kernels number their tiles (128 rows x 128 bf16 or 64 FP32 columns) in 32 bits
  const int64_t col_tiles = ceil_div(cols, f32 ? 64 : 128);
  if (cols > 0 && ceil_div(rows, 128) > static_cast<int64_t>(UINT32_MAX) / col_tiles)
    return MX_ERR_UNSUPPORTED;
  // rows of x start on 16-byte boundaries
  if (!aligned16(x) || ldx % (f32 ? 4 : 8) != 0) return MX_ERR_MISALIGNED;
  if (rbits && (!aligned16(rbits) || ldr % 8 != 0)) return MX_ERR_MISALIGNED;
  if ((row && (!aligned16(q_row) || !aligned16(s_row))) ||
      (col && (!aligned16(q_col) || !aligned16(s_col))))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  mx_status s = device_state(&st);
  if (s != MX_OK) return s;
  mx::QuantizeParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.q_row = row ? q_row : nullptr;
  p.s_row = row ? s_row : nullptr;
  p.q_col = col ? q_col : nullptr;
  p.s_col = col ? s_col : nullptr;
  p.fmt = fmt;
  p.rule = rule;
  p.status = st->status;
  p.wait_limit_ns = g_wait_ns.load(std::memory_order_relaxed);
  p.ldq_col = rows;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!all_on_device(st->device, {x, rbits, p.q_row, p.s_row, p.q_col, p.s_col}))
    return MX_ERR_INVALID_ARG;
  CUtensorMap tmap, tmap_r;
  s = f32 ? encode_f32_map(&tmap, x, cols, rows, ldx) : encode_bf16_map(&tmap, x, cols, rows, ldx);
  if (s != MX_OK) return s;
  // the random integers are 16-bit like bf16: the bf16 box geometry
  if (rbits && (s = encode_bf16_map(&tmap_r, rbits, cols, rows, ldr)) != MX_OK) return s;
  const CUtensorMap* tr = rbits ? &tmap_r : nullptr;
  const cudaError_t err = f32 ? mx::launch_quantize_f32(p, tmap, tr, st->num_sms, stream)
                              : mx::launch_quantize(p, tmap, tr, st->num_sms, stream);
  return err == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

}  // namespace

extern "C" {

mx_status mx_quantize(const void* x, mx_dtype x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                      mx_fmt fmt, mx_axis axis, mx_scale_rule rule, uint8_t* q_row,
                      uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, cudaStream_t stream) {
  return quantize_common(x, x_dtype, rows, cols, ldx, nullptr, 0, fmt, axis, rule, q_row, s_row,
                         q_col, s_col, stream);
}

mx_status mx_quantize_sr(const void* x, mx_dtype x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                         const uint16_t* rbits, int64_t ldr, mx_fmt fmt, mx_axis axis,
                         mx_scale_rule rule, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                         uint8_t* s_col, cudaStream_t stream) {
  if (!rbits) return MX_ERR_INVALID_ARG;
  return quantize_common(x, x_dtype, rows, cols, ldx, rbits, ldr, fmt, axis, rule, q_row, s_row,
                         q_col, s_col, stream);
}

mx_status mx_quantize_grouped(const void* x, mx_dtype x_dtype, int64_t total_rows, int64_t cols,
                              int64_t ldx, mx_fmt fmt, mx_scale_rule rule, int32_t groups,
                              const int32_t* d_offsets, uint8_t* q, uint8_t* s,
                              cudaStream_t stream) {
  if (!q || !s) return MX_ERR_INVALID_ARG;
  return mx_quantize_grouped_ex(x, x_dtype, total_rows, cols, ldx, fmt, MX_ROWWISE, rule, groups,
                                d_offsets, q, s, nullptr, 0, nullptr, stream);
}

int64_t mx_grouped_cols_capacity(int64_t total_rows, int32_t groups) {
  if (total_rows < 0 || groups < 0) return 0;
  return (total_rows / 128 + groups) * 128;
}

mx_status mx_quantize_grouped_ex(const void* x, mx_dtype x_dtype, int64_t total_rows,
                                 int64_t cols, int64_t ldx, mx_fmt fmt, mx_axis axis,
                                 mx_scale_rule rule, int32_t groups, const int32_t* d_offsets,
                                 uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, int64_t ldq_col,
                                 uint8_t* s_col, cudaStream_t stream) {
  if (x_dtype != MX_BF16 && x_dtype != MX_FP32) return MX_ERR_INVALID_ARG;
  const bool f32 = x_dtype == MX_FP32;
  if (!valid_gemm_fmt(fmt) || (rule != MX_SCALE_FLOOR && rule != MX_SCALE_CEIL))
    return MX_ERR_INVALID_ARG;
  if (!valid_fmt(fmt)) return MX_ERR_UNSUPPORTED;  // grouped: FP8 codes
  if (axis != MX_ROWWISE && axis != MX_COLWISE && axis != MX_BOTH) return MX_ERR_INVALID_ARG;
  const bool row = axis & MX_ROWWISE;
  const bool col = axis & MX_COLWISE;
  if (!x || !d_offsets || (row && (!q_row || !s_row)) || (col && (!q_col || !s_col)))
    return MX_ERR_INVALID_ARG;
  if (groups < 1 || groups > 1000) return MX_ERR_INVALID_ARG;
  if (total_rows < 0 || total_rows > INT32_MAX || cols < 0 || ldx < cols || cols % 8 != 0)
    return MX_ERR_INVALID_ARG;
  if (row && cols % 16 != 0) return MX_ERR_INVALID_ARG;
  if (col && (ldq_col <= 0 || ldq_col % 128 != 0)) return MX_ERR_INVALID_ARG;
  if (ceil_div(cols, 128) > 65535) return MX_ERR_UNSUPPORTED;
  // the columnwise pass numbers its tiles (128 rows x 128 bf16 or 64 FP32
  // columns) in 32 bits
  if (col && (ceil_div(total_rows, 128) + groups) * ceil_div(cols, f32 ? 64 : 128) > UINT32_MAX)
    return MX_ERR_UNSUPPORTED;
  if (!aligned16(x) || ldx % (f32 ? 4 : 8) != 0) return MX_ERR_MISALIGNED;
  if ((row && (!aligned16(q_row) || !aligned16(s_row))) ||
      (col && (!aligned16(q_col) || !aligned16(s_col))))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  mx_status status = device_state(&st);
  if (status != MX_OK) return status;
  mx::QuantizeParams p{};
  p.x = x;
  p.rows = total_rows;
  p.cols = cols;
  p.ldx = ldx;
  p.q_row = row ? q_row : nullptr;
  p.s_row = row ? s_row : nullptr;
  p.q_col = col ? q_col : nullptr;
  p.s_col = col ? s_col : nullptr;
  p.ldq_col = col ? ldq_col : 0;
  p.fmt = fmt;
  p.rule = rule;
  p.offsets = d_offsets;
  p.groups = groups;
  p.status = st->status;
  p.wait_limit_ns = g_wait_ns.load(std::memory_order_relaxed);
  if (cols == 0) return MX_OK;
  if (!all_on_device(st->device, {x, d_offsets, p.q_row, p.s_row, p.q_col, p.s_col}))
    return MX_ERR_INVALID_ARG;
  CUtensorMap tmap;
  // an empty token set still needs a valid map (1 row) for the offsets check
  const int64_t map_rows = total_rows > 0 ? total_rows : 1;
  status = f32 ? encode_f32_map(&tmap, x, cols, map_rows, ldx)
               : encode_bf16_map(&tmap, x, cols, map_rows, ldx);
  if (status != MX_OK) return status;
  const cudaError_t err = f32 ? mx::launch_quantize_grouped_f32(p, tmap, st->num_sms, stream)
                              : mx::launch_quantize_grouped(p, tmap, st->num_sms, stream);
  return err == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

mx_status mx_gemm(int64_t m, int64_t n, int64_t k, const uint8_t* a, const uint8_t* sa, mx_fmt fa,
                  const uint8_t* b, const uint8_t* sb, mx_fmt fb, void* y, mx_dtype y_dtype,
                  int64_t ldy, cudaStream_t stream) {
  return gemm_common(dense_shape(m, n, k), a, sa, fa, b, sb, fb, y, y_dtype, ldy, stream);
}

mx_status mx_gemm_bias_act(int64_t m, int64_t n, int64_t k, const uint8_t* a, const uint8_t* sa,
                           mx_fmt fa, const uint8_t* b, const uint8_t* sb, mx_fmt fb,
                           const float* bias, mx_activation act, void* y, mx_dtype y_dtype,
                           int64_t ldy, cudaStream_t stream) {
  if (act != MX_ACT_NONE && act != MX_ACT_SILU) return MX_ERR_INVALID_ARG;
  if (bias != nullptr && !aligned16(bias)) return MX_ERR_MISALIGNED;
  return gemm_common(dense_shape(m, n, k), a, sa, fa, b, sb, fb, y, y_dtype, ldy, stream, bias,
                     act);
}

mx_status mx_grouped_gemm(int32_t groups, const int32_t* d_offsets, int64_t total_m, int64_t n,
                          int64_t k, const uint8_t* a, const uint8_t* sa, mx_fmt fa,
                          const uint8_t* b, const uint8_t* sb, mx_fmt fb, void* y,
                          mx_dtype y_dtype, cudaStream_t stream) {
  if (groups < 1 || groups > 1000 || !d_offsets) return MX_ERR_INVALID_ARG;
  if (n % 128 != 0) return MX_ERR_INVALID_ARG;
  GemmShape g = dense_shape(total_m, n, k);
  g.b_rows = static_cast<int64_t>(groups) * n;
  g.groups = groups;
  g.d_offsets = d_offsets;
  g.mode = mx::kModeGroupM;
  return gemm_common(g, a, sa, fa, b, sb, fb, y, y_dtype, n, stream);
}

mx_status mx_grouped_gemm_bcat(int32_t groups, const int32_t* d_offsets, int64_t total_m,
                               int64_t n, int64_t k, const uint8_t* a, const uint8_t* sa,
                               mx_fmt fa, const uint8_t* b, int64_t ldb, const uint8_t* sb,
                               mx_fmt fb, void* y, mx_dtype y_dtype, cudaStream_t stream) {
  if (groups < 1 || groups > 1000 || !d_offsets) return MX_ERR_INVALID_ARG;
  if (k <= 0 || k % 128 != 0 || ldb < static_cast<int64_t>(groups) * k) return MX_ERR_INVALID_ARG;
  GemmShape g = dense_shape(total_m, n, k);
  g.ldb = ldb;
  g.b_rows = n;
  g.groups = groups;
  g.d_offsets = d_offsets;
  g.mode = mx::kModeGroupM;
  g.b_concat = 1;
  return gemm_common(g, a, sa, fa, b, sb, fb, y, y_dtype, n, stream);
}

mx_status mx_grouped_gemm_wgrad(int32_t groups, const int32_t* d_offsets, int64_t total_tokens,
                                int64_t m, int64_t n, int64_t ldk, const uint8_t* a,
                                const uint8_t* sa, mx_fmt fa, const uint8_t* b,
                                const uint8_t* sb, mx_fmt fb, void* y, mx_dtype y_dtype,
                                cudaStream_t stream) {
  if (groups < 1 || groups > 1000 || !d_offsets) return MX_ERR_INVALID_ARG;
  if (total_tokens < 0 || total_tokens > INT32_MAX || ldk <= 0 || ldk % 128 != 0)
    return MX_ERR_INVALID_ARG;
  // k carries the token total for the device-side offsets check; each
  // group contracts its own share of the tokens
  GemmShape g;
  g.m = m;
  g.n = n;
  g.k = total_tokens;
  g.lda = ldk;
  g.ldb = ldk;
  g.b_rows = n;
  g.groups = groups;
  g.d_offsets = d_offsets;
  g.mode = mx::kModeGroupK;
  return gemm_common(g, a, sa, fa, b, sb, fb, y, y_dtype, n, stream);
}

}  // extern "C"

namespace {

bool valid_dtype(mx_dtype d) { return d == MX_BF16 || d == MX_FP32; }

bool aligned_elt(const void* p, mx_dtype d) {
  return (reinterpret_cast<uintptr_t>(p) & (d == MX_FP32 ? 3u : 1u)) == 0;
}

constexpr int64_t kNormMaxCols = 16384;

// Checks shared by the norm and its gradient.
mx_status norm_check(int64_t rows, int64_t cols, mx_dtype c_dtype, mx_dtype s_dtype,
                     mx_dtype w_dtype, const void* gate, int64_t gates, float eps) {
  if (!valid_dtype(c_dtype) || !valid_dtype(s_dtype) || !valid_dtype(w_dtype))
    return MX_ERR_INVALID_ARG;
  if (rows < 0 || cols < 1 || !(eps >= 0.f)) return MX_ERR_INVALID_ARG;
  if (gate && (gates < 1 || rows % gates != 0)) return MX_ERR_INVALID_ARG;
  if (cols > kNormMaxCols || rows > INT32_MAX) return MX_ERR_UNSUPPORTED;
  if (c_dtype == MX_FP32 && s_dtype == MX_BF16) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

bool moe_few_sizes_ok(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                      int32_t top_k) {
  return tokens >= 0 && tokens <= 64 && hidden >= 16 && hidden <= 65536 && hidden % 16 == 0 &&
         inter >= 16 && inter <= 65536 && inter % 16 == 0 && experts >= 1 && experts <= 512 &&
         top_k >= 1 && top_k <= experts && top_k <= 32;
}

}  // namespace

extern "C" {

mx_status mx_norm_residual(int64_t rows, int64_t cols, const void* block, int64_t ldb,
                           mx_dtype c_dtype, const void* residual, int64_t ldr, mx_dtype s_dtype,
                           const void* w_post, const void* w_pre, const void* gate, int64_t gates,
                           mx_dtype w_dtype, float alpha, float eps, void* res_out, int64_t ldo,
                           void* y, int64_t ldy, cudaStream_t stream) {
  if (!block || !residual || !w_pre || !res_out || !y) return MX_ERR_INVALID_ARG;
  mx_status s = norm_check(rows, cols, c_dtype, s_dtype, w_dtype, gate, gates, eps);
  if (s != MX_OK) return s;
  if (ldb < cols || ldr < cols || ldo < cols || ldy < cols) return MX_ERR_INVALID_ARG;
  if (!aligned_elt(block, c_dtype) || !aligned_elt(y, c_dtype) ||
      !aligned_elt(residual, s_dtype) || !aligned_elt(res_out, s_dtype) ||
      !aligned_elt(w_post, w_dtype) || !aligned_elt(w_pre, w_dtype) || !aligned_elt(gate, w_dtype))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (rows == 0) return MX_OK;
  if (!all_on_device(st->device, {block, residual, w_post, w_pre, gate, res_out, y}))
    return MX_ERR_INVALID_ARG;
  mx::NormParams p{};
  p.block = block;
  p.residual = residual;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.gate = gate;
  p.res_out = res_out;
  p.y = y;
  p.rows = rows;
  p.cols = cols;
  p.gates = gate ? gates : 0;
  p.ldb = ldb;
  p.ldr = ldr;
  p.ldo = ldo;
  p.ldy = ldy;
  p.c_fp32 = c_dtype == MX_FP32;
  p.s_fp32 = s_dtype == MX_FP32;
  p.w_fp32 = w_dtype == MX_FP32;
  p.alpha = alpha;
  p.eps = eps;
  return mx::launch_norm_residual(p, st->num_sms, stream) == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

size_t mx_norm_residual_backward_workspace(int64_t rows, int64_t cols, int64_t gates) {
  if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > kNormMaxCols || gates < 0 ||
      (gates > 0 && rows % gates != 0))
    return 0;
  return mx::norm_backward_workspace(rows, cols, gates);
}

mx_status mx_norm_residual_backward(int64_t rows, int64_t cols, const void* d_res, int64_t ldd,
                                    const void* dy, int64_t lddy, const void* block, int64_t ldb,
                                    mx_dtype c_dtype, const void* res_out, int64_t ldr,
                                    mx_dtype s_dtype, const void* w_post, const void* w_pre,
                                    const void* gate, int64_t gates, mx_dtype w_dtype, float alpha,
                                    float eps, void* d_block, int64_t lddb, void* d_residual,
                                    int64_t lddr, float* d_w_post, float* d_w_pre, float* d_gate,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!dy || !block || !res_out || !w_pre || !d_block || !d_residual || !d_w_pre)
    return MX_ERR_INVALID_ARG;
  if ((w_post == nullptr) != (d_w_post == nullptr) || (gate == nullptr) != (d_gate == nullptr))
    return MX_ERR_INVALID_ARG;
  mx_status s = norm_check(rows, cols, c_dtype, s_dtype, w_dtype, gate, gates, eps);
  if (s != MX_OK) return s;
  if ((d_res && ldd < cols) || lddy < cols || ldb < cols || ldr < cols || lddb < cols ||
      lddr < cols)
    return MX_ERR_INVALID_ARG;
  const size_t need = mx::norm_backward_workspace(rows, cols, gate ? gates : 0);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MX_ERR_INVALID_ARG;
  if (!aligned_elt(d_res, s_dtype) || !aligned_elt(dy, c_dtype) || !aligned_elt(block, c_dtype) ||
      !aligned_elt(res_out, s_dtype) || !aligned_elt(w_post, w_dtype) ||
      !aligned_elt(w_pre, w_dtype) || !aligned_elt(gate, w_dtype) ||
      !aligned_elt(d_block, c_dtype) || !aligned_elt(d_residual, s_dtype) ||
      !aligned_elt(d_w_post, MX_FP32) || !aligned_elt(d_w_pre, MX_FP32) ||
      !aligned_elt(d_gate, MX_FP32) || !aligned16(workspace))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (!all_on_device(st->device, {d_w_post, d_w_pre, d_gate, w_post, w_pre, gate}))
    return MX_ERR_INVALID_ARG;
  if (rows > 0 &&
      !all_on_device(st->device, {d_res, dy, block, res_out, d_block, d_residual, workspace}))
    return MX_ERR_INVALID_ARG;
  mx::NormBackParams p{};
  p.d_res = d_res;
  p.dy = dy;
  p.block = block;
  p.res_out = res_out;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.gate = gate;
  p.d_block = d_block;
  p.d_residual = d_residual;
  p.d_w_post = d_w_post;
  p.d_w_pre = d_w_pre;
  p.d_gate = d_gate;
  p.workspace = static_cast<float*>(workspace);
  p.status = st->status;
  p.wait_limit_ns = g_wait_ns.load(std::memory_order_relaxed);
  p.rows = rows;
  p.cols = cols;
  p.gates = gate ? gates : 0;
  p.ldd = ldd;
  p.lddy = lddy;
  p.ldb = ldb;
  p.ldr = ldr;
  p.lddb = lddb;
  p.lddr = lddr;
  p.c_fp32 = c_dtype == MX_FP32;
  p.s_fp32 = s_dtype == MX_FP32;
  p.w_fp32 = w_dtype == MX_FP32;
  p.alpha = alpha;
  p.eps = eps;
  return mx::launch_norm_residual_backward(p, st->num_sms, stream) == cudaSuccess ? MX_OK
                                                                                   : MX_ERR_CUDA;
}

size_t mx_moe_few_tokens_workspace(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                                   int32_t top_k) {
  if (!moe_few_sizes_ok(tokens, hidden, inter, experts, top_k)) return 0;
  return mx::moe_few_workspace(tokens, hidden, inter, experts, top_k);
}

mx_status mx_moe_few_tokens(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                            int32_t top_k, const void* x, int64_t ldx, const void* router,
                            mx_dtype router_dtype, const uint8_t* gate, const uint8_t* gate_scales,
                            const uint8_t* up, const uint8_t* up_scales, mx_fmt fmt_gu,
                            const uint8_t* down, const uint8_t* down_scales, mx_fmt fmt_d,
                            int32_t renormalize, void* y, int64_t ldy, int32_t* ids,
                            float* weights, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  if (!x || !router || !gate || !gate_scales || !up || !up_scales || !down || !down_scales || !y ||
      !ids || !weights)
    return MX_ERR_INVALID_ARG;
  if (!valid_dtype(router_dtype) || !valid_gemm_fmt(fmt_gu) || !valid_gemm_fmt(fmt_d))
    return MX_ERR_INVALID_ARG;
  if (tokens > 64) return MX_ERR_UNSUPPORTED;
  if (!moe_few_sizes_ok(tokens, hidden, inter, experts, top_k)) return MX_ERR_INVALID_ARG;
  if (ldx < hidden || ldy < hidden) return MX_ERR_INVALID_ARG;
  for (mx_fmt f : {fmt_gu, fmt_d})
    if (!valid_fmt(f) && f != MX_E2M1_PACKED) return MX_ERR_UNSUPPORTED;
  // packed operands: whole 128-element K tiles, as for the GEMMs
  if ((is_packed(fmt_gu) && hidden % 128 != 0) || (is_packed(fmt_d) && inter % 128 != 0))
    return MX_ERR_INVALID_ARG;
  const size_t need = mx::moe_few_workspace(tokens, hidden, inter, experts, top_k);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MX_ERR_INVALID_ARG;
  if (!aligned16(x) || ldx % 8 != 0 || !aligned16(router) || !aligned16(gate) ||
      !aligned16(gate_scales) || !aligned16(up) || !aligned16(up_scales) || !aligned16(down) ||
      !aligned16(down_scales) || !aligned16(y) || ldy % 8 != 0 || !aligned16(workspace) ||
      !aligned_elt(ids, MX_FP32) || !aligned_elt(weights, MX_FP32))
    return MX_ERR_MISALIGNED;
  if ((is_packed(fmt_gu) && ((reinterpret_cast<uintptr_t>(gate) & 31u) != 0 ||
                             (reinterpret_cast<uintptr_t>(up) & 31u) != 0)) ||
      (is_packed(fmt_d) && (reinterpret_cast<uintptr_t>(down) & 31u) != 0))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  mx_status s = device_state(&st);
  if (s != MX_OK) return s;
  if (tokens == 0) return MX_OK;
  if (!all_on_device(st->device, {x, router, gate, gate_scales, up, up_scales, down, down_scales,
                                  y, ids, weights, workspace}))
    return MX_ERR_INVALID_ARG;
  mx::MoeFewParams p{};
  p.x = x;
  p.router = router;
  p.gate_scales = gate_scales;
  p.up_scales = up_scales;
  p.down_scales = down_scales;
  p.y = y;
  p.ids = ids;
  p.weights = weights;
  p.workspace = static_cast<uint8_t*>(workspace);
  p.ldx = ldx;
  p.ldy = ldy;
  p.hidden = static_cast<int32_t>(hidden);
  p.inter = static_cast<int32_t>(inter);
  p.tokens = tokens;
  p.experts = experts;
  p.top_k = top_k;
  p.renormalize = renormalize;
  p.router_fp32 = router_dtype == MX_FP32;
  p.type_gu = mma_type_code(fmt_gu);
  p.type_d = mma_type_code(fmt_d);
  p.bits_gu = is_packed(fmt_gu) ? code_bits(fmt_gu) : 8;
  p.bits_d = is_packed(fmt_d) ? code_bits(fmt_d) : 8;
  p.status = st->status;
  p.wait_limit_ns = g_wait_ns.load(std::memory_order_relaxed);
  CUtensorMap tg, tu, td;
  if ((s = encode_operand_map(&tg, gate, fmt_gu, hidden, experts * inter)) != MX_OK) return s;
  if ((s = encode_operand_map(&tu, up, fmt_gu, hidden, experts * inter)) != MX_OK) return s;
  if ((s = encode_operand_map(&td, down, fmt_d, inter, experts * hidden)) != MX_OK) return s;
  return mx::launch_moe_few(p, tg, tu, td, st->num_sms, stream) == cudaSuccess ? MX_OK
                                                                                : MX_ERR_CUDA;
}

}  // extern "C"

namespace {

// Checks of the heads' norms with rotation that both directions share.
mx_status rotate_check(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim,
                       int64_t rotary, mx_dtype x_dtype, mx_dtype w_dtype, int32_t position_bits,
                       float eps) {
  if (!valid_dtype(x_dtype) || !valid_dtype(w_dtype)) return MX_ERR_INVALID_ARG;
  if (tokens < 0 || q_heads < 1 || k_heads < 1 || dim < 2) return MX_ERR_INVALID_ARG;
  if (rotary < 2 || rotary % 2 != 0 || rotary > dim) return MX_ERR_INVALID_ARG;
  if ((position_bits != 32 && position_bits != 64) || !(eps >= 0.f)) return MX_ERR_INVALID_ARG;
  if (dim > 512 || q_heads > 65536 || k_heads > 65536 || tokens > (1 << 30) ||
      tokens * (q_heads + k_heads) > INT32_MAX)
    return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

// Heads [tokens, heads, dim] whose rows are apart from one another.
bool rows_apart(int64_t tokens, int64_t heads, int64_t dim, int64_t st, int64_t sh) {
  if (tokens == 0) return true;
  return (sh >= dim && st >= (heads - 1) * sh + dim) ||
         (st >= dim && sh >= (tokens - 1) * st + dim);
}

// (in bytes they stay below 2^31)
bool strides_fit(std::initializer_list<int64_t> strides) {
  for (int64_t s : strides)
    if (s >= (1 << 29)) return false;
  return true;
}

bool chunk_aligned(const void* p, int64_t st, int64_t sh, mx_dtype d) {
  const uintptr_t bytes = d == MX_FP32 ? 16 : 8;
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 && st % 4 == 0 && sh % 4 == 0;
}

mx_status route_check(int64_t tokens, int32_t experts, int32_t top_k, int64_t ld,
                      mx_dtype dtype) {
  if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts || top_k > 32 || ld < experts)
    return MX_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return MX_ERR_INVALID_ARG;
  if (experts > 512 || tokens > INT32_MAX / 512) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

// Rows that can be read four elements at a time.
bool quads(const void* p, int64_t ld, int64_t n, mx_dtype d) {
  const uintptr_t bytes = d == MX_FP32 ? 16 : 8;
  return n % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace

extern "C" {

mx_status mx_norm_rotate(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim,
                         int64_t rotary, const void* q, int64_t q_st, int64_t q_sh, const void* k,
                         int64_t k_st, int64_t k_sh, mx_dtype x_dtype, const void* w_q,
                         const void* w_k, mx_dtype w_dtype, const void* positions,
                         int32_t position_bits, const double* frequencies, int32_t interleaved,
                         float scale, float eps, void* out_q, int64_t oq_st, int64_t oq_sh,
                         void* out_k, int64_t ok_st, int64_t ok_sh, cudaStream_t stream) {
  if (!q || !k || !w_q || !w_k || !positions || !frequencies || !out_q || !out_k)
    return MX_ERR_INVALID_ARG;
  mx_status s = rotate_check(tokens, q_heads, k_heads, dim, rotary, x_dtype, w_dtype,
                             position_bits, eps);
  if (s != MX_OK) return s;
  if (q_st < 0 || q_sh < 0 || k_st < 0 || k_sh < 0) return MX_ERR_INVALID_ARG;
  if (!strides_fit({q_st, q_sh, k_st, k_sh, oq_st, oq_sh, ok_st, ok_sh}))
    return MX_ERR_UNSUPPORTED;
  if (!rows_apart(tokens, q_heads, dim, oq_st, oq_sh) ||
      !rows_apart(tokens, k_heads, dim, ok_st, ok_sh))
    return MX_ERR_INVALID_ARG;
  if (!aligned_elt(q, x_dtype) || !aligned_elt(k, x_dtype) || !aligned_elt(w_q, w_dtype) ||
      !aligned_elt(w_k, w_dtype) || !aligned_elt(out_q, x_dtype) || !aligned_elt(out_k, x_dtype) ||
      (reinterpret_cast<uintptr_t>(frequencies) & 7u) != 0 ||
      (reinterpret_cast<uintptr_t>(positions) & (position_bits / 8 - 1)) != 0)
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (tokens == 0) return MX_OK;
  if (!all_on_device(st->device, {q, k, w_q, w_k, positions, frequencies, out_q, out_k}))
    return MX_ERR_INVALID_ARG;
  mx::RotateParams p{};
  p.q = q;
  p.k = k;
  p.w_q = w_q;
  p.w_k = w_k;
  p.positions = positions;
  p.frequencies = frequencies;
  p.out_q = out_q;
  p.out_k = out_k;
  p.q_st = q_st;
  p.q_sh = q_sh;
  p.k_st = k_st;
  p.k_sh = k_sh;
  p.oq_st = oq_st;
  p.oq_sh = oq_sh;
  p.ok_st = ok_st;
  p.ok_sh = ok_sh;
  p.tokens = static_cast<int32_t>(tokens);
  p.q_heads = static_cast<int32_t>(q_heads);
  p.k_heads = static_cast<int32_t>(k_heads);
  p.dim = static_cast<int32_t>(dim);
  p.rotary = static_cast<int32_t>(rotary);
  p.interleaved = interleaved != 0;
  p.x_fp32 = x_dtype == MX_FP32;
  p.w_fp32 = w_dtype == MX_FP32;
  p.positions_64 = position_bits == 64;
  p.scale = scale;
  p.eps = eps;
  p.chunks = dim % 8 == 0 && rotary % 8 == 0 && chunk_aligned(q, q_st, q_sh, x_dtype) &&
             chunk_aligned(k, k_st, k_sh, x_dtype) && chunk_aligned(out_q, oq_st, oq_sh, x_dtype) &&
             chunk_aligned(out_k, ok_st, ok_sh, x_dtype);
  return mx::launch_norm_rotate(p, st->num_sms, stream) == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

size_t mx_norm_rotate_backward_workspace(int64_t tokens, int64_t dim) {
  if (tokens < 0 || tokens > (1 << 30) || dim < 2 || dim > 512) return 0;
  return mx::norm_rotate_backward_workspace(tokens, dim);
}

mx_status mx_norm_rotate_backward(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim,
                                  int64_t rotary, const void* d_q, int64_t dq_st, int64_t dq_sh,
                                  const void* d_k, int64_t dk_st, int64_t dk_sh, const void* q,
                                  int64_t q_st, int64_t q_sh, const void* k, int64_t k_st,
                                  int64_t k_sh, mx_dtype x_dtype, const void* w_q, const void* w_k,
                                  mx_dtype w_dtype, const void* positions, int32_t position_bits,
                                  const double* frequencies, int32_t interleaved, float scale,
                                  float eps, void* dx_q, void* dx_k, float* dw_q, float* dw_k,
                                  void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!d_q || !d_k || !q || !k || !w_q || !w_k || !positions || !frequencies || !dx_q || !dx_k ||
      !dw_q || !dw_k)
    return MX_ERR_INVALID_ARG;
  mx_status s = rotate_check(tokens, q_heads, k_heads, dim, rotary, x_dtype, w_dtype,
                             position_bits, eps);
  if (s != MX_OK) return s;
  if (q_st < 0 || q_sh < 0 || k_st < 0 || k_sh < 0 || dq_st < 0 || dq_sh < 0 || dk_st < 0 ||
      dk_sh < 0)
    return MX_ERR_INVALID_ARG;
  if (!strides_fit({q_st, q_sh, k_st, k_sh, dq_st, dq_sh, dk_st, dk_sh}))
    return MX_ERR_UNSUPPORTED;
  const size_t need = mx::norm_rotate_backward_workspace(tokens, dim);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MX_ERR_INVALID_ARG;
  if (!aligned_elt(d_q, x_dtype) || !aligned_elt(d_k, x_dtype) || !aligned_elt(q, x_dtype) ||
      !aligned_elt(k, x_dtype) || !aligned_elt(w_q, w_dtype) || !aligned_elt(w_k, w_dtype) ||
      !aligned_elt(dx_q, x_dtype) || !aligned_elt(dx_k, x_dtype) || !aligned_elt(dw_q, MX_FP32) ||
      !aligned_elt(dw_k, MX_FP32) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(frequencies) & 7u) != 0 ||
      (reinterpret_cast<uintptr_t>(positions) & (position_bits / 8 - 1)) != 0)
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (!all_on_device(st->device, {w_q, w_k, frequencies, dw_q, dw_k})) return MX_ERR_INVALID_ARG;
  if (tokens == 0)
    return cudaMemsetAsync(dw_q, 0, dim * sizeof(float), stream) == cudaSuccess &&
                   cudaMemsetAsync(dw_k, 0, dim * sizeof(float), stream) == cudaSuccess
               ? MX_OK
               : MX_ERR_CUDA;
  if (!all_on_device(st->device, {d_q, d_k, q, k, positions, dx_q, dx_k, workspace}))
    return MX_ERR_INVALID_ARG;
  mx::RotateParams p{};
  p.q = q;
  p.k = k;
  p.d_q = d_q;
  p.d_k = d_k;
  p.w_q = w_q;
  p.w_k = w_k;
  p.positions = positions;
  p.frequencies = frequencies;
  p.out_q = dx_q;
  p.out_k = dx_k;
  p.dw_q = dw_q;
  p.dw_k = dw_k;
  p.workspace = static_cast<float*>(workspace);
  p.q_st = q_st;
  p.q_sh = q_sh;
  p.k_st = k_st;
  p.k_sh = k_sh;
  p.dq_st = dq_st;
  p.dq_sh = dq_sh;
  p.dk_st = dk_st;
  p.dk_sh = dk_sh;
  p.oq_st = q_heads * dim;
  p.ok_st = k_heads * dim;
  p.oq_sh = p.ok_sh = dim;
  p.tokens = static_cast<int32_t>(tokens);
  p.q_heads = static_cast<int32_t>(q_heads);
  p.k_heads = static_cast<int32_t>(k_heads);
  p.dim = static_cast<int32_t>(dim);
  p.rotary = static_cast<int32_t>(rotary);
  p.interleaved = interleaved != 0;
  p.x_fp32 = x_dtype == MX_FP32;
  p.w_fp32 = w_dtype == MX_FP32;
  p.positions_64 = position_bits == 64;
  p.scale = scale;
  p.eps = eps;
  p.chunks = dim % 8 == 0 && rotary % 8 == 0 && chunk_aligned(q, q_st, q_sh, x_dtype) &&
             chunk_aligned(k, k_st, k_sh, x_dtype) && chunk_aligned(d_q, dq_st, dq_sh, x_dtype) &&
             chunk_aligned(d_k, dk_st, dk_sh, x_dtype) && chunk_aligned(dx_q, 0, 0, x_dtype) &&
             chunk_aligned(dx_k, 0, 0, x_dtype);
  return mx::launch_norm_rotate_backward(p, st->num_sms, stream) == cudaSuccess ? MX_OK
                                                                                : MX_ERR_CUDA;
}

size_t mx_route_workspace(int64_t tokens, int32_t experts) {
  if (route_check(tokens, experts, 1, experts, MX_FP32) != MX_OK) return 0;
  return mx::route_workspace(tokens, experts);
}

mx_status mx_route(int64_t tokens, int32_t experts, int32_t top_k, const void* logits, int64_t ld,
                   mx_dtype dtype, const uint8_t* mask, int32_t renormalize, int32_t* ids,
                   float* weights, float* lse, int32_t* counts, int32_t* offsets, int32_t* order,
                   float* balance, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!logits || !ids || !weights || !lse || !counts || !offsets || !order || !balance)
    return MX_ERR_INVALID_ARG;
  mx_status s = route_check(tokens, experts, top_k, ld, dtype);
  if (s != MX_OK) return s;
  const size_t need = mx::route_workspace(tokens, experts);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MX_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(ids), static_cast<const void*>(weights),
                        static_cast<const void*>(lse), static_cast<const void*>(counts),
                        static_cast<const void*>(offsets), static_cast<const void*>(order),
                        static_cast<const void*>(balance)})
    if (!aligned_elt(p, MX_FP32)) return MX_ERR_MISALIGNED;
  if (!aligned_elt(logits, dtype) || !aligned16(workspace)) return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (!all_on_device(st->device, {counts, offsets, balance})) return MX_ERR_INVALID_ARG;
  if (tokens > 0 &&
      !all_on_device(st->device, {logits, mask, ids, weights, lse, order, workspace}))
    return MX_ERR_INVALID_ARG;
  mx::RouteParams p{};
  p.logits = logits;
  p.mask = mask;
  p.ld = ld;
  p.tokens = static_cast<int32_t>(tokens);
  p.experts = experts;
  p.top_k = top_k;
  p.renormalize = renormalize != 0;
  p.logits_fp32 = dtype == MX_FP32;
  p.vec = quads(logits, ld, experts, dtype);
  p.ids = ids;
  p.weights = weights;
  p.lse = lse;
  p.counts = counts;
  p.offsets = offsets;
  p.order = order;
  p.balance = balance;
  p.workspace = static_cast<int32_t*>(workspace);
  return mx::launch_route(p, stream) == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

mx_status mx_route_backward(int64_t tokens, int32_t experts, int32_t top_k, const float* d_weights,
                            const float* d_balance, const float* d_lse, const void* logits,
                            int64_t ld, mx_dtype dtype, const uint8_t* mask, int32_t renormalize,
                            const int32_t* ids, const float* weights, const float* lse,
                            const int32_t* counts, void* d_logits, cudaStream_t stream) {
  if (!logits || !ids || !weights || !lse || !counts || !d_logits) return MX_ERR_INVALID_ARG;
  mx_status s = route_check(tokens, experts, top_k, ld, dtype);
  if (s != MX_OK) return s;
  for (const void* p : {static_cast<const void*>(d_weights), static_cast<const void*>(d_balance),
                        static_cast<const void*>(d_lse), static_cast<const void*>(ids),
                        static_cast<const void*>(weights), static_cast<const void*>(lse),
                        static_cast<const void*>(counts)})
    if (!aligned_elt(p, MX_FP32)) return MX_ERR_MISALIGNED;
  if (!aligned_elt(logits, dtype) || !aligned_elt(d_logits, dtype)) return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (tokens == 0) return MX_OK;
  if (!all_on_device(st->device, {d_weights, d_balance, d_lse, logits, mask, ids, weights, lse,
                                  counts, d_logits}))
    return MX_ERR_INVALID_ARG;
  mx::RouteParams p{};
  p.logits = logits;
  p.mask = mask;
  p.ld = ld;
  p.tokens = static_cast<int32_t>(tokens);
  p.experts = experts;
  p.top_k = top_k;
  p.renormalize = renormalize != 0;
  p.logits_fp32 = dtype == MX_FP32;
  p.vec = quads(logits, ld, experts, dtype);
  p.d_weights = d_weights;
  p.d_balance = d_balance;
  p.d_lse = d_lse;
  p.w_in = weights;
  p.ids_in = ids;
  p.counts_in = counts;
  p.lse_in = lse;
  p.d_logits = d_logits;
  p.vec_out = quads(d_logits, experts, experts, dtype);
  return mx::launch_route_backward(p, st->num_sms, stream) == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

}  // extern "C"

namespace {

// Sizes of the vocabulary loss: tiles of 256 rows x 256 columns are numbered in
// 32 bits, rows of x and of the weights start on 16 bytes.
constexpr int64_t kVocabTile = 256;
// Bytes of dz that a piece of the vocabulary takes at most, and columns that it has
// all the same, since every piece adds to all of dx (131072 tokens over 32768 x 4096:
// 66.9 ms with the 2048 columns of 512 MB, 65.0 with 4096).
constexpr int64_t kVocabPieceBytes = int64_t{1} << 29;
constexpr int64_t kVocabPieceCols = 4096;
// Bytes of the parts over which dx of more than 64 tokens is summed side by side, at
// most.  (What the device's places ask for stays below 26 MB at any sizes: it limits
// none of them, but bounds the workspace.)
constexpr int64_t kVocabPartBytes = (int64_t{32} << 20) - 16;
constexpr int64_t kVocabUnitBytes = 16;  // what dz is held in units of, behind the parts

mx_status vocab_check(int64_t tokens, int64_t hidden, int64_t vocab, int64_t ldx, int64_t ldw,
                      int32_t label_bits) {
  if (tokens < 0 || hidden < 8 || hidden % 8 != 0 || vocab < 1) return MX_ERR_INVALID_ARG;
  if (ldx < hidden || ldw < hidden) return MX_ERR_INVALID_ARG;
  if (label_bits != 32 && label_bits != 64) return MX_ERR_INVALID_ARG;
  if (tokens > (1 << 24) || hidden > (1 << 20) || vocab > (1 << 24)) return MX_ERR_UNSUPPORTED;
  if (ceil_div(tokens, kVocabTile) * ceil_div(vocab, kVocabTile) > INT32_MAX ||
      ceil_div(vocab, kVocabTile) * ceil_div(hidden, kVocabTile) > INT32_MAX)
    return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

// Few tokens have kernels of their own (vocab_few.cu).
bool vocab_few(int64_t tokens) { return tokens <= mx::kVocabFewTokens; }

// Parts of a contraction of `steps` steps, four at least a part, for `tiles` tiles on
// `places` places: as many as leave fewest places empty in the last round, and no
// more than that takes.
int64_t vocab_splits(int64_t tiles, int64_t steps, int64_t places) {
  int64_t best = 1;
  double used = 0.0;
  for (int64_t s = 1; s <= 32 && s * 4 <= steps; ++s) {
    const int64_t per = ceil_div(steps, s), parts = ceil_div(steps, per);
    // steps that are work, of those that all places could take meanwhile
    const double u = static_cast<double>(tiles * steps) /
                     static_cast<double>(ceil_div(tiles * parts, places) * places * per);
    if (u > used + 0.03) best = parts, used = u;
  }
  return best;
}

// How the gradient goes through the vocabulary: columns of a piece (whole
// tiles), and the parts over which dx sums each piece.
struct VocabPieces {
  int64_t cols;
  int32_t splits, steps;
  bool direct;  // dx is written by its one product
  size_t dz_bytes, dx_bytes;
};

VocabPieces vocab_pieces(int64_t tokens, int64_t hidden, int64_t vocab) {
  VocabPieces v;
  const bool few = vocab_few(tokens);
  const int64_t row = tokens * (few ? 4 : 2);  // bytes of dz a column (few tokens: two terms)
  const int64_t most = kVocabPieceBytes / (row > 0 ? row : 1) / kVocabTile * kVocabTile;
  const int64_t all = ceil_div(vocab, kVocabTile) * kVocabTile;
  const int64_t cols = most < kVocabPieceCols ? kVocabPieceCols : most;
  v.cols = cols < all ? cols : all;
  // dx has few tiles where tokens and hidden are small: then parts of the
  // contraction side by side
  const int64_t tiles = few ? ceil_div(hidden, 128)
                            : ceil_div(tokens, kVocabTile) * ceil_div(hidden, kVocabTile);
  // (steps of the first piece: each part has some, so the join reads what was written)
  const int64_t steps = ceil_div(v.cols < vocab ? v.cols : vocab, 64);
  int64_t splits = 1;
  if (few) {
    splits = vocab_splits(tiles, steps, mx::kVocabFewBlocks);
  } else {
    // dW's tiles share the launch and fill what dx leaves: a part of dx only has to
    // be shorter than a pair of blocks' share of all steps
    const int64_t dw_steps = ceil_div(v.cols, kVocabTile) * ceil_div(hidden, kVocabTile) *
                             ceil_div(tokens, 64);
    const int64_t share = (tiles * steps + dw_steps) / 76;
    while (splits < 32 && (splits + 1) * 4 <= steps && ceil_div(steps, splits) * 4 > share * 3 &&
           (splits + 1) * tokens * hidden * 4 <= kVocabPartBytes)
      ++splits;
  }
  v.steps = static_cast<int32_t>(ceil_div(steps, splits));
  v.splits = static_cast<int32_t>(ceil_div(steps, v.steps));
  v.direct = !few && v.splits == 1 && v.cols >= vocab;
  v.dz_bytes = static_cast<size_t>(row * v.cols);
  v.dx_bytes = v.direct ? 0 : static_cast<size_t>(tokens * hidden * 4 * v.splits);
  return v;
}

// Parts that a token's softmax is joined from: two a tile of columns, or four a
// block.
int64_t vocab_slots(int64_t tokens, int64_t vocab) {
  return vocab_few(tokens) ? 4 * mx::vocab_few_blocks(vocab, 1) : 2 * ceil_div(vocab, kVocabTile);
}

// Workspaces do not shrink as tokens grow, so that one for the most tokens of a
// program's calls suffices for all of them, although few tokens take more bytes each.
size_t vocab_forward_bytes(int64_t tokens, int64_t vocab) {
  // the label's logits (rounded up to 16 bytes), then the parts
  auto need = [&](int64_t t) { return ceil_div(t, 4) * 16 + t * vocab_slots(t, vocab) * 8; };
  const int64_t few = need(mx::kVocabFewTokens), all = need(tokens);
  return static_cast<size_t>(vocab_few(tokens) || all > few ? all : few);
}

// No less than dz_bytes + dx_bytes of VocabPieces: dz of the most columns that a piece
// of `tokens` or fewer has, and dx over the most parts.
size_t vocab_backward_bytes(int64_t tokens, int64_t hidden, int64_t vocab) {
  auto most = [](int64_t a, int64_t b) { return a > b ? a : b; };
  auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
  auto dz_of = [&](int64_t t) {
    const int64_t row = t * (vocab_few(t) ? 4 : 2);
    return least(row * ceil_div(vocab, kVocabTile) * kVocabTile,
                 most(row * kVocabPieceCols, kVocabPieceBytes));
  };
  const int64_t dz = vocab_few(tokens) ? dz_of(tokens) : most(dz_of(tokens), dz_of(mx::kVocabFewTokens));
  // 32 parts at most, of few tokens any, of more up to kVocabPartBytes; one part as it is
  const int64_t one = tokens * hidden * 4;
  const int64_t parts = most(kVocabPartBytes, 32 * mx::kVocabFewTokens * hidden * 4);
  return static_cast<size_t>(dz + most(one, least(32 * one, parts)) +
                             (tokens > 0 ? kVocabUnitBytes : 0));
}

// 2-D bf16 tensor map, box 64 columns x box_rows, 128-byte swizzle, zero fill.
mx_status encode_bf16_box(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                          int64_t ld, uint32_t box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * 2)};
  cuuint32_t box[2] = {64u, box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

// 3-D map of an output [parts][rows][cols] (contiguous parts), box of 128 bytes x
// 32 rows, 128-byte swizzle.
mx_status encode_output_map(CUtensorMap* map, void* base, bool f32, int64_t cols, int64_t rows,
                            int64_t ld, int64_t parts) {
  const int64_t elt = f32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(parts)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * elt),
                           static_cast<cuuint64_t>(ld * elt * rows)};
  cuuint32_t box[3] = {f32 ? 32u : 64u, 32u, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = g_encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MX_OK : MX_ERR_CUDA;
}

mx::VocabParams vocab_params(const DeviceState* st, int64_t tokens, int64_t vocab,
                             const void* labels, int32_t label_bits, int64_t ignore_index) {
  mx::VocabParams p{};
  p.splits = 1;
  p.tokens = static_cast<int32_t>(tokens);
  p.labels = labels;
  p.labels_64 = label_bits == 64;
  p.ignore_index = ignore_index;
  p.vocab = static_cast<int32_t>(vocab);
  p.status = st->status;
  p.wait_limit_ns = g_wait_ns.load(std::memory_order_relaxed);
  return p;
}

bool aligned_label(const void* p, int32_t bits) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bits / 8 - 1)) == 0;
}

}  // namespace

extern "C" {

size_t mx_linear_cross_entropy_workspace(int64_t tokens, int64_t hidden, int64_t vocab) {
  if (vocab_check(tokens, hidden, vocab, hidden, hidden, 64) != MX_OK) return 0;
  return vocab_forward_bytes(tokens, vocab);
}

mx_status mx_linear_cross_entropy(int64_t tokens, int64_t hidden, int64_t vocab, const void* x,
                                  int64_t ldx, const void* w, int64_t ldw, const void* labels,
                                  int32_t label_bits, int64_t ignore_index, float* loss,
                                  float* lse, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
  if (!x || !w || !labels || !loss || !lse) return MX_ERR_INVALID_ARG;
  mx_status s = vocab_check(tokens, hidden, vocab, ldx, ldw, label_bits);
  if (s != MX_OK) return s;
  const size_t need = vocab_forward_bytes(tokens, vocab);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || ldx % 8 != 0 || ldw % 8 != 0 || !aligned16(workspace) ||
      !aligned_label(labels, label_bits) || !aligned_elt(loss, MX_FP32) ||
      !aligned_elt(lse, MX_FP32))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (tokens == 0) return MX_OK;
  if (!all_on_device(st->device, {x, w, labels, loss, lse, workspace})) return MX_ERR_INVALID_ARG;
  mx::VocabParams p = vocab_params(st, tokens, vocab, labels, label_bits, ignore_index);
  p.k = static_cast<int32_t>(hidden);
  p.steps = static_cast<int32_t>(ceil_div(hidden, 64));
  p.slots = static_cast<int32_t>(vocab_slots(tokens, vocab));
  p.z_label = static_cast<float*>(workspace);
  p.partial = reinterpret_cast<float2*>(p.z_label + ceil_div(tokens, 4) * 4);
  CUtensorMap tx, tw;
  const bool few = vocab_few(tokens);
  const uint32_t box = few ? static_cast<uint32_t>(mx::vocab_few_box(tokens)) : 128u;
  if ((s = encode_bf16_box(&tx, x, hidden, tokens, ldx, box)) != MX_OK) return s;
  if ((s = encode_bf16_box(&tw, w, hidden, vocab, ldw, 128)) != MX_OK) return s;
  p.m = static_cast<int32_t>(few ? vocab : tokens);
  p.n = static_cast<int32_t>(few ? tokens : vocab);
  const cudaError_t err =
      few ? mx::launch_vocab_few(mx::VocabProduct::kStats, p, tw, tx, stream)
          : mx::launch_vocab_logits(mx::VocabProduct::kStats, p, tx, tw, tx, st->num_sms, stream);
  if (err != cudaSuccess || mx::launch_vocab_finish(p, loss, lse, stream) != cudaSuccess)
    return MX_ERR_CUDA;
  return MX_OK;
}

size_t mx_linear_cross_entropy_backward_workspace(int64_t tokens, int64_t hidden, int64_t vocab) {
  if (vocab_check(tokens, hidden, vocab, hidden, hidden, 64) != MX_OK) return 0;
  return vocab_backward_bytes(tokens, hidden, vocab);
}

mx_status mx_linear_cross_entropy_backward(int64_t tokens, int64_t hidden, int64_t vocab,
                                           const float* d_loss, const float* d_lse, const void* x,
                                           int64_t ldx, const void* w, int64_t ldw,
                                           const void* labels, int32_t label_bits,
                                           int64_t ignore_index, const float* lse, void* dx,
                                           void* dw, mx_dtype dw_dtype, void* workspace,
                                           size_t workspace_bytes, cudaStream_t stream) {
  if (!x || !w || !labels || !lse || (!dx && !dw)) return MX_ERR_INVALID_ARG;
  if (!valid_dtype(dw_dtype)) return MX_ERR_INVALID_ARG;
  mx_status s = vocab_check(tokens, hidden, vocab, ldx, ldw, label_bits);
  if (s != MX_OK) return s;
  const VocabPieces v = vocab_pieces(tokens, hidden, vocab);
  const size_t need = vocab_backward_bytes(tokens, hidden, vocab);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MX_ERR_INVALID_ARG;
  const bool dw_f32 = dw_dtype == MX_FP32;
  if (!aligned16(x) || !aligned16(w) || ldx % 8 != 0 || ldw % 8 != 0 || !aligned16(dx) ||
      !aligned16(dw) || !aligned16(workspace) ||
      !aligned_label(labels, label_bits) || !aligned_elt(d_loss, MX_FP32) ||
      !aligned_elt(d_lse, MX_FP32) || !aligned_elt(lse, MX_FP32))
    return MX_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((s = device_state(&st)) != MX_OK) return s;
  if (!all_on_device(st->device, {w, dw})) return MX_ERR_INVALID_ARG;
  const int64_t dw_elt = dw_f32 ? 4 : 2;
  if (tokens == 0 && !dw) return MX_OK;
  if (tokens == 0)
    return cudaMemsetAsync(dw, 0, static_cast<size_t>(vocab * hidden * dw_elt), stream) ==
                   cudaSuccess
               ? MX_OK
               : MX_ERR_CUDA;
  if (!all_on_device(st->device, {d_loss, d_lse, x, labels, lse, dx, workspace}))
    return MX_ERR_INVALID_ARG;
  uint8_t* dz = static_cast<uint8_t*>(workspace);
  float* parts = reinterpret_cast<float*>(dz + v.dz_bytes);
  for (int64_t col0 = 0; col0 < vocab; col0 += v.cols) {
    const int64_t cols = v.cols < vocab - col0 ? v.cols : vocab - col0;
    const void* w_piece = static_cast<const uint8_t*>(w) + col0 * ldw * 2;
    mx::VocabParams p = vocab_params(st, tokens, vocab, labels, label_bits, ignore_index);
    CUtensorMap ta, tb, ty;
    // dz of the piece
    const bool few = vocab_few(tokens);
    const uint32_t box = few ? static_cast<uint32_t>(mx::vocab_few_box(tokens)) : 128u;
    p.m = static_cast<int32_t>(few ? cols : tokens);
    p.n = static_cast<int32_t>(few ? tokens : cols);
    p.k = static_cast<int32_t>(hidden);
    p.steps = static_cast<int32_t>(ceil_div(hidden, 64));
    p.col0 = static_cast<int32_t>(col0);
    p.lse = lse;
    p.d_loss = d_loss;
    p.d_lse = d_lse;
    p.scale = few ? nullptr : reinterpret_cast<float*>(dz + v.dz_bytes + v.dx_bytes);
    p.out = dz;
    p.ld_out = v.cols;
    if ((s = encode_bf16_box(&ta, x, hidden, tokens, ldx, box)) != MX_OK) return s;
    if ((s = encode_bf16_box(&tb, w_piece, hidden, cols, ldw, 128)) != MX_OK) return s;
    if ((s = encode_output_map(&ty, dz, false, cols, tokens, v.cols, 1)) != MX_OK) return s;
    cudaError_t err =
        few ? mx::launch_vocab_few(mx::VocabProduct::kGrad, p, tb, ta, stream)
            : mx::launch_vocab_logits(mx::VocabProduct::kGrad, p, ta, tb, ty, st->num_sms, stream);
    if (err != cudaSuccess) return MX_ERR_CUDA;
    // dx of the piece: contiguous along the vocabulary times contiguous along hidden
    mx::VocabParams px = p, pw = p;
    CUtensorMap xa, xb, xy, wa, wb, wy;
    if (dx) {
      px.m = static_cast<int32_t>(few ? hidden : tokens);
      px.n = static_cast<int32_t>(few ? tokens : hidden);
      px.k = static_cast<int32_t>(cols);
      px.steps = v.steps;
      px.splits = static_cast<int32_t>(ceil_div(ceil_div(cols, 64), v.steps));
      px.y_fp32 = !v.direct;
      px.add = col0 > 0;
      px.out = parts;
      px.ld_out = hidden;
      if ((s = encode_bf16_box(&xa, dz, cols, few ? 2 * tokens : tokens, v.cols, box)) != MX_OK)
        return s;
      if ((s = encode_bf16_box(&xb, w_piece, hidden, cols, ldw, 64)) != MX_OK) return s;
      if ((s = encode_output_map(&xy, v.direct ? dx : parts, !v.direct, hidden, tokens, hidden,
                                 v.splits)) != MX_OK)
        return s;
    }
    // dW of the piece: both operands contiguous along their rows
    if (dw) {
      pw.m = static_cast<int32_t>(cols);
      pw.n = static_cast<int32_t>(hidden);
      pw.k = static_cast<int32_t>(tokens);
      pw.steps = static_cast<int32_t>(ceil_div(tokens, 64));
      if (few) {
        pw.low_row = static_cast<int32_t>(tokens);
        pw.k = 128;
        pw.steps = 2;
      }
      pw.splits = 1;
      pw.y_fp32 = dw_f32;
      if ((s = encode_bf16_box(&wa, dz, cols, few ? 2 * tokens : tokens, v.cols, 64)) != MX_OK)
        return s;
      if ((s = encode_bf16_box(&wb, x, hidden, tokens, ldx, 64)) != MX_OK) return s;
      if ((s = encode_output_map(&wy, static_cast<uint8_t*>(dw) + col0 * hidden * dw_elt, dw_f32,
                                 hidden, cols, hidden, 1)) != MX_OK)
        return s;
    }
    if (dx && few) {
      if (mx::launch_vocab_few(mx::VocabProduct::kDx, px, xb, xa, stream) != cudaSuccess)
        return MX_ERR_CUDA;
    }
    const mx::VocabGradient gx = {&px, &xa, &xb, &xy}, gw = {&pw, &wa, &wb, &wy};
    if (mx::launch_vocab_gradients(dx && !few ? &gx : nullptr, dw ? &gw : nullptr, st->num_sms,
                                   stream) != cudaSuccess)
      return MX_ERR_CUDA;
  }
  if (dx && !v.direct && mx::launch_vocab_join(parts, v.splits, tokens * hidden, dx, st->num_sms,
                                         stream) != cudaSuccess)
    return MX_ERR_CUDA;
  return MX_OK;
}

mx_status mx_device_status(cudaStream_t stream) {
  DeviceState* st = nullptr;
  mx_status s = device_state(&st);
  if (s != MX_OK) return s;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return MX_ERR_CUDA;
  uint32_t word = 0;
  if (cudaMemcpy(&word, st->status, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
    return MX_ERR_CUDA;
  if (word != 0) {
    // clear only the bits read here (a kernel on another stream may set one
    // meanwhile; it then stays for the next query)
    if (mx::launch_status_clear(st->status, word, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
      return MX_ERR_CUDA;
  }
  if (word & 1u) return MX_ERR_TIMEOUT;
  if (word & 6u) return MX_ERR_DEVICE_ARG;
  return MX_OK;
}

mx_status mx_set_wait_timeout_ns(uint64_t ns) {
  g_wait_ns.store(ns == 0 ? kDefaultWaitNs : ns, std::memory_order_relaxed);
  return MX_OK;
}

mx_status mx_selftest_wait_timeout(uint64_t ns, cudaStream_t stream) {
  if (ns == 0 || ns > 10000000000ull) return MX_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  mx_status s = device_state(&st);
  if (s != MX_OK) return s;
  return mx::launch_wait_selftest(st->status, ns, stream) == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

const char* mx_status_str(mx_status status) {
  switch (status) {
    case MX_OK: return "MX_OK";
    case MX_ERR_INVALID_ARG: return "MX_ERR_INVALID_ARG";
    case MX_ERR_MISALIGNED: return "MX_ERR_MISALIGNED";
    case MX_ERR_UNSUPPORTED: return "MX_ERR_UNSUPPORTED";
    case MX_ERR_CUDA: return "MX_ERR_CUDA";
    case MX_ERR_TIMEOUT: return "MX_ERR_TIMEOUT";
    case MX_ERR_DEVICE_ARG: return "MX_ERR_DEVICE_ARG";
  }
  return "MX_ERR_UNKNOWN";
}

}  // extern "C"
