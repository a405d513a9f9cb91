// binding.cpp -- the tensor API of the operators around the products, in C++:
// argument checks, outputs, workspace and the C call in one step.  These operators are
// called for single tokens, where the same work in Python and ctypes took
// longer than the kernels.
//
// A module of the CPython C API (`_binding`).  Each function takes its
// arguments by position, raises ValueError for a tensor that the kernels
// could not read or write, and returns its outputs, or the status of the C
// call (an int) when that is not MX_OK, or None where a forward pass is to be
// recorded for autograd (the caller then calls again from within a Function,
// where that is off).  The C entry points are handed over as
// addresses by `init`, so the module is bound to the libmx that the package
// loaded.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/core/StorageImpl.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "mx.h"

namespace {

decltype(&mx_norm_residual) norm_residual_fn;
decltype(&mx_norm_residual_backward) norm_backward_fn;
decltype(&mx_norm_residual_backward_workspace) norm_workspace_fn;
decltype(&mx_moe_few_tokens) moe_fn;
decltype(&mx_moe_few_tokens_workspace) moe_workspace_fn;
decltype(&mx_norm_rotate) rotate_fn;
decltype(&mx_norm_rotate_backward) rotate_backward_fn;
decltype(&mx_norm_rotate_backward_workspace) rotate_workspace_fn;
decltype(&mx_route) route_fn;
decltype(&mx_route_backward) route_backward_fn;
decltype(&mx_route_workspace) route_workspace_fn;
decltype(&mx_linear_cross_entropy) loss_fn;
decltype(&mx_linear_cross_entropy_workspace) loss_workspace_fn;
decltype(&mx_linear_cross_entropy_backward) loss_backward_fn;
decltype(&mx_linear_cross_entropy_backward_workspace) loss_backward_workspace_fn;
PyObject* out_of_memory;  // torch's exception for it

struct Refused {
  std::string what;
};

std::string shape_text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

[[noreturn]] void refuse(const char* name, const std::string& want) {
  throw Refused{std::string(name) + " must be " + want + " on the current CUDA device"};
}

bool wide(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
mx_dtype code_of(at::ScalarType t) { return t == at::kFloat ? MX_FP32 : MX_BF16; }
const char* name_of(at::ScalarType t) {
  return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16"
         : t == at::kInt ? "torch.int32" : t == at::kByte ? "torch.uint8" : t == at::kDouble ? "torch.float64"
         : "torch.bfloat16 or torch.float32";
}

// One call's arguments, which have to be on the current device (asked for
// when the first CUDA tensor is seen, so that host tensors are refused on a
// machine without a GPU too).
struct Call {
  PyObject* const* args;
  mutable c10::DeviceIndex device = -1;

  bool given(int i) const { return args[i] != Py_None; }
  // Whether autograd is on and one of these arguments asks for a gradient.
  bool recorded(std::initializer_list<int> which) const {
    if (!c10::GradMode::is_enabled()) return false;
    for (int i : which)
      if (given(i) && THPVariable_Check(args[i]) && THPVariable_Unpack(args[i]).requires_grad()) return true;
    return false;
  }
  // Refuses tangents of forward-mode differentiation: a kernel does not carry them
  // along, and an output without one would stand for a derivative of zero.
  void refuse_tangents(Py_ssize_t n) const {
    for (Py_ssize_t i = 0; i < n; ++i) {
      // (asking a number or None whether it is a tensor takes as long as the rest of it)
      if (args[i] == Py_None || PyLong_Check(args[i]) || PyFloat_Check(args[i])) continue;
      if (THPVariable_Check(args[i]) && THPVariable_Unpack(args[i])._fw_grad(0).defined())
        throw Refused{"forward-mode derivatives are not computed: no argument may be a dual tensor"};
    }
  }
  const at::Tensor& tensor(int i, const char* name) const {
    if (!THPVariable_Check(args[i])) throw Refused{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(args[i]);
  }
  bool here(const at::Tensor& t) const {
    if (!t.is_cuda()) return false;
    if (device < 0) device = c10::cuda::current_device();
    return t.get_device() == device;
  }

  // A [rows, cols] operand of `type` (at::ScalarType::Undefined: bf16 or FP32)
  // with unit column stride and rows that do not overlap; its leading
  // dimension (that of a single row is its length).
  const at::Tensor& rows_of(int i, const char* name, int64_t rows, int64_t cols,
                            at::ScalarType type, int64_t* ld) const {
    const at::Tensor& t = tensor(i, name);
    const bool ok = (type == at::ScalarType::Undefined ? wide(t.scalar_type()) : t.scalar_type() == type) &&
                    t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && here(t);
    if (ok && (cols <= 1 || t.stride(1) == 1)) {
      *ld = rows <= 1 ? cols : t.stride(0);
      if (*ld >= cols) return t;
    }
    refuse(name, std::string("a ") + name_of(type) + " tensor of shape " + shape_text({rows, cols}) +
                     ", row-major with unit column stride,");
  }
  // A contiguous operand.
  const at::Tensor& dense(int i, const char* name, at::IntArrayRef shape, at::ScalarType type) const {
    const at::Tensor& t = tensor(i, name);
    const bool ok = (type == at::ScalarType::Undefined ? wide(t.scalar_type()) : t.scalar_type() == type) &&
                    t.sizes() == shape && here(t) && t.is_contiguous();
    if (!ok) refuse(name, std::string("a contiguous ") + name_of(type) + " tensor of shape " + shape_text(shape));
    return t;
  }
  // Heads [tokens, heads, dim] with contiguous channels; their strides (those of
  // a single token or head are the contiguous ones).
  const at::Tensor& heads_of(int i, const char* name, int64_t tokens, int64_t heads, int64_t dim,
                             at::ScalarType type, int64_t* st, int64_t* sh) const {
    const at::Tensor& t = tensor(i, name);
    const bool ok = (type == at::ScalarType::Undefined ? wide(t.scalar_type()) : t.scalar_type() == type) &&
                    t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads && t.size(2) == dim &&
                    here(t) && (dim <= 1 || t.stride(2) == 1);
    if (!ok)
      refuse(name, std::string("a ") + name_of(type) + " tensor of shape " +
                       shape_text({tokens, heads, dim}) + " with unit channel stride,");
    *st = tokens <= 1 ? heads * dim : t.stride(0);
    *sh = heads <= 1 ? dim : t.stride(1);
    return t;
  }
  // A contiguous int32 or int64 operand; its bits.
  const at::Tensor& whole_numbers(int i, const char* name, int64_t n, int32_t* bits) const {
    const at::Tensor& t = tensor(i, name);
    if ((t.scalar_type() != at::kInt && t.scalar_type() != at::kLong) || t.dim() != 1 ||
        t.size(0) != n || !here(t) || !t.is_contiguous())
      refuse(name, "a contiguous torch.int32 or torch.int64 tensor of shape " + shape_text({n}));
    *bits = t.scalar_type() == at::kLong ? 64 : 32;
    return t;
  }
  // A contiguous mask of bool or uint8, or no address.
  const uint8_t* mask_of(int i, int64_t n) const {
    if (!given(i)) return nullptr;
    const at::Tensor& t = tensor(i, "mask");
    if ((t.scalar_type() != at::kBool && t.scalar_type() != at::kByte) || t.dim() != 1 ||
        t.size(0) != n || !here(t) || !t.is_contiguous())
      refuse("mask", "a contiguous torch.bool or torch.uint8 tensor of shape " + shape_text({n}));
    return static_cast<const uint8_t*>(t.data_ptr());
  }
  // A contiguous FP32 operand, or no address.
  const float* floats(int i, const char* name, at::IntArrayRef shape) const {
    return given(i) ? static_cast<const float*>(dense(i, name, shape, at::kFloat).data_ptr()) : nullptr;
  }
  int64_t integer(int i) const {
    const int64_t v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) throw Refused{""};
    return v;
  }
  double real(int i) const {
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{""};
    return v;
  }
  cudaStream_t stream(int i) const {
    return given(i) ? reinterpret_cast<cudaStream_t>(integer(i))
                    : c10::cuda::getCurrentCUDAStream(device).stream();
  }
};

// Whether torch's own operator has to make new tensors: a dispatch mode wants to see
// them, or what they hold at first is to be filled in.
bool through_torch() { return c10::impl::dispatch_mode_enabled() || at::globalContext().deterministicAlgorithms(); }

// A contiguous tensor in new memory of the current device, for the current stream,
// straight from the caching allocator: through torch's own operator it takes about a
// microsecond longer, as long as a kernel of a single token.
at::Tensor fresh(at::IntArrayRef shape, c10::ScalarType type) {
  if (through_torch()) return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA));
  int64_t bytes = static_cast<int64_t>(c10::elementSize(type));
  for (int64_t n : shape) bytes *= n;
  c10::Allocator* allocator = c10::cuda::CUDACachingAllocator::get();
  c10::Storage storage(c10::make_intrusive<c10::StorageImpl>(
      c10::StorageImpl::use_byte_size_t(), bytes, allocator->allocate(static_cast<size_t>(bytes)), allocator, true));
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// The memory that a call takes for itself, on the stream that its kernels run
// on.  While this stands that stream is the current one, so the allocator hands
// out memory whose last use is ordered before the kernels, and takes freed
// memory back (a workspace, routing that is not returned) for use behind them.
// Outputs are also kept until the caller's stream is past its uses.
class Memory {
 public:
  Memory(const Call& c, int i_stream)
      : c_(c), caller_(c10::cuda::getCurrentCUDAStream(c.device)), stream_(c.stream(i_stream)) {
    if (stream_ == caller_.stream()) return;
    guard_.reset_stream(stream_ ? c10::cuda::getStreamFromExternal(stream_, c.device)
                                : c10::cuda::getDefaultCUDAStream(c.device));
  }
  cudaStream_t stream() const { return stream_; }
  at::Tensor output(at::IntArrayRef shape, at::ScalarType type) const {
    const at::Tensor t = fresh(shape, type);
    if (stream_ != caller_.stream()) t.record_stream(caller_);
    return t;
  }
  // The caller's workspace, or one of `need` bytes.
  at::Tensor workspace(int i, size_t need) const {
    if (c_.given(i)) {
      const at::Tensor& t = c_.tensor(i, "workspace");
      if (t.scalar_type() != at::kByte || !c_.here(t) || !t.is_contiguous() ||
          static_cast<size_t>(t.numel()) < need)
        refuse("workspace", "a contiguous uint8 tensor of at least " + std::to_string(need) + " bytes");
      return t;
    }
    return fresh({need < 16 ? 16 : static_cast<int64_t>(need)}, at::kByte);
  }

 private:
  const Call& c_;
  c10::cuda::CUDAStream caller_;
  cudaStream_t stream_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};

// Small outputs out of one allocation, each on 16 bytes: an allocation each takes
// longer than the kernels of a call for a single token.  (Up to kSmall bytes; what is
// larger is its own, so that the caller can free one without the other.)
constexpr int64_t kSmall = 1 << 20;
class Together {
 public:
  Together(const Memory& memory, int64_t tensors, int64_t bytes) : memory_(memory) {
    if (!through_torch()) block_ = memory.output({bytes + 16 * tensors}, at::kByte);
  }
  at::Tensor take(at::IntArrayRef shape, at::ScalarType type) {
    if (!block_.defined()) return memory_.output(shape, type);
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(block_.storage()), block_.key_set(), c10::scalarTypeToTypeMeta(type));
    const int64_t size = static_cast<int64_t>(c10::elementSize(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(at_ / size);
    at_ = (at_ + t.numel() * size + 15) / 16 * 16;
    return t;
  }

 private:
  const Memory& memory_;
  at::Tensor block_;
  int64_t at_ = 0;
};

// A tensor of the caller's was written: what autograd saved of it is not valid
// any more.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The norm's weights, which share one type; gates is 0 without a gate.
struct Weights {
  void *pre = nullptr, *post = nullptr, *gate = nullptr;
  int64_t gates = 0;
  mx_dtype type = MX_BF16;
  at::IntArrayRef gate_shape;

  Weights(const Call& c, int i_pre, int i_post, int i_gate, int64_t rows, int64_t cols) {
    const at::Tensor& p = c.dense(i_pre, "w_pre", {cols}, at::ScalarType::Undefined);
    const at::ScalarType t = p.scalar_type();
    pre = p.data_ptr();
    type = code_of(t);
    if (c.given(i_post)) post = c.dense(i_post, "w_post", {cols}, t).data_ptr();
    if (!c.given(i_gate)) return;
    const at::Tensor& g = c.tensor(i_gate, "gate");
    if (g.dim() == 2) {
      gates = g.size(0);
      gate = c.dense(i_gate, "gate", {gates, cols}, t).data_ptr();
    } else {
      gates = 1;
      gate = c.dense(i_gate, "gate", {cols}, t).data_ptr();
    }
    gate_shape = g.sizes();
    if (gates < 1 || rows % gates)
      throw Refused{std::to_string(rows) + " rows cannot be split evenly over " + std::to_string(gates) + " gates"};
  }
};

PyObject* status_of(mx_status s) { return PyLong_FromLong(s); }

// block, residual, w_pre, w_post, gate, alpha, eps, out_residual, out, stream
PyObject* norm_residual(const Call& c) {
  if (c.recorded({0, 1, 2, 3, 4, 7, 8})) Py_RETURN_NONE;
  const at::Tensor& block = c.tensor(0, "block");
  if (block.dim() != 2) throw Refused{"block must be a 2-D tensor"};
  const int64_t rows = block.size(0), cols = block.size(1);
  int64_t ldb, ldr, ldo = cols, ldy = cols;
  c.rows_of(0, "block", rows, cols, at::ScalarType::Undefined, &ldb);
  const at::Tensor& residual = c.rows_of(1, "residual", rows, cols, at::ScalarType::Undefined, &ldr);
  const Weights w(c, 2, 3, 4, rows, cols);
  const float alpha = static_cast<float>(c.real(5)), eps = static_cast<float>(c.real(6));
  const Memory memory(c, 9);
  const at::Tensor res_out =
      c.given(7) ? c.rows_of(7, "out_residual", rows, cols, residual.scalar_type(), &ldo)
                 : memory.output({rows, cols}, residual.scalar_type());
  const at::Tensor y = c.given(8) ? c.rows_of(8, "out", rows, cols, block.scalar_type(), &ldy)
                                  : memory.output({rows, cols}, block.scalar_type());
  if (rows > 0) {
    mx_status s;
    Py_BEGIN_ALLOW_THREADS
    s = norm_residual_fn(rows, cols, block.data_ptr(), ldb, code_of(block.scalar_type()),
                         residual.data_ptr(), ldr, code_of(residual.scalar_type()), w.post, w.pre,
                         w.gate, w.gates, w.type, alpha, eps, res_out.data_ptr(), ldo, y.data_ptr(),
                         ldy, memory.stream());
    Py_END_ALLOW_THREADS
    if (s != MX_OK) return status_of(s);
  }
  if (c.given(7)) written(res_out);
  if (c.given(8)) written(y);
  PyObject* out = PyTuple_New(2);
  if (!out) return nullptr;
  if (c.given(7)) {
    Py_INCREF(c.args[7]);
    PyTuple_SET_ITEM(out, 0, c.args[7]);
  } else {
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(res_out));
  }
  if (c.given(8)) {
    Py_INCREF(c.args[8]);
    PyTuple_SET_ITEM(out, 1, c.args[8]);
  } else {
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(y));
  }
  return out;
}

// d_residual, d_y, block, residual, w_pre, w_post, gate, alpha, eps, workspace, stream
PyObject* norm_residual_backward(const Call& c) {
  const at::Tensor& block = c.tensor(2, "block");
  if (block.dim() != 2) throw Refused{"block must be a 2-D tensor"};
  const int64_t rows = block.size(0), cols = block.size(1);
  int64_t ldb, ldr, lddy, ldd = cols;
  c.rows_of(2, "block", rows, cols, at::ScalarType::Undefined, &ldb);
  const at::Tensor& residual = c.rows_of(3, "residual", rows, cols, at::ScalarType::Undefined, &ldr);
  const at::Tensor& dy = c.rows_of(1, "d_y", rows, cols, block.scalar_type(), &lddy);
  const void* d_res = nullptr;
  if (c.given(0))
    d_res = c.rows_of(0, "d_residual", rows, cols, residual.scalar_type(), &ldd).data_ptr();
  const Weights w(c, 4, 5, 6, rows, cols);
  const float alpha = static_cast<float>(c.real(7)), eps = static_cast<float>(c.real(8));
  const Memory memory(c, 10);
  const size_t need = norm_workspace_fn(rows, cols, w.gates);
  const at::Tensor ws = memory.workspace(9, need);
  constexpr at::ScalarType f32 = at::kFloat;
  const at::Tensor d_block = memory.output({rows, cols}, block.scalar_type());
  const at::Tensor d_residual = memory.output({rows, cols}, residual.scalar_type());
  const at::Tensor d_pre = memory.output({cols}, f32);
  at::Tensor d_post, d_gate;
  if (w.post) d_post = memory.output({cols}, f32);
  if (w.gate) d_gate = memory.output(w.gate_shape, f32);
  // a tensor without rows has no address; the workspace's stands in, unused
  void* none = ws.data_ptr();
  const bool empty = rows == 0;
  mx_status s;
  Py_BEGIN_ALLOW_THREADS
  s = norm_backward_fn(rows, cols, empty ? nullptr : d_res, ldd, empty ? none : dy.data_ptr(), lddy,
                       empty ? none : block.data_ptr(), ldb, code_of(block.scalar_type()),
                       empty ? none : residual.data_ptr(), ldr, code_of(residual.scalar_type()),
                       w.post, w.pre, w.gate, w.gates, w.type, alpha, eps,
                       empty ? none : d_block.data_ptr(), cols, empty ? none : d_residual.data_ptr(),
                       cols, static_cast<float*>(address(d_post)), static_cast<float*>(d_pre.data_ptr()),
                       static_cast<float*>(address(d_gate)), ws.data_ptr(),
                       static_cast<size_t>(ws.numel()), memory.stream());
  Py_END_ALLOW_THREADS
  if (s != MX_OK) return status_of(s);
  PyObject* out = PyTuple_New(5);
  if (!out) return nullptr;
  const at::Tensor* grads[5] = {&d_block, &d_residual, &d_pre, &d_post, &d_gate};
  for (int i = 0; i < 5; ++i)  // (an undefined tensor becomes None)
    PyTuple_SET_ITEM(out, i, THPVariable_Wrap(*grads[i]));
  return out;
}

// x, router, gate codes, gate scales, up codes, up scales, format, bits, down
// codes, down scales, format, bits, top_k, renormalize, out, workspace, stream
PyObject* moe_few_tokens(const Call& c) {
  if (c.recorded({0, 1, 14})) Py_RETURN_NONE;
  const at::Tensor& x = c.tensor(0, "x");
  if (x.dim() != 2) throw Refused{"x must be a 2-D tensor"};
  const at::Tensor& router = c.tensor(1, "router");
  if (router.dim() != 2) throw Refused{"router must be a 2-D tensor"};
  const at::Tensor& gate = c.tensor(2, "gate codes");
  if (gate.dim() != 3) throw Refused{"gate codes must be [experts, inter, hidden]"};
  const int64_t tokens = x.size(0), hidden = x.size(1), experts = router.size(0), inter = gate.size(1);
  int64_t ldx, ldy = hidden;
  c.rows_of(0, "x", tokens, hidden, at::kBFloat16, &ldx);
  c.dense(1, "router", {experts, hidden}, at::ScalarType::Undefined);
  const int64_t fmt_gu = c.integer(6), bits_gu = c.integer(7), fmt_d = c.integer(10), bits_d = c.integer(11);
  c.dense(2, "gate codes", {experts, inter, hidden * bits_gu / 8}, at::kByte);
  const at::Tensor& up = c.dense(4, "up codes", {experts, inter, hidden * bits_gu / 8}, at::kByte);
  const at::Tensor& down = c.dense(8, "down codes", {experts, hidden, inter * bits_d / 8}, at::kByte);
  const int64_t scales = experts * ((inter + 127) / 128) * ((hidden + 127) / 128) * 512;
  const void* s[3];
  const int at_scales[3] = {3, 5, 9};
  for (int i = 0; i < 3; ++i) {
    const at::Tensor& t = c.tensor(at_scales[i], "scales");
    if (t.scalar_type() != at::kByte || !c.here(t) || !t.is_contiguous() || t.numel() < scales)
      refuse(i == 0 ? "gate scales" : i == 1 ? "up scales" : "down scales",
             "a contiguous torch.uint8 tensor of at least " + std::to_string(scales) + " bytes");
    s[i] = t.data_ptr();
  }
  const int64_t top_k = c.integer(12);
  if (top_k < 1 || top_k > experts)
    throw Refused{"top_k must be 1 to " + std::to_string(experts) + ", got " + std::to_string(top_k)};
  const Memory memory(c, 16);
  const at::Tensor y = c.given(14) ? c.rows_of(14, "out", tokens, hidden, at::kBFloat16, &ldy)
                                   : memory.output({tokens, hidden}, x.scalar_type());
  const at::Tensor ids = memory.output({tokens, top_k}, at::kInt);
  const at::Tensor weights = memory.output({tokens, top_k}, at::kFloat);
  if (tokens > 0) {
    const bool fits = tokens <= INT32_MAX && experts <= INT32_MAX;
    const size_t need =
        fits ? moe_workspace_fn(static_cast<int32_t>(tokens), hidden, inter,
                                static_cast<int32_t>(experts), static_cast<int32_t>(top_k))
             : 0;
    const at::Tensor ws = memory.workspace(15, need);
    mx_status status = MX_ERR_UNSUPPORTED;
    const int32_t renormalize = static_cast<int32_t>(c.integer(13));
    if (fits) {
      Py_BEGIN_ALLOW_THREADS
      status = moe_fn(static_cast<int32_t>(tokens), hidden, inter, static_cast<int32_t>(experts),
                      static_cast<int32_t>(top_k), x.data_ptr(), ldx, router.data_ptr(),
                      code_of(router.scalar_type()), static_cast<const uint8_t*>(gate.data_ptr()),
                      static_cast<const uint8_t*>(s[0]), static_cast<const uint8_t*>(up.data_ptr()),
                      static_cast<const uint8_t*>(s[1]), static_cast<mx_fmt>(fmt_gu),
                      static_cast<const uint8_t*>(down.data_ptr()), static_cast<const uint8_t*>(s[2]),
                      static_cast<mx_fmt>(fmt_d), renormalize, y.data_ptr(), ldy,
                      static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(weights.data_ptr()),
                      ws.data_ptr(), static_cast<size_t>(ws.numel()), memory.stream());
      Py_END_ALLOW_THREADS
    }
    if (status != MX_OK) return status_of(status);
  }
  if (c.given(14)) written(y);
  PyObject* out = PyTuple_New(3);
  if (!out) return nullptr;
  if (c.given(14)) {
    Py_INCREF(c.args[14]);
    PyTuple_SET_ITEM(out, 0, c.args[14]);
  } else {
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(y));
  }
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(ids));
  PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(weights));
  return out;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> tensors) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : tensors) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}

// The arguments that the heads' norms and their gradient share: q, k, w_q, w_k,
// positions, frequencies, interleaved, scale, eps, from argument `i` on.
struct Heads {
  at::Tensor q, k;
  int64_t tokens, q_heads, k_heads, dim, rotary, q_st, q_sh, k_st, k_sh;
  const void *w_q, *w_k, *positions;
  const double* frequencies;
  int32_t position_bits, interleaved;
  mx_dtype x_type, w_type;
  float scale, eps;

  // of q and k together
  int64_t bytes() const { return tokens * (q_heads + k_heads) * dim * (x_type == MX_FP32 ? 4 : 2); }

  Heads(const Call& c, int i) {
    q = c.tensor(i, "q");
    k = c.tensor(i + 1, "k");
    if (q.dim() != 3 || k.dim() != 3) throw Refused{"q and k must be 3-D tensors [tokens, heads, dim]"};
    tokens = q.size(0), q_heads = q.size(1), dim = q.size(2), k_heads = k.size(1);
    c.heads_of(i, "q", tokens, q_heads, dim, at::ScalarType::Undefined, &q_st, &q_sh);
    c.heads_of(i + 1, "k", tokens, k_heads, dim, q.scalar_type(), &k_st, &k_sh);
    x_type = code_of(q.scalar_type());
    const at::Tensor& w = c.dense(i + 2, "w_q", {dim}, at::ScalarType::Undefined);
    w_q = w.data_ptr();
    w_type = code_of(w.scalar_type());
    w_k = c.dense(i + 3, "w_k", {dim}, w.scalar_type()).data_ptr();
    positions = c.whole_numbers(i + 4, "positions", tokens, &position_bits).data_ptr();
    const at::Tensor& f = c.tensor(i + 5, "frequencies");
    if (f.dim() != 1 || f.size(0) < 1 || 2 * f.size(0) > dim)
      throw Refused{"frequencies must be a 1-D tensor of 1 to dim / 2 (" + std::to_string(dim / 2) + ") entries"};
    frequencies = static_cast<const double*>(c.dense(i + 5, "frequencies", {f.size(0)}, at::kDouble).data_ptr());
    rotary = 2 * f.size(0);
    interleaved = static_cast<int32_t>(c.integer(i + 6));
    scale = static_cast<float>(c.real(i + 7));
    eps = static_cast<float>(c.real(i + 8));
  }
};

// q, k, w_q, w_k, positions, frequencies, interleaved, scale, eps, out_q, out_k, stream
PyObject* norm_rotate(const Call& c) {
  if (c.recorded({5})) throw Refused{"frequencies must not ask for a gradient: norm_rotate has none for them"};
  if (c.recorded({0, 1, 2, 3, 9, 10})) Py_RETURN_NONE;
  const Heads h(c, 0);
  int64_t oq_st = h.q_heads * h.dim, oq_sh = h.dim, ok_st = h.k_heads * h.dim, ok_sh = h.dim;
  const Memory memory(c, 11);
  at::Tensor out_q, out_k;
  if (c.given(9))
    out_q = c.heads_of(9, "out_q", h.tokens, h.q_heads, h.dim, h.q.scalar_type(), &oq_st, &oq_sh);
  if (c.given(10))
    out_k = c.heads_of(10, "out_k", h.tokens, h.k_heads, h.dim, h.q.scalar_type(), &ok_st, &ok_sh);
  if (!c.given(9) && !c.given(10) && h.bytes() <= kSmall) {
    Together outputs(memory, 2, h.bytes());
    out_q = outputs.take({h.tokens, h.q_heads, h.dim}, h.q.scalar_type());
    out_k = outputs.take({h.tokens, h.k_heads, h.dim}, h.q.scalar_type());
  } else {
    if (!c.given(9)) out_q = memory.output({h.tokens, h.q_heads, h.dim}, h.q.scalar_type());
    if (!c.given(10)) out_k = memory.output({h.tokens, h.k_heads, h.dim}, h.q.scalar_type());
  }
  if (h.tokens > 0) {
    mx_status s;
    Py_BEGIN_ALLOW_THREADS
    s = rotate_fn(h.tokens, h.q_heads, h.k_heads, h.dim, h.rotary, h.q.data_ptr(), h.q_st, h.q_sh,
                  h.k.data_ptr(), h.k_st, h.k_sh, h.x_type, h.w_q, h.w_k, h.w_type, h.positions,
                  h.position_bits, h.frequencies, h.interleaved, h.scale, h.eps, out_q.data_ptr(), oq_st,
                  oq_sh, out_k.data_ptr(), ok_st, ok_sh, memory.stream());
    Py_END_ALLOW_THREADS
    if (s != MX_OK) return status_of(s);
  }
  PyObject* out = PyTuple_New(2);
  if (!out) return nullptr;
  const at::Tensor* results[2] = {&out_q, &out_k};
  for (int i = 0; i < 2; ++i) {
    if (c.given(9 + i)) {
      written(*results[i]);
      Py_INCREF(c.args[9 + i]);
      PyTuple_SET_ITEM(out, i, c.args[9 + i]);
    } else {
      PyTuple_SET_ITEM(out, i, THPVariable_Wrap(*results[i]));
    }
  }
  return out;
}

// d_q, d_k, q, k, w_q, w_k, positions, frequencies, interleaved, scale, eps, workspace, stream
PyObject* norm_rotate_backward(const Call& c) {
  const Heads h(c, 2);
  int64_t dq_st, dq_sh, dk_st, dk_sh;
  const at::Tensor& d_q = c.heads_of(0, "d_q", h.tokens, h.q_heads, h.dim, h.q.scalar_type(), &dq_st, &dq_sh);
  const at::Tensor& d_k = c.heads_of(1, "d_k", h.tokens, h.k_heads, h.dim, h.q.scalar_type(), &dk_st, &dk_sh);
  const Memory memory(c, 12);
  const at::Tensor ws = memory.workspace(11, rotate_workspace_fn(h.tokens, h.dim));
  const bool small = h.bytes() <= kSmall;
  Together outputs(memory, 4, (small ? h.bytes() : 0) + 8 * h.dim);
  const at::Tensor dw_q = outputs.take({h.dim}, at::kFloat), dw_k = outputs.take({h.dim}, at::kFloat);
  at::Tensor dx_q, dx_k;
  if (small) {
    dx_q = outputs.take({h.tokens, h.q_heads, h.dim}, h.q.scalar_type());
    dx_k = outputs.take({h.tokens, h.k_heads, h.dim}, h.q.scalar_type());
  } else {
    dx_q = memory.output({h.tokens, h.q_heads, h.dim}, h.q.scalar_type());
    dx_k = memory.output({h.tokens, h.k_heads, h.dim}, h.q.scalar_type());
  }
  // a tensor without tokens has no address; the workspace's stands in, unused
  void* none = ws.data_ptr();
  const bool empty = h.tokens == 0;
  mx_status s;
  Py_BEGIN_ALLOW_THREADS
  s = rotate_backward_fn(h.tokens, h.q_heads, h.k_heads, h.dim, h.rotary, empty ? none : d_q.data_ptr(), dq_st,
                         dq_sh, empty ? none : d_k.data_ptr(), dk_st, dk_sh, empty ? none : h.q.data_ptr(),
                         h.q_st, h.q_sh, empty ? none : h.k.data_ptr(), h.k_st, h.k_sh, h.x_type, h.w_q,
                         h.w_k, h.w_type, empty ? none : h.positions, h.position_bits, h.frequencies,
                         h.interleaved, h.scale, h.eps, empty ? none : dx_q.data_ptr(),
                         empty ? none : dx_k.data_ptr(), static_cast<float*>(dw_q.data_ptr()),
                         static_cast<float*>(dw_k.data_ptr()), ws.data_ptr(),
                         static_cast<size_t>(ws.numel()), memory.stream());
  Py_END_ALLOW_THREADS
  if (s != MX_OK) return status_of(s);
  return tuple_of({dx_q, dx_k, dw_q, dw_k});
}

// Logits [tokens, experts] and top_k.
struct Logits {
  at::Tensor z;
  int64_t tokens, experts, ld, top_k;
  Logits(const Call& c, int i, int i_top_k) {
    z = c.tensor(i, "logits");
    if (z.dim() != 2) throw Refused{"logits must be a 2-D tensor [tokens, experts]"};
    tokens = z.size(0), experts = z.size(1);
    c.rows_of(i, "logits", tokens, experts, at::ScalarType::Undefined, &ld);
    top_k = c.integer(i_top_k);
    if (top_k < 1 || top_k > experts)
      throw Refused{"top_k must be 1 to " + std::to_string(experts) + ", got " + std::to_string(top_k)};
    if (experts > 512) throw Refused{"logits of at most 512 experts are taken, got " + std::to_string(experts)};
    if (top_k > 32) throw Refused{"top_k must be at most 32, got " + std::to_string(top_k)};
  }
};

// logits, top_k, renormalize, mask, workspace, stream
PyObject* route(const Call& c) {
  if (c.recorded({0})) Py_RETURN_NONE;
  const Logits l(c, 0, 1);
  const uint8_t* mask = c.mask_of(3, l.tokens);
  const int32_t renormalize = static_cast<int32_t>(c.integer(2));
  const Memory memory(c, 5);
  const size_t need = route_workspace_fn(l.tokens, static_cast<int32_t>(l.experts));
  const at::Tensor ws = need > 0 || c.given(4) ? memory.workspace(4, need) : at::Tensor();
  const int64_t pairs = l.tokens * l.top_k;
  // (what is kept of many tokens' routing, a balance loss say, keeps the experts' sums alive
  // but not the tokens' arrays)
  const int64_t of_tokens = 4 * (3 * pairs + l.tokens), of_experts = 4 * (2 * l.experts + 2);
  const bool small = of_tokens + of_experts <= kSmall;
  Together outputs(memory, 7, of_experts + (small ? of_tokens : 0));
  auto take = [&](at::IntArrayRef shape, at::ScalarType type) {
    return small ? outputs.take(shape, type) : memory.output(shape, type);
  };
  const at::Tensor ids = take({l.tokens, l.top_k}, at::kInt);
  const at::Tensor weights = take({l.tokens, l.top_k}, at::kFloat);
  const at::Tensor order = take({pairs}, at::kInt);
  const at::Tensor lse = take({l.tokens}, at::kFloat);
  const at::Tensor counts = outputs.take({l.experts}, at::kInt);
  const at::Tensor offsets = outputs.take({l.experts + 1}, at::kInt);
  const at::Tensor balance = outputs.take({}, at::kFloat);
  // a tensor without tokens has no address; another one's stands in, unused
  void* none = counts.data_ptr();
  const bool empty = l.tokens == 0;
  mx_status s;
  Py_BEGIN_ALLOW_THREADS
  s = route_fn(l.tokens, static_cast<int32_t>(l.experts), static_cast<int32_t>(l.top_k),
               empty ? none : l.z.data_ptr(), l.ld, code_of(l.z.scalar_type()), mask, renormalize,
               static_cast<int32_t*>(empty ? none : ids.data_ptr()),
               static_cast<float*>(empty ? none : weights.data_ptr()),
               static_cast<float*>(empty ? none : lse.data_ptr()), static_cast<int32_t*>(counts.data_ptr()),
               static_cast<int32_t*>(offsets.data_ptr()), static_cast<int32_t*>(empty ? none : order.data_ptr()),
               static_cast<float*>(balance.data_ptr()), address(ws),
               ws.defined() ? static_cast<size_t>(ws.numel()) : 0,
               memory.stream());
  Py_END_ALLOW_THREADS
  if (s != MX_OK) return status_of(s);
  return tuple_of({ids, weights, counts, offsets, order, balance, lse});
}

// d_weights, d_balance, d_lse, logits, ids, weights, counts, lse, renormalize, mask, stream
PyObject* route_backward(const Call& c) {
  const at::Tensor& ids = c.tensor(4, "ids");
  if (ids.dim() != 2) throw Refused{"ids must be a 2-D tensor [tokens, top_k]"};
  const int64_t top_k = ids.size(1);
  const at::Tensor& z = c.tensor(3, "logits");
  if (z.dim() != 2) throw Refused{"logits must be a 2-D tensor [tokens, experts]"};
  const int64_t tokens = z.size(0), experts = z.size(1);
  int64_t ld;
  c.rows_of(3, "logits", tokens, experts, at::ScalarType::Undefined, &ld);
  if (top_k < 1 || top_k > experts || top_k > 32 || experts > 512)
    throw Refused{"ids must have 1 to min(experts, 32) columns, logits at most 512"};
  c.dense(4, "ids", {tokens, top_k}, at::kInt);
  const at::Tensor& weights = c.dense(5, "weights", {tokens, top_k}, at::kFloat);
  const at::Tensor& counts = c.dense(6, "counts", {experts}, at::kInt);
  const at::Tensor& lse = c.dense(7, "lse", {tokens}, at::kFloat);
  const float* d_weights = c.floats(0, "d_weights", {tokens, top_k});
  const float* d_balance = nullptr;
  if (c.given(1)) {
    const at::Tensor& t = c.tensor(1, "d_balance");
    if (t.scalar_type() != at::kFloat || t.numel() != 1 || !c.here(t))
      refuse("d_balance", "a torch.float32 tensor of one element");
    d_balance = static_cast<const float*>(t.data_ptr());
  }
  const float* d_lse = c.floats(2, "d_lse", {tokens});
  const uint8_t* mask = c.mask_of(9, tokens);
  const int32_t renormalize = static_cast<int32_t>(c.integer(8));
  const Memory memory(c, 10);
  const at::Tensor d = memory.output({tokens, experts}, z.scalar_type());
  if (tokens > 0) {
    mx_status s;
    Py_BEGIN_ALLOW_THREADS
    s = route_backward_fn(tokens, static_cast<int32_t>(experts), static_cast<int32_t>(top_k), d_weights,
                          d_balance, d_lse, z.data_ptr(), ld, code_of(z.scalar_type()), mask, renormalize,
                          static_cast<const int32_t*>(ids.data_ptr()),
                          static_cast<const float*>(weights.data_ptr()),
                          static_cast<const float*>(lse.data_ptr()),
                          static_cast<const int32_t*>(counts.data_ptr()), d.data_ptr(), memory.stream());
    Py_END_ALLOW_THREADS
    if (s != MX_OK) return status_of(s);
  }
  return THPVariable_Wrap(d);
}

// x, weight, labels, from argument `i` on.
struct Vocabulary {
  at::Tensor x, w;
  int64_t tokens, hidden, vocab, ldx, ldw;
  const void* labels;
  int32_t label_bits;
  Vocabulary(const Call& c, int i) {
    x = c.tensor(i, "x");
    w = c.tensor(i + 1, "weight");
    if (x.dim() != 2 || w.dim() != 2) throw Refused{"x and weight must be 2-D tensors"};
    tokens = x.size(0), hidden = x.size(1), vocab = w.size(0);
    c.rows_of(i, "x", tokens, hidden, at::kBFloat16, &ldx);
    c.rows_of(i + 1, "weight", vocab, hidden, at::kBFloat16, &ldw);
    labels = c.whole_numbers(i + 2, "labels", tokens, &label_bits).data_ptr();
    if (hidden < 8 || hidden % 8 || vocab < 1)
      throw Refused{"hidden must be a positive multiple of 8 and the vocabulary not empty"};
  }
};

// x, weight, labels, ignore_index, workspace, stream
PyObject* linear_cross_entropy(const Call& c) {
  if (c.recorded({0, 1})) Py_RETURN_NONE;
  const Vocabulary v(c, 0);
  const int64_t ignore = c.integer(3);
  const Memory memory(c, 5);
  at::Tensor loss, lse;
  if (8 * v.tokens <= kSmall) {
    Together outputs(memory, 2, 8 * v.tokens);
    loss = outputs.take({v.tokens}, at::kFloat);
    lse = outputs.take({v.tokens}, at::kFloat);
  } else {
    loss = memory.output({v.tokens}, at::kFloat);
    lse = memory.output({v.tokens}, at::kFloat);
  }
  if (v.tokens > 0) {
    const at::Tensor ws = memory.workspace(4, loss_workspace_fn(v.tokens, v.hidden, v.vocab));
    mx_status s;
    Py_BEGIN_ALLOW_THREADS
    s = loss_fn(v.tokens, v.hidden, v.vocab, v.x.data_ptr(), v.ldx, v.w.data_ptr(), v.ldw, v.labels,
                v.label_bits, ignore, static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()),
                ws.data_ptr(), static_cast<size_t>(ws.numel()), memory.stream());
    Py_END_ALLOW_THREADS
    if (s != MX_OK) return status_of(s);
  }
  return tuple_of({loss, lse});
}

// d_loss, d_lse, x, weight, labels, lse, ignore_index, weight gradient in FP32, x and
// weight wanted, workspace, stream
PyObject* linear_cross_entropy_backward(const Call& c) {
  const Vocabulary v(c, 2);
  const float* d_loss = c.floats(0, "d_loss", {v.tokens});
  const float* d_lse = c.floats(1, "d_lse", {v.tokens});
  const at::Tensor& lse = c.dense(5, "lse", {v.tokens}, at::kFloat);
  const int64_t ignore = c.integer(6);
  const bool f32 = c.integer(7) != 0;
  const bool need_x = c.integer(8) != 0, need_w = c.integer(9) != 0;
  if (!need_x && !need_w) return tuple_of({at::Tensor(), at::Tensor()});
  const Memory memory(c, 11);
  const at::Tensor ws = memory.workspace(10, loss_backward_workspace_fn(v.tokens, v.hidden, v.vocab));
  at::Tensor dx, dw;
  if (need_x) dx = memory.output({v.tokens, v.hidden}, v.x.scalar_type());
  if (need_w) dw = memory.output({v.vocab, v.hidden}, f32 ? at::kFloat : at::kBFloat16);
  void* none = ws.data_ptr();
  const bool empty = v.tokens == 0;
  mx_status s;
  Py_BEGIN_ALLOW_THREADS
  s = loss_backward_fn(v.tokens, v.hidden, v.vocab, empty ? nullptr : d_loss, empty ? nullptr : d_lse,
                       empty ? none : v.x.data_ptr(), v.ldx, v.w.data_ptr(), v.ldw, empty ? none : v.labels,
                       v.label_bits, ignore, static_cast<const float*>(empty ? none : lse.data_ptr()),
                       !need_x ? nullptr : empty ? none : dx.data_ptr(), address(dw), f32 ? MX_FP32 : MX_BF16, ws.data_ptr(),
                       static_cast<size_t>(ws.numel()), memory.stream());
  Py_END_ALLOW_THREADS
  if (s != MX_OK) return status_of(s);
  return tuple_of({dx, dw});
}

// No C++ exception leaves the module: a refusal is a ValueError, torch's own
// errors (out of memory among them) and anything else a RuntimeError.
template <PyObject* (*F)(const Call&), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  if (!norm_residual_fn) {
    PyErr_SetString(PyExc_RuntimeError, "the binding is not initialized");
    return nullptr;
  }
  try {
    const Call call{args};
    call.refuse_tangents(n);
    return F(call);
  } catch (const Refused& r) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(out_of_memory, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// One C entry point of `init`'s tuple.
template <typename Fn>
bool take(PyObject* addresses, Py_ssize_t i, Fn* fn) {
  void* at = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
  *fn = reinterpret_cast<Fn>(at);
  return at != nullptr;
}

PyObject* init(PyObject*, PyObject* args) {
  PyObject *a, *oom;
  if (!PyArg_ParseTuple(args, "O!O", &PyTuple_Type, &a, &oom)) return nullptr;
  if (PyTuple_GET_SIZE(a) != 15) {
    PyErr_SetString(PyExc_TypeError, "15 addresses are expected");
    return nullptr;
  }
  Py_INCREF(oom);
  Py_XSETREF(out_of_memory, oom);
  const bool all = take(a, 14, &loss_backward_workspace_fn) && take(a, 13, &loss_backward_fn) &&
                   take(a, 12, &loss_workspace_fn) && take(a, 11, &loss_fn) && take(a, 10, &route_workspace_fn) &&
                   take(a, 9, &route_backward_fn) && take(a, 8, &route_fn) && take(a, 7, &rotate_workspace_fn) &&
                   take(a, 6, &rotate_backward_fn) && take(a, 5, &rotate_fn) && take(a, 4, &moe_workspace_fn) &&
                   take(a, 3, &moe_fn) && take(a, 2, &norm_workspace_fn) && take(a, 1, &norm_backward_fn) &&
                   take(a, 0, &norm_residual_fn);
  if (!all) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is missing");
    return nullptr;
  }
  Py_RETURN_NONE;
}

template <PyObject* (*F)(const Call&), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, "Takes the addresses of the C entry points and torch's out-of-memory exception."},
    method<norm_residual, 10>("norm_residual"),
    method<norm_residual_backward, 11>("norm_residual_backward"),
    method<moe_few_tokens, 17>("moe_few_tokens"),
    method<norm_rotate, 12>("norm_rotate"),
    method<norm_rotate_backward, 13>("norm_rotate_backward"),
    method<route, 6>("route"),
    method<route_backward, 11>("route_backward"),
    method<linear_cross_entropy, 6>("linear_cross_entropy"),
    method<linear_cross_entropy_backward, 12>("linear_cross_entropy_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
