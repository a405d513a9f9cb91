// binding.cpp -- the tensor API of the block operators, in C++: argument
// checks, outputs, workspace and the C call in one step.  These operators are
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

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
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
         : t == at::kInt ? "torch.int32" : t == at::kByte ? "torch.uint8" : "torch.bfloat16 or torch.float32";
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
  at::Tensor output(at::IntArrayRef shape, const at::TensorOptions& options) const {
    const at::Tensor t = at::empty(shape, options);
    if (stream_ != caller_.stream()) t.record_stream(caller_);
    return t;
  }
  // The caller's workspace, or one of `need` bytes.
  at::Tensor workspace(int i, size_t need, const at::Tensor& like) const {
    if (c_.given(i)) {
      const at::Tensor& t = c_.tensor(i, "workspace");
      if (t.scalar_type() != at::kByte || !c_.here(t) || !t.is_contiguous() ||
          static_cast<size_t>(t.numel()) < need)
        refuse("workspace", "a contiguous uint8 tensor of at least " + std::to_string(need) + " bytes");
      return t;
    }
    return at::empty({need < 16 ? 16 : static_cast<int64_t>(need)}, like.options().dtype(at::kByte));
  }

 private:
  const Call& c_;
  c10::cuda::CUDAStream caller_;
  cudaStream_t stream_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
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
                 : memory.output({rows, cols}, residual.options());
  const at::Tensor y = c.given(8) ? c.rows_of(8, "out", rows, cols, block.scalar_type(), &ldy)
                                  : memory.output({rows, cols}, block.options());
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
  const at::Tensor ws = memory.workspace(9, need, block);
  const at::TensorOptions f32 = block.options().dtype(at::kFloat);
  const at::Tensor d_block = memory.output({rows, cols}, block.options());
  const at::Tensor d_residual = memory.output({rows, cols}, residual.options());
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
                                   : memory.output({tokens, hidden}, x.options());
  const at::Tensor ids = memory.output({tokens, top_k}, x.options().dtype(at::kInt));
  const at::Tensor weights = memory.output({tokens, top_k}, x.options().dtype(at::kFloat));
  if (tokens > 0) {
    const bool fits = tokens <= INT32_MAX && experts <= INT32_MAX;
    const size_t need =
        fits ? moe_workspace_fn(static_cast<int32_t>(tokens), hidden, inter,
                                static_cast<int32_t>(experts), static_cast<int32_t>(top_k))
             : 0;
    const at::Tensor ws = memory.workspace(15, need, x);
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
    return F(Call{args});
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

PyObject* init(PyObject*, PyObject* args) {
  unsigned long long a[5];
  PyObject* oom;
  if (!PyArg_ParseTuple(args, "KKKKKO", &a[0], &a[1], &a[2], &a[3], &a[4], &oom)) return nullptr;
  Py_INCREF(oom);
  Py_XSETREF(out_of_memory, oom);
  norm_residual_fn = reinterpret_cast<decltype(norm_residual_fn)>(a[0]);
  norm_backward_fn = reinterpret_cast<decltype(norm_backward_fn)>(a[1]);
  norm_workspace_fn = reinterpret_cast<decltype(norm_workspace_fn)>(a[2]);
  moe_fn = reinterpret_cast<decltype(moe_fn)>(a[3]);
  moe_workspace_fn = reinterpret_cast<decltype(moe_workspace_fn)>(a[4]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(const Call&), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, "Takes the addresses of the five C entry points and torch's out-of-memory exception."},
    method<norm_residual, 10>("norm_residual"),
    method<norm_residual_backward, 11>("norm_residual_backward"),
    method<moe_few_tokens, 17>("moe_few_tokens"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
