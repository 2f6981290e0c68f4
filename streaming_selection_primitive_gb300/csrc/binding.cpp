// Native half of the Python calls in _lm.py: checks the tensors, makes the
// outputs and calls the C-ABI (libprofk.so) on the current stream.  A call of
// a few microseconds spends most of them here if this is done in Python: one
// decoding step's route takes 19.5 us through ctypes, 6.5 us with this file.
//
// Functions take positional arguments only (the keyword forms are in _lm.py)
// and return the outputs, or the library's status where it is not PROFK_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <climits>
#include <optional>
#include <string>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/profk.h"

namespace {

using at::Tensor;

// Sets the Python error and leaves for the handler at the function's end.
template <typename... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw python_error();
}

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

// A forward-mode tangent of what the outputs are a function of would be lost.
const Tensor& without_tangent(const Tensor& t, const char* name) {
  if (t._fw_grad(0).defined()) refuse(PyExc_NotImplementedError, "%s has a forward-mode derivative, which this call has not", name);
  return t;
}

struct Logits {
  const Tensor* t;
  int64_t rows, n, ld;
  int type;
};

Logits logits_of(PyObject* o) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "logits must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  const at::ScalarType s = t.scalar_type();
  if (!t.is_cuda() || (s != at::kFloat && s != at::kBFloat16 && s != at::kHalf))
    refuse(PyExc_TypeError, "logits must be a float32, bfloat16 or float16 CUDA tensor");
  if (t.dim() != 2) refuse(PyExc_ValueError, "logits must be 2-D");
  without_tangent(t, "logits");
  const int64_t rows = t.size(0), n = t.size(1);
  if (n > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "logits must have unit column stride");
  return {&t, rows, n, rows > 1 ? t.stride(0) : n, s == at::kFloat ? PROFK_F32 : s == at::kBFloat16 ? PROFK_BF16 : PROFK_F16};
}

// A tensor of the given type on the logits' device.
const Tensor& on_device(PyObject* o, const char* name, at::ScalarType type, const Tensor& like) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  const Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type || t.device() != like.device())
    refuse(PyExc_TypeError, "%s must be a %s tensor on %s", name, c10::toString(type), like.device().str().c_str());
  return t;
}

// The same, contiguous and of the given shape: its address.
void* array(PyObject* o, const char* name, at::ScalarType type, const Tensor& like, at::IntArrayRef shape) {
  const Tensor& t = on_device(o, name, type, like);
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, "%s must have shape %s, not %s", name, text(shape).c_str(), text(t.sizes()).c_str());
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}

// A 2-D tensor of the given shape with unit column stride: its row stride.
int64_t rows_of(const Tensor& t, const char* name, int64_t rows, int64_t n) {
  const int64_t shape[2] = {rows, n};
  if (t.sizes() != at::IntArrayRef(shape))
    refuse(PyExc_ValueError, "%s must have shape %s, not %s", name, text(shape).c_str(), text(t.sizes()).c_str());
  if (n > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "%s must have unit column stride", name);
  return rows > 1 ? t.stride(0) : n;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// The tensors' device, and the call's stream: the one given, made current for the
// call, else the device's current one.  Outputs come from the stream's own blocks
// (one of the current stream's may still be in use by work queued there), and
// where a stream is given they are marked as used on the current one as well, so
// that what the caller queues on them there outlives them.
class Place {
 public:
  Place(PyObject* o, const Tensor& like)
      : like_(like), device_(like.device()), stream_(c10::cuda::getCurrentCUDAStream(like.device().index())) {
    if (o == Py_None) return;
    void* given = PyLong_AsVoidPtr(o);
    if (!given && PyErr_Occurred()) throw python_error();
    callers_ = stream_;
    stream_ = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(given), like.device().index());
    side_.emplace(stream_);
  }
  cudaStream_t stream() const { return stream_.stream(); }
  Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    Tensor t = at::detail::empty_cuda(shape, like_.options().dtype(type));
    if (callers_) t.record_stream(*callers_);
    return t;
  }

 private:
  const Tensor& like_;
  c10::cuda::CUDAGuard device_;
  c10::cuda::CUDAStream stream_;
  std::optional<c10::cuda::CUDAStream> callers_;
  std::optional<c10::cuda::CUDAStreamGuard> side_;
};

PyObject* tuple_of(std::initializer_list<Tensor> tensors) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (!t) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& x : tensors) PyTuple_SET_ITEM(t, i++, x.defined() ? THPVariable_Wrap(x) : Py_NewRef(Py_None));
  return t;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
}

// logits, noise, temperature, top_k, top_p, min_p, mask, out, stream
PyObject* sample_tokens(PyObject*, PyObject* const* arg, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  expect(count, 9);
  const Logits x = logits_of(arg[0]);
  const Tensor& like = *x.t;
  const Tensor& noise = on_device(arg[1], "noise", at::kFloat, like);
  const int64_t noise_ld = rows_of(noise, "noise", x.rows, x.n);
  profk_sampling how{};
  const int64_t rows[1] = {x.rows};
  if (THPVariable_Check(arg[2])) {
    without_tangent(THPVariable_Unpack(arg[2]), "temperature");
    how.temperature = static_cast<float*>(array(arg[2], "temperature", at::kFloat, like, rows));
  } else {
    how.all_temperature = static_cast<float>(number(arg[2]));
  }
  if (THPVariable_Check(arg[3]))
    how.top_k = static_cast<int32_t*>(array(arg[3], "top_k", at::kInt, like, rows));
  else
    how.all_top_k = static_cast<int32_t>(std::clamp<int64_t>(whole(arg[3]), 0, INT_MAX));
  if (THPVariable_Check(arg[4]))
    how.top_p = static_cast<float*>(array(arg[4], "top_p", at::kFloat, like, rows));
  else
    how.all_top_p = static_cast<float>(number(arg[4]));
  if (THPVariable_Check(arg[5]))
    how.min_p = static_cast<float*>(array(arg[5], "min_p", at::kFloat, like, rows));
  else
    how.all_min_p = static_cast<float>(number(arg[5]));
  const uint32_t* mask = nullptr;
  int64_t mask_ld = 0;
  if (arg[6] != Py_None) {
    const Tensor& m = on_device(arg[6], "mask", at::kInt, like);
    mask_ld = rows_of(m, "mask", x.rows, (x.n + 31) / 32);
    mask = static_cast<const uint32_t*>(m.data_ptr());
  }
  const Place place(arg[8], like);
  Tensor tokens, logprobs;
  if (arg[7] == Py_None) {
    tokens = place.empty(rows, at::kLong);
    logprobs = place.empty(rows, at::kFloat);
  } else {
    if (!PyTuple_Check(arg[7]) || PyTuple_GET_SIZE(arg[7]) != 2)
      refuse(PyExc_TypeError, "out must be a tuple of two tensors");
    array(PyTuple_GET_ITEM(arg[7], 0), "out[0]", at::kLong, like, rows);
    array(PyTuple_GET_ITEM(arg[7], 1), "out[1]", at::kFloat, like, rows);
    tokens = THPVariable_Unpack(PyTuple_GET_ITEM(arg[7], 0));
    logprobs = THPVariable_Unpack(PyTuple_GET_ITEM(arg[7], 1));
  }
  const int code = profk_sample_tokens(like.data_ptr(), x.type, x.rows, x.n, x.ld, static_cast<float*>(noise.data_ptr()),
                                       noise_ld, mask, mask_ld, &how, static_cast<int64_t*>(tokens.data_ptr()),
                                       static_cast<float*>(logprobs.data_ptr()), place.stream());
  return code == PROFK_OK ? tuple_of({tokens, logprobs}) : PyLong_FromLong(code);
  END_HANDLE_TH_ERRORS
}

// logits, k, score, normalize, bias, mask, balance, stream
PyObject* route(PyObject*, PyObject* const* arg, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  expect(count, 8);
  const Logits x = logits_of(arg[0]);
  const Tensor& like = *x.t;
  const int64_t k = whole(arg[1]);
  profk_routing how{static_cast<int>(whole(arg[2])), arg[3] == Py_True, nullptr, nullptr};
  if (arg[4] != Py_None) how.bias = static_cast<float*>(array(arg[4], "bias", at::kFloat, like, {x.n}));
  if (arg[5] != Py_None) how.mask = static_cast<uint8_t*>(array(arg[5], "mask", at::kBool, like, {x.rows}));
  if (k < 1 || k > x.n) refuse(PyExc_ValueError, "k must be in 1 .. experts");
  const Place place(arg[7], like);
  const Tensor gates = place.empty({x.rows, k}, at::kFloat), experts = place.empty({x.rows, k}, at::kLong),
               counts = place.empty({x.n}, at::kLong);
  Tensor loss;
  if (arg[6] == Py_True) loss = place.empty({}, at::kFloat);
  const int code = profk_route(like.data_ptr(), x.type, x.rows, x.n, x.ld, k, &how, static_cast<float*>(gates.data_ptr()),
                               static_cast<int64_t*>(experts.data_ptr()), static_cast<int64_t*>(counts.data_ptr()),
                               loss.defined() ? static_cast<float*>(loss.data_ptr()) : nullptr, place.stream());
  return code == PROFK_OK ? tuple_of({gates, experts, counts, loss}) : PyLong_FromLong(code);
  END_HANDLE_TH_ERRORS
}

// logits, experts, counts, score, normalize, grad_gates, grad_loss, out, stream
PyObject* route_backward(PyObject*, PyObject* const* arg, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  expect(count, 9);
  const Logits x = logits_of(arg[0]);
  const Tensor& like = *x.t;
  const Tensor& experts = on_device(arg[1], "routing.experts", at::kLong, like);
  if (experts.dim() != 2) refuse(PyExc_ValueError, "routing.experts must be 2-D");
  const int64_t k = experts.size(1);
  const auto* chosen = static_cast<const int64_t*>(array(arg[1], "routing.experts", at::kLong, like, {x.rows, k}));
  const profk_routing how{static_cast<int>(whole(arg[3])), arg[4] == Py_True, nullptr, nullptr};
  const float *grad_gates = nullptr, *grad_loss = nullptr;
  const int64_t* counts = nullptr;
  if (arg[5] != Py_None) {
    grad_gates = static_cast<float*>(array(arg[5], "grad_gates", at::kFloat, like, {x.rows, k}));
    without_tangent(THPVariable_Unpack(arg[5]), "grad_gates");
  }
  if (arg[6] != Py_None) {
    const Tensor& g = without_tangent(on_device(arg[6], "grad_loss", at::kFloat, like), "grad_loss");
    if (g.numel() != 1) refuse(PyExc_ValueError, "grad_loss must hold one element");
    grad_loss = static_cast<float*>(g.data_ptr());
    counts = static_cast<int64_t*>(array(arg[2], "routing.counts", at::kLong, like, {x.n}));
  }
  const Place place(arg[8], like);
  Tensor out;
  int64_t out_ld = x.n;
  if (arg[7] == Py_None) {
    out = place.empty({x.rows, x.n}, like.scalar_type());
  } else {
    out = on_device(arg[7], "out", like.scalar_type(), like);
    out_ld = rows_of(out, "out", x.rows, x.n);
  }
  const int code = profk_route_backward(like.data_ptr(), x.type, x.rows, x.n, x.ld, k, &how, chosen, counts, grad_gates,
                                        grad_loss, out.data_ptr(), out_ld, place.stream());
  return code == PROFK_OK ? THPVariable_Wrap(out) : PyLong_FromLong(code);
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"sample_tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(sample_tokens)), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(route)), METH_FASTCALL, nullptr},
    {"route_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(route_backward)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "profk_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_profk_torch() { return PyModule_Create(&module); }
