// The int8, row and token operators for torch tensors: checks of the arguments,
// allocation of the outputs and the call of the C entry point, in one step.
//
// Compiled because these operators take a few microseconds on the GPU at
// decode sizes, and the same checks in Python took about 10 us a call (two
// thirds of it attribute reads and ctypes conversions), which then set the
// time of every small call.  Nothing is computed here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <utility>

#include "fp8bg.h"
#include "fp8bg_internal.h"
#include "fp8bg_tokens.h"

namespace {

PyObject* g_error = nullptr;  // the package's exception: (status, what)

[[noreturn]] void fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw python_error();
}
[[noreturn]] void value_error(const std::string& what) { fail(PyExc_ValueError, what); }
[[noreturn]] void type_error(const std::string& what) { fail(PyExc_TypeError, what); }

void check_status(int status, const char* what) {
  if (status == FBG_SUCCESS) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", status, what)) {
    PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
    Py_DECREF(e);
  }
  throw python_error();
}

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int code(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kBFloat16: return FBG_OUT_BF16;
    case at::kHalf: return FBG_OUT_FP16;
    case at::kFloat: return FBG_OUT_FP32;
    default: type_error(std::string(name) + ": dtype " + c10::toString(t) + ", expected BFloat16, Half or Float");
  }
}

at::ScalarType dtype_arg(PyObject* o) {
  if (!THPDtype_Check(o)) type_error("out_dtype must be a torch dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

void check_kind(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type));
  if (t.sizes() != shape) value_error(std::string(name) + ": shape " + text(t.sizes()) + ", expected " + text(shape));
  if (t.device() != device) value_error(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
}

// A matrix with unit column stride; returns its row pitch in elements.
int64_t pitch(const at::Tensor& t, const char* name, at::ScalarType type, int64_t rows, int64_t cols, at::Device device) {
  check_kind(t, name, type, {rows, cols}, device);
  if (t.stride(1) != 1 && cols > 1) value_error(std::string(name) + " must have unit column stride");
  return t.stride(0);
}

// Matrices stacked so that their rows are all one distance apart, with unit
// column stride; returns that distance in elements.
int64_t stack_pitch(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  check_kind(t, name, type, shape, device);
  if (t.is_contiguous()) return t.size(2);
  const int64_t ld = t.stride(t.size(1) > 1 ? 1 : 0);
  if ((t.stride(2) != 1 && t.size(2) > 1) || (t.size(0) > 1 && t.stride(0) != t.size(1) * ld))
    value_error(std::string(name) + " must have unit column stride and rows at one distance through all of it");
  return ld;
}

void* whole(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  check_kind(t, name, type, shape, device);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

const at::Tensor& matrix(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2 || !t.is_cuda()) value_error(std::string(name) + " must be a 2-D CUDA tensor");
  return t;
}

// The device and the stream of a call.  With a stream of the caller's own the
// outputs are allocated as that stream's too, so that the allocator does not
// hand their memory to another stream while the call may still run.
class Launch {
 public:
  Launch(PyObject* stream, at::Device device) {
    if (stream == Py_None) {
      device_.emplace(device);
    } else {
      if (!THPStream_Check(stream)) type_error("stream must be a torch.cuda.Stream");
      const auto* s = reinterpret_cast<THPStream*>(stream);
      const auto st = c10::Stream::unpack3(s->stream_id, static_cast<c10::DeviceIndex>(s->device_index),
                                           static_cast<c10::DeviceType>(s->device_type));
      if (st.device() != device) value_error("stream is on " + st.device().str() + ", expected " + device.str());
      stream_.emplace(st);
    }
    raw_ = c10::hip::getCurrentHIPStream(device.index()).stream();
  }
  void* get() const { return raw_; }

 private:
  std::optional<c10::DeviceGuard> device_;
  std::optional<c10::StreamGuard> stream_;
  void* raw_ = nullptr;
};

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

// Two int32 outputs in one allocation, each a tensor of its own at a 16-byte
// boundary (5.3 us a small call, with an allocation each 5.7).
std::pair<at::Tensor, at::Tensor> make_two(at::IntArrayRef shape0, at::IntArrayRef shape1, at::Device device) {
  const int64_t n0 = (c10::multiply_integers(shape0) + 3) / 4 * 4, n1 = c10::multiply_integers(shape1);
  const at::Tensor both = make({n0 + n1}, at::kInt, device);
  const auto part = [&](at::IntArrayRef shape, int64_t at) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(both.storage()), both.key_set(), both.dtype());
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    return t;
  };
  return {part(shape0, 0), part(shape1, n0)};
}

// An int8 matrix whose rows start on 16-byte boundaries: the products read it
// in aligned chunks (16 x 4096 x 4001 takes 6.5 us, from rows 4001 bytes apart
// 12.8; 4096 x 4096 x 1000 53 and 59).
at::Tensor make_codes(int64_t rows, int64_t cols, at::Device device) {
  const int64_t ld = (cols + 15) / 16 * 16;
  at::Tensor q = make({rows, ld}, at::kChar, device);
  return ld == cols ? q : q.narrow(1, 0, cols);
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}

// (A, a_s, B, b_s, bias, out_dtype, out, stream)
PyObject* int8_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const at::Tensor &A = matrix(v[0], "A"), &B = matrix(v[2], "B");
  const int64_t M = A.size(0), K = A.size(1), N = B.size(0);
  const at::Device dev = A.device();
  const int64_t lda = pitch(A, "A", at::kChar, M, K, dev), ldb = pitch(B, "B", at::kChar, N, K, dev);
  const auto* a_s = static_cast<const float*>(whole(tensor(v[1], "a_s"), "a_s", at::kFloat, {M}, dev));
  const auto* b_s = static_cast<const float*>(whole(tensor(v[3], "b_s"), "b_s", at::kFloat, {N}, dev));
  const auto* bias =
      v[4] == Py_None ? nullptr : static_cast<const float*>(whole(tensor(v[4], "bias"), "bias", at::kFloat, {N}, dev));
  const at::ScalarType type = dtype_arg(v[5]);
  const int out_code = code(type, "out_dtype");
  const Launch launch(v[7], dev);
  const at::Tensor out = v[6] == Py_None ? make({M, N}, type, dev) : tensor(v[6], "out");
  const int64_t ldc = v[6] == Py_None ? N : pitch(out, "out", type, M, N, dev);
  check_status(fbg_int8_gemm(A.data_ptr(), lda, a_s, B.data_ptr(), ldb, b_s, bias, out.data_ptr(), ldc, M, N, K,
                             out_code, launch.get()),
               "fbg_int8_gemm");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (A, a_s, B, b_s, offsets, out_dtype, out, stream)
PyObject* int8_grouped_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const at::Tensor &A = matrix(v[0], "A"), &B = tensor(v[2], "B");
  if (B.dim() != 3) value_error("B must be 3-D [E, N, K]");
  const int64_t M = A.size(0), K = A.size(1), E = B.size(0), N = B.size(1);
  const at::Device dev = A.device();
  const int64_t lda = pitch(A, "A", at::kChar, M, K, dev);
  const auto* a_s = static_cast<const float*>(whole(tensor(v[1], "a_s"), "a_s", at::kFloat, {M}, dev));
  const int64_t ldb = stack_pitch(B, "B", at::kChar, {E, N, K}, dev);
  const auto* b_s = static_cast<const float*>(whole(tensor(v[3], "b_s"), "b_s", at::kFloat, {E, N}, dev));
  const auto* offsets =
      static_cast<const int32_t*>(whole(tensor(v[4], "offsets"), "offsets", at::kInt, {E + 1}, dev));
  const at::ScalarType type = dtype_arg(v[5]);
  const int out_code = code(type, "out_dtype");
  const Launch launch(v[7], dev);
  const at::Tensor out = v[6] == Py_None ? make({M, N}, type, dev) : tensor(v[6], "out");
  const int64_t ldc = v[6] == Py_None ? N : pitch(out, "out", type, M, N, dev);
  check_status(fbg::int8_grouped_gemm(A.data_ptr(), lda, a_s, B.data_ptr(), ldb, b_s, out.data_ptr(), ldc, offsets, E,
                                      M, N, K, out_code, launch.get()),
               "fbg_int8_grouped_gemm");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (x, q, scale, stream) -> (q, scale)
PyObject* quantize_tokens(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 4);
  const at::Tensor& x = matrix(v[0], "x");
  const int64_t M = x.size(0), K = x.size(1);
  const at::Device dev = x.device();
  const int in_code = code(x.scalar_type(), "x");
  const int64_t ldx = pitch(x, "x", x.scalar_type(), M, K, dev);
  const Launch launch(v[3], dev);
  const at::Tensor q = v[1] == Py_None ? make_codes(M, K, dev) : tensor(v[1], "q");
  const int64_t ldq = pitch(q, "q", at::kChar, M, K, dev);
  const at::Tensor s = v[2] == Py_None ? make({M}, at::kFloat, dev) : tensor(v[2], "scale");
  auto* scale = static_cast<float*>(whole(s, "scale", at::kFloat, {M}, dev));
  check_status(fbg_quantize_tokens(x.data_ptr(), ldx, in_code, M, K, q.data_ptr(), ldq, scale, launch.get()),
               "fbg_quantize_tokens");
  return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(s));
  END_HANDLE_TH_ERRORS
}

// (h, x, post_weight, gate, pre_weight, residual_scale, eps, weight_offset,
//  quantize, stream) -> (r, y) or (r, codes, scale)
PyObject* block_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 10);
  const at::Tensor& h = matrix(v[0], "h");
  const int64_t M = h.size(0), D = h.size(1);
  const at::Device dev = h.device();
  const at::ScalarType type = h.scalar_type();
  const int io = code(type, "h");
  const int64_t ldh = pitch(h, "h", type, M, D, dev);

  const void* x = nullptr;
  int64_t ldx = 0;
  if (v[1] != Py_None) {
    const at::Tensor& t = tensor(v[1], "x");
    ldx = pitch(t, "x", type, M, D, dev);
    x = t.data_ptr();
  }
  const void* gate = nullptr;
  int64_t gate_row = 0, gate_col = 0;
  if (v[3] != Py_None) {
    const at::Tensor& t = tensor(v[3], "gate");
    const int64_t dim = t.dim(), cols = dim > 0 ? t.size(dim - 1) : 0, rows = dim == 2 ? t.size(0) : 1;
    if (dim < 1 || dim > 2 || (rows != 1 && rows != M) || (cols != 1 && cols != D))
      value_error("gate: shape " + text(t.sizes()) + " does not broadcast to " + text({M, D}));
    check_kind(t, "gate", type, t.sizes(), dev);
    gate = t.data_ptr();
    gate_row = rows == 1 ? 0 : t.stride(0);
    gate_col = cols == 1 ? 0 : t.stride(dim - 1);
  }
  at::ScalarType wtype = type;
  const void *post = nullptr, *pre = nullptr;
  if (v[2] != Py_None || v[4] != Py_None) {
    wtype = tensor(v[2] != Py_None ? v[2] : v[4], "weights").scalar_type();
    if (wtype != type && wtype != at::kFloat)
      type_error(std::string("weights: dtype ") + c10::toString(wtype) + ", expected " + c10::toString(type) + " or Float");
    if (v[2] != Py_None) post = whole(tensor(v[2], "post_weight"), "post_weight", wtype, {D}, dev);
    if (v[4] != Py_None) pre = whole(tensor(v[4], "pre_weight"), "pre_weight", wtype, {D}, dev);
  }
  const bool second = v[4] != Py_None;
  const double residual_scale = PyFloat_AsDouble(v[5]), eps = PyFloat_AsDouble(v[6]), offset = PyFloat_AsDouble(v[7]);
  if (PyErr_Occurred()) throw python_error();
  int quant = FBG_QUANT_NONE;
  if (v[8] != Py_None) {
    const char* s = PyUnicode_Check(v[8]) ? PyUnicode_AsUTF8(v[8]) : "";
    if (!s) throw python_error();
    quant = std::string(s) == "int8" ? FBG_QUANT_INT8 : std::string(s) == "fp8" ? FBG_QUANT_FP8 : -1;
    if (quant < 0) value_error("quantize must be None, \"int8\" or \"fp8\"");
    if (!second) value_error("quantize needs pre_weight");
  }
  const Launch launch(v[9], dev);
  const at::Tensor r = make({M, D}, type, dev);
  at::Tensor y, scale;
  if (second) {
    y = quant == FBG_QUANT_NONE ? make({M, D}, type, dev)
        : quant == FBG_QUANT_INT8 ? make_codes(M, D, dev)
                                  : make({M, D}, at::kFloat8_e4m3fn, dev);
    if (quant == FBG_QUANT_INT8) scale = make({M}, at::kFloat, dev);
    if (quant == FBG_QUANT_FP8) scale = make({M, D / 128}, at::kFloat, dev);
  }
  check_status(
      fbg_block_norm(h.data_ptr(), ldh, x, ldx, gate, gate_row, gate_col, post, pre, io, code(wtype, "weights"), M, D,
                     (float)residual_scale, (float)eps, (float)offset, r.data_ptr(), D, second ? y.data_ptr() : nullptr,
                     second ? y.stride(0) : D, scale.defined() ? static_cast<float*>(scale.data_ptr()) : nullptr,
                     quant, launch.get()),
      "fbg_block_norm");
  PyObject* yo = second ? THPVariable_Wrap(y) : Py_NewRef(Py_None);
  return scale.defined() ? Py_BuildValue("(NNN)", THPVariable_Wrap(r), yo, THPVariable_Wrap(scale))
                         : Py_BuildValue("(NN)", THPVariable_Wrap(r), yo);
  END_HANDLE_TH_ERRORS
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// Forward only.  A tensor of the caller's that is written (None: the call makes its own)
// would stand in a graph that leaves this step out, with gradients that miss it: as
// torch refuses `out=` there, so is that here.
void check_forward_only(std::initializer_list<PyObject*> written, std::initializer_list<PyObject*> read) {
  bool writes = false;
  for (PyObject* o : written) writes |= o != Py_None;
  if (!writes || !at::GradMode::is_enabled()) return;
  for (const auto& list : {written, read})
    for (PyObject* o : list)
      if (o != Py_None && THPVariable_Unpack(o).requires_grad())
        value_error("the operator has no backward: it does not write into a tensor of the caller's while one of its "
                    "tensors requires a gradient (use torch.no_grad())");
}

// What was saved of them for a backward pass is out of date.
void count_writes(std::initializer_list<PyObject*> written) {
  for (PyObject* o : written) {
    if (o == Py_None) continue;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
}

// Which of two words `o` is.
int one_of(PyObject* o, const char* name, const char* zero, const char* one) {
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : "";
  if (!s) throw python_error();
  if (std::string(s) == zero) return 0;
  if (std::string(s) == one) return 1;
  value_error(std::string(name) + " must be \"" + zero + "\" or \"" + one + "\"");
}

// (logits, topk, score, bias, groups, topk_groups, group_score, renormalize,
//  scale, mask, weights, experts, stream) -> (weights, experts)
PyObject* route_experts(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 13);
  const at::Tensor& logits = matrix(v[0], "logits");
  const int64_t T = logits.size(0), E = logits.size(1), topk = integer(v[1]);
  const at::Device dev = logits.device();
  const int in_code = code(logits.scalar_type(), "logits");
  const int64_t ld = pitch(logits, "logits", logits.scalar_type(), T, E, dev);
  if (topk < 0) value_error("topk must not be negative");
  const int score = one_of(v[2], "score", "softmax", "sigmoid") ? FBG_SCORE_SIGMOID : FBG_SCORE_SOFTMAX;
  const auto* bias =
      v[3] == Py_None ? nullptr : static_cast<const float*>(whole(tensor(v[3], "bias"), "bias", at::kFloat, {E}, dev));
  const int64_t groups = integer(v[4]), topk_groups = integer(v[5]);
  const int group_score = one_of(v[6], "group_score", "max", "top2") ? FBG_GROUP_TOP2 : FBG_GROUP_MAX;
  const int renormalize = PyObject_IsTrue(v[7]);
  const double scale = PyFloat_AsDouble(v[8]);
  if (PyErr_Occurred()) throw python_error();
  const uint8_t* mask = nullptr;
  if (v[9] != Py_None) {
    const at::Tensor& m = tensor(v[9], "mask");
    const at::ScalarType type = m.scalar_type() == at::kByte ? at::kByte : at::kBool;
    mask = static_cast<const uint8_t*>(whole(m, "mask", type, {T}, dev));
  }
  const Launch launch(v[12], dev);
  const at::Tensor w = v[10] == Py_None ? make({T, topk}, at::kFloat, dev) : tensor(v[10], "weights");
  const at::Tensor e = v[11] == Py_None ? make({T, topk}, at::kInt, dev) : tensor(v[11], "experts");
  auto* weights = static_cast<float*>(whole(w, "weights", at::kFloat, {T, topk}, dev));
  auto* experts = static_cast<int32_t*>(whole(e, "experts", at::kInt, {T, topk}, dev));
  check_forward_only({v[10], v[11]}, {v[0], v[3]});
  check_status(fbg_route_experts(logits.data_ptr(), ld, in_code, T, E, topk, score, bias, groups, topk_groups,
                                 group_score, renormalize, (float)scale, mask, weights, experts, launch.get()),
               "fbg_route_experts");
  count_writes({v[10], v[11]});
  return Py_BuildValue("(NN)", THPVariable_Wrap(w), THPVariable_Wrap(e));
  END_HANDLE_TH_ERRORS
}

// (experts, E, x, x_scale, first_expert, rows, row_scale, stream)
//  -> (rows, row_scale or None, offsets, slots)
PyObject* dispatch_tokens(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const at::Tensor &experts = matrix(v[0], "experts"), &x = matrix(v[2], "x");
  const int64_t T = experts.size(0), topk = experts.size(1), E = integer(v[1]), K = x.size(1);
  const at::Device dev = x.device();
  if (E < 0) value_error("E must not be negative");
  const auto* ids = static_cast<const int32_t*>(whole(experts, "experts", at::kInt, {T, topk}, dev));
  const at::ScalarType type = x.scalar_type();
  const int64_t ldx = pitch(x, "x", type, T, K, dev);
  const int64_t size = x.element_size();
  if (size != 1 && size != 2 && size != 4) type_error("x: elements of 1, 2 or 4 bytes expected");
  const float* x_scale = nullptr;
  int64_t S = 0;
  at::DimVector scale_shape;
  if (v[3] != Py_None) {
    const at::Tensor& t = tensor(v[3], "x_scale");
    if (t.dim() != 1 && t.dim() != 2) value_error("x_scale must be [T] or [T, S]");
    S = t.dim() == 1 ? 1 : t.size(1);
    scale_shape.push_back(T);
    if (t.dim() == 2) scale_shape.push_back(S);
    x_scale = static_cast<const float*>(whole(t, "x_scale", at::kFloat, scale_shape, dev));
    scale_shape[0] = T * topk;
  }
  const int64_t first = integer(v[4]);
  if (E > fbg::kMaxRouted) check_status(FBG_ERROR_UNSUPPORTED, "fbg_dispatch_tokens");
  const Launch launch(v[7], dev);
  const at::Tensor rows = v[5] != Py_None      ? tensor(v[5], "rows")
                          : type == at::kChar ? make_codes(T * topk, K, dev)
                                              : make({T * topk, K}, type, dev);
  const int64_t ldrows = pitch(rows, "rows", type, T * topk, K, dev);
  at::Tensor row_scale;
  if (v[3] != Py_None) {
    row_scale = v[6] == Py_None ? make(scale_shape, at::kFloat, dev) : tensor(v[6], "row_scale");
    whole(row_scale, "row_scale", at::kFloat, scale_shape, dev);
  } else if (v[6] != Py_None) {
    value_error("row_scale needs x_scale");
  }
  check_forward_only({v[5], v[6]}, {v[2], v[3]});
  const auto [offsets, slots] = make_two({E + 1}, {T, topk}, dev);
  check_status(fbg_dispatch_tokens(ids, T, topk, first, E, x.data_ptr(), ldx, K, (int)size, x_scale, S,
                                   rows.data_ptr(), ldrows,
                                   row_scale.defined() ? static_cast<float*>(row_scale.data_ptr()) : nullptr,
                                   static_cast<int32_t*>(offsets.data_ptr()), static_cast<int32_t*>(slots.data_ptr()),
                                   launch.get()),
               "fbg_dispatch_tokens");
  count_writes({v[5], v[6]});
  PyObject* so = row_scale.defined() ? THPVariable_Wrap(row_scale) : Py_NewRef(Py_None);
  return Py_BuildValue("(NNNN)", THPVariable_Wrap(rows), so, THPVariable_Wrap(offsets), THPVariable_Wrap(slots));
  END_HANDLE_TH_ERRORS
}

// (rows, slots, weights, base, out_dtype, out, stream)
PyObject* combine_experts(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 7);
  const at::Tensor &rows = matrix(v[0], "rows"), &slots = matrix(v[1], "slots");
  const int64_t R = rows.size(0), D = rows.size(1), T = slots.size(0), topk = slots.size(1);
  const at::Device dev = rows.device();
  const at::ScalarType type = rows.scalar_type();
  const int in_code = code(type, "rows");
  const int64_t ldrows = pitch(rows, "rows", type, R, D, dev);
  const auto* at_slots = static_cast<const int32_t*>(whole(slots, "slots", at::kInt, {T, topk}, dev));
  const auto* weights =
      static_cast<const float*>(whole(tensor(v[2], "weights"), "weights", at::kFloat, {T, topk}, dev));
  const at::ScalarType out_type = v[4] == Py_None ? v[5] == Py_None ? type : tensor(v[5], "out").scalar_type() : dtype_arg(v[4]);
  const int out_code = code(out_type, "out_dtype");
  const void* base = nullptr;
  int64_t ldbase = 0;
  int base_code = in_code;
  if (v[3] != Py_None) {
    const at::Tensor& t = tensor(v[3], "base");
    const at::ScalarType bt = t.scalar_type();
    if (bt != type && bt != out_type)
      type_error(std::string("base: dtype ") + c10::toString(bt) + ", expected " + c10::toString(type) + " or " +
                 c10::toString(out_type));
    ldbase = pitch(t, "base", bt, T, D, dev);
    base = t.data_ptr();
    base_code = code(bt, "base");
  }
  const Launch launch(v[6], dev);
  const at::Tensor out = v[5] == Py_None ? make({T, D}, out_type, dev) : tensor(v[5], "out");
  const int64_t ldout = pitch(out, "out", out_type, T, D, dev);
  check_forward_only({v[5]}, {v[0], v[2], v[3]});
  check_status(fbg_combine_experts(rows.data_ptr(), ldrows, in_code, R, at_slots, weights, base, ldbase, base_code,
                                   out.data_ptr(), ldout, out_code, T, topk, D, launch.get()),
               "fbg_combine_experts");
  count_writes({v[5]});
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (y, x, A, B, adapters, scales, out, stream)
PyObject* add_adapters(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const at::Tensor &y = matrix(v[0], "y"), &x = matrix(v[1], "x"), &A = tensor(v[2], "A"), &B = tensor(v[3], "B");
  if (A.dim() != 3 || B.dim() != 3) value_error("A must be [L, R, K] and B [L, N, R]");
  const int64_t M = y.size(0), N = y.size(1), K = x.size(1), L = A.size(0), R = A.size(1);
  const at::Device dev = y.device();
  const at::ScalarType type = x.scalar_type(), out_type = y.scalar_type();
  const int in_code = code(type, "x"), out_code = code(out_type, "y");
  if (in_code == FBG_OUT_FP32) type_error("x: dtype Float, expected BFloat16 or Half");
  const int64_t ldy = pitch(y, "y", out_type, M, N, dev), ldx = pitch(x, "x", type, M, K, dev);
  const void* pa = whole(A, "A", type, {L, R, K}, dev);
  const void* pb = whole(B, "B", type, {L, N, R}, dev);
  const auto* ids = static_cast<const int32_t*>(whole(tensor(v[4], "adapters"), "adapters", at::kInt, {M}, dev));
  const auto* scales = v[5] == Py_None
                           ? nullptr
                           : static_cast<const float*>(whole(tensor(v[5], "scales"), "scales", at::kFloat, {L}, dev));
  const size_t need = fbg_add_adapters_workspace_size(M, N, K, R);
  if (need == (size_t)-1) check_status(FBG_ERROR_UNSUPPORTED, "fbg_add_adapters");
  const Launch launch(v[7], dev);
  const at::Tensor out = v[6] == Py_None ? y : tensor(v[6], "out");
  const int64_t ldout = pitch(out, "out", out_type, M, N, dev);
  PyObject* const written = v[6] == Py_None ? v[0] : v[6];
  check_forward_only({written}, {v[0], v[1], v[2], v[3], v[5]});
  const at::Tensor work = need ? make({(int64_t)need}, at::kByte, dev) : at::Tensor();
  check_status(fbg_add_adapters(y.data_ptr(), ldy, x.data_ptr(), ldx, pa, pb, ids, scales, out.data_ptr(), ldout, M, N,
                                K, R, L, in_code, out_code, need ? work.data_ptr() : nullptr, need, launch.get()),
               "fbg_add_adapters");
  count_writes({written});
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"int8_gemm", FAST(int8_gemm), nullptr},
                         {"int8_grouped_gemm", FAST(int8_grouped_gemm), nullptr},
                         {"quantize_tokens", FAST(quantize_tokens), nullptr},
                         {"block_norm", FAST(block_norm), nullptr},
                         {"route_experts", FAST(route_experts), nullptr},
                         {"dispatch_tokens", FAST(dispatch_tokens), nullptr},
                         {"combine_experts", FAST(combine_experts), nullptr},
                         {"add_adapters", FAST(add_adapters), nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8bg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8bg_torch() { return PyModule_Create(&module); }
