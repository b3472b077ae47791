// The Python binding of the operators around the grouped products (dispatch,
// combine and its gradient, the router's gradient, 8-bit integers): the checks of
// a call, the memory of its results and the library's call in one step.  A
// decode-sized call takes a few microseconds on the GPU, less than the same steps
// took in Python (combine 4.6 us a call against 8.2, dispatch 7.0 and 12.1, a
// product of few rows 4.4 and 10.0; a launch alone is 3.3).
//
// Arguments come by position from the functions of the package, which document
// them.  Wrong types raise TypeError, wrong shapes and places ValueError, what the
// library refuses MoEError.
#include <Python.h>

#include <ATen/ops/empty_strided.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <tuple>

#include "moe.h"

namespace {

using at::ScalarType;
using at::Tensor;

// Of the package: the raw handle of a stream argument, memory of another stream
// than the current one, the library's error; of torch: the current stream.
PyObject *py_stream, *py_empty, *py_error, *py_current;

[[noreturn]] void raised() { throw python_error(); }

// A result of a Python call, released at the end of the scope.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {
    if (!p) raised();
  }
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref&) = delete;
};

// Other threads run Python meanwhile: an allocation or a launch may wait.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

const char* name_of(ScalarType t) { return c10::toString(t); }

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

// The library takes sizes, and divisors, as int32.
int32_t size32(int64_t v) {
  TORCH_CHECK_VALUE(v == (int32_t)v, "a size, or a divisor, does not fit 32 bits");
  return (int32_t)v;
}

// numpy's integers and integer tensors of one element too
int32_t integer(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(PyIndex_Check(o), name, " must be an integer");
  const Ref i(PyNumber_Index(o));
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i.p, &over);
  TORCH_CHECK_VALUE(!over, "a size, or a divisor, does not fit 32 bits");
  return size32(v);
}

ScalarType dtype(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPDtype_Check(o), name, " must be a torch.dtype");
  return ((THPDtype*)o)->scalar_type;
}

moe_out_t out_type(ScalarType t, const char* name) {
  TORCH_CHECK_TYPE(t == ScalarType::BFloat16 || t == ScalarType::Float, name,
                   " must be torch.bfloat16 or torch.float32, got ", name_of(t));
  return t == ScalarType::Float ? MOE_OUT_FP32 : MOE_OUT_BF16;
}

struct Matrix {
  void* p;
  int64_t stride;  // elements
};

// The tensors of one call: all on one GPU, whose current stream (or `given`) it
// runs on; results made here are from that stream's memory.
struct Call {
  c10::Device device;
  PyObject* given;
  void* stream = nullptr;

  Call(const Tensor& like, PyObject* stream_arg) : device(like.device()), given(stream_arg) {}

  void here(const Tensor& t, const char* name) const {
    TORCH_CHECK_VALUE(t.device() == device, name, " is on ", t.device(), ", the other operands on ", device);
  }

  // A contiguous tensor of this type and shape.
  void* need(const Tensor& t, const char* name, ScalarType type, at::IntArrayRef shape) const {
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", name_of(type), ", got ", name_of(t.scalar_type()));
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    here(t, name);
    return t.data_ptr();
  }
  void* need(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) const {
    return need(tensor(o, name), name, type, shape);
  }
  void* optional(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) const {
    return o == Py_None ? nullptr : need(o, name, type, shape);
  }

  // A [rows, width] operand whose rows may be strided; rows < 0: any number.
  // One row has no stride of its own, no row at all no address.
  Matrix matrix(const Tensor& t, const char* name, std::initializer_list<ScalarType> types, int64_t width,
                int64_t rows = -1) const {
    bool known = false;
    for (const ScalarType s : types) known = known || t.scalar_type() == s;
    TORCH_CHECK_TYPE(known, name, " must not be ", name_of(t.scalar_type()));
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(1) == width && (rows < 0 || t.size(0) == rows), name,
                      " must have ", width, " columns and the rows of the call, got ", t.sizes());
    TORCH_CHECK_VALUE(t.stride(1) == 1 || width <= 1, name, "'s rows must be contiguous");
    size32(t.size(0));
    here(t, name);
    return place(t);
  }
  static Matrix place(const Tensor& t) {
    return Matrix{t.data_ptr() ? t.data_ptr() : (void*)16, t.size(0) > 1 ? t.stride(0) : t.size(1)};
  }

  // Every given tensor has been looked at: the stream, before anything is made.
  void begin() {
    TORCH_CHECK_VALUE(device.is_cuda(), "the operands must be GPU tensors");
    if (given == Py_None) {
      const Ref index(PyLong_FromLong(device.index())), s(PyObject_CallOneArg(py_current, index.p));
      stream = PyLong_AsVoidPtr(s.p);
    } else {
      const Ref s(PyObject_CallOneArg(py_stream, given));
      stream = PyLong_AsVoidPtr(s.p);
    }
    if (PyErr_Occurred()) raised();
  }

  Tensor empty(at::IntArrayRef shape, ScalarType type, bool scratch = false) const {
    if (given == Py_None) {
      int64_t steps[2] = {1, 1};
      if (shape.size() == 2) steps[0] = shape[1];
      const NoGil released;
      return at::empty_strided(shape, at::IntArrayRef(steps, shape.size()), at::TensorOptions(device).dtype(type));
    }
    const Ref dims(PyTuple_New((Py_ssize_t)shape.size()));
    for (size_t i = 0; i < shape.size(); ++i) PyTuple_SET_ITEM(dims.p, i, PyLong_FromLongLong(shape[i]));
    const Ref t(PyObject_CallFunction(py_empty, "OOiOi", dims.p, (PyObject*)torch::getTHPDtype(type),
                                      (int)device.index(), given, (int)scratch));
    return THPVariable_Unpack(t.p);
  }

  template <typename F>
  void run(const char* name, const F& call) const {
    moe_status_t code;
    {
      const NoGil released;
      const c10::DeviceGuard guard(device);
      code = call(stream);
    }
    if (code == MOE_OK) return;
    const Ref e(PyObject_CallFunction(py_error, "si", name, (int)code));
    PyErr_SetObject(py_error, e.p);
    raised();
  }
};

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject* tuple(std::initializer_list<PyObject*> items) {  // takes the references
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_XDECREF(o);
  }
  return t;
}

void want(Py_ssize_t have, Py_ssize_t n) { TORCH_CHECK_TYPE(have == n, "takes ", n, " arguments, got ", have); }

const std::initializer_list<ScalarType> kRowTypes = {ScalarType::BFloat16, ScalarType::Float};

// x, ids, E, out, first_expert, stream
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 6);
  const Tensor& ids = tensor(a[1], "ids");
  TORCH_CHECK_VALUE(ids.dim() == 2, "ids must have shape (tokens, top_k)");
  moe_dispatch_args_t d = {};
  d.M = size32(ids.size(0));
  d.top_k = size32(ids.size(1));
  d.E = integer(a[2], "E");
  d.first_expert = integer(a[4], "first_expert");
  const int64_t P = size32((int64_t)d.M * d.top_k);
  Call call(ids, a[5]);
  d.ids = (const int32_t*)call.need(ids, "ids", ScalarType::Int, {d.M, d.top_k});
  const bool copy = a[0] != Py_None;
  TORCH_CHECK_VALUE(copy || a[3] == Py_None, "out needs x");
  Tensor x, out;
  if (copy) {
    x = tensor(a[0], "x");
    const int64_t esz = x.element_size();
    TORCH_CHECK_VALUE(x.dim() == 2 && (esz == 1 || esz == 2 || esz == 4) && !x.is_complex(),
                      "x must be a [tokens, H] tensor of a type of 1, 2 or 4 bytes");
    d.row_bytes = size32(x.size(1) * esz);
    const Matrix xm = call.matrix(x, "x", {x.scalar_type()}, x.size(1), d.M);
    d.x = xm.p;
    d.x_stride = xm.stride * esz;
    if (a[3] != Py_None) {
      out = tensor(a[3], "out");
      call.matrix(out, "out", {x.scalar_type()}, x.size(1), P);
    }
  }
  call.begin();
  if (copy) {
    if (!out.defined()) out = call.empty({P, x.size(1)}, x.scalar_type());
    const Matrix om = Call::place(out);
    d.rows = om.p;
    d.rows_stride = om.stride * x.element_size();
  }
  const Tensor offsets = call.empty({std::max(d.E, 0) + (int64_t)1}, ScalarType::Int);
  const Tensor positions = call.empty({d.M, d.top_k}, ScalarType::Int), pairs = call.empty({P}, ScalarType::Int);
  d.offsets = (int32_t*)offsets.data_ptr();
  d.positions = (int32_t*)positions.data_ptr();
  d.pairs = (int32_t*)pairs.data_ptr();
  d.workspace_bytes = moe_dispatch_workspace_size(d.M, d.top_k, d.E);
  Tensor workspace;
  if (d.workspace_bytes) {
    workspace = call.empty({(int64_t)d.workspace_bytes}, ScalarType::Byte, true);
    d.workspace = workspace.data_ptr();
  }
  call.run("moe_dispatch", [&](void* s) { return moe_dispatch(&d, s); });
  return tuple({wrap(out), wrap(offsets), wrap(positions), wrap(pairs)});
  END_HANDLE_TH_ERRORS
}

// rows, positions, weights, out, out_dtype, stream
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 6);
  const Tensor &rows = tensor(a[0], "rows"), &positions = tensor(a[1], "positions");
  TORCH_CHECK_VALUE(rows.dim() == 2 && positions.dim() == 2,
                    "rows must be a [rows, H] tensor and positions [tokens, top_k]");
  moe_combine_args_t c = {};
  c.R = size32(rows.size(0));
  c.H = size32(rows.size(1));
  c.M = size32(positions.size(0));
  c.top_k = size32(positions.size(1));
  size32((int64_t)c.M * c.top_k);
  Call call(rows, a[5]);
  const Matrix rm = call.matrix(rows, "rows", kRowTypes, c.H);
  c.rows = rm.p;
  c.rows_stride = rm.stride;
  c.rows_type = out_type(rows.scalar_type(), "rows");
  c.positions = (const int32_t*)call.need(positions, "positions", ScalarType::Int, {c.M, c.top_k});
  c.weights = (const float*)call.optional(a[2], "weights", ScalarType::Float, {c.M, c.top_k});
  Tensor out;
  ScalarType type = rows.scalar_type();
  if (a[3] != Py_None) {
    out = tensor(a[3], "out");
    call.matrix(out, "out", kRowTypes, c.H, c.M);
    type = out.scalar_type();
  } else if (a[4] != Py_None) {
    type = dtype(a[4], "out_dtype");
  }
  c.y_type = out_type(type, "out_dtype");
  call.begin();
  if (!out.defined()) out = call.empty({c.M, c.H}, type);
  const Matrix om = Call::place(out);
  c.y = om.p;
  c.y_stride = om.stride;
  call.run("moe_combine", [&](void* s) { return moe_combine(&c, s); });
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// dy, rows, positions, weights, drows, dweights, num_rows, out_dtype, stream
PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 9);
  const Tensor &dy = tensor(a[0], "dy"), &positions = tensor(a[2], "positions");
  TORCH_CHECK_VALUE(dy.dim() == 2 && positions.dim() == 2,
                    "dy must be a [tokens, H] tensor and positions [tokens, top_k]");
  moe_combine_grad_args_t c = {};
  c.M = size32(dy.size(0));
  c.H = size32(dy.size(1));
  c.top_k = size32(positions.size(1));
  const int64_t P = size32((int64_t)c.M * c.top_k);
  Call call(dy, a[8]);
  const Matrix dm = call.matrix(dy, "dy", kRowTypes, c.H);
  c.dy = dm.p;
  c.dy_stride = dm.stride;
  c.dy_type = out_type(dy.scalar_type(), "dy");
  c.positions = (const int32_t*)call.need(positions, "positions", ScalarType::Int, {c.M, c.top_k});
  c.weights = (const float*)call.optional(a[3], "weights", ScalarType::Float, {c.M, c.top_k});
  if (a[1] != Py_None) {
    const Tensor& rows = tensor(a[1], "rows");
    const Matrix rm = call.matrix(rows, "rows", kRowTypes, c.H);
    c.R = size32(rows.size(0));
    c.rows = rm.p;
    c.rows_stride = rm.stride;
    c.rows_type = out_type(rows.scalar_type(), "rows");
    if (a[6] != Py_None) {
      const int32_t num = integer(a[6], "num_rows");
      TORCH_CHECK_VALUE(num == c.R, "num_rows is ", num, ", rows has ", c.R);
    }
  } else {
    TORCH_CHECK_VALUE(a[5] == Py_None, "dweights needs rows");
    c.R = a[6] == Py_None ? (int32_t)P : integer(a[6], "num_rows");
    TORCH_CHECK_VALUE(c.R >= 0, "num_rows is negative");
  }
  Tensor drows, dweights;
  const bool give = a[4] != Py_None || a[7] != Py_None;  // no drows given and none to be made: not wanted
  TORCH_CHECK_VALUE(give || c.rows, "neither drows nor dweights: rows and out_dtype are both None");
  ScalarType type = ScalarType::BFloat16;
  if (a[4] != Py_None) {
    drows = tensor(a[4], "drows");
    call.matrix(drows, "drows", kRowTypes, c.H, c.R);
    type = drows.scalar_type();
  } else if (give) {
    type = dtype(a[7], "out_dtype");
  }
  c.drows_type = out_type(type, "out_dtype");
  if (a[5] != Py_None) {
    dweights = tensor(a[5], "dweights");
    call.need(dweights, "dweights", ScalarType::Float, {c.M, c.top_k});
  }
  call.begin();
  if (give) {
    if (!drows.defined()) drows = call.empty({c.R, c.H}, type);
    const Matrix om = Call::place(drows);
    c.drows = om.p;
    c.drows_stride = om.stride;
  }
  if (c.rows) {
    if (!dweights.defined()) dweights = call.empty({c.M, c.top_k}, ScalarType::Float);
    c.dweights = (float*)dweights.data_ptr();
  }
  call.run("moe_combine_grad", [&](void* s) { return moe_combine_grad(&c, s); });
  return tuple({wrap(drows), wrap(dweights)});
  END_HANDLE_TH_ERRORS
}

// ids, weights, dweights, E, out, stream
PyObject* route_topk_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 6);
  const Tensor& ids = tensor(a[0], "ids");
  TORCH_CHECK_VALUE(ids.dim() == 2, "ids must have shape (tokens, top_k)");
  const int32_t M = size32(ids.size(0)), k = size32(ids.size(1)), E = integer(a[3], "E");
  Call call(ids, a[5]);
  const auto* ip = (const int32_t*)call.need(ids, "ids", ScalarType::Int, {M, k});
  const auto* wp = (const float*)call.need(a[1], "weights", ScalarType::Float, {M, k});
  const auto* dp = (const float*)call.need(a[2], "dweights", ScalarType::Float, {M, k});
  Tensor out;
  if (a[4] != Py_None) {
    out = tensor(a[4], "out");
    call.need(out, "out", ScalarType::Float, {M, E});
  }
  call.begin();
  if (!out.defined()) out = call.empty({M, std::max(E, 0)}, ScalarType::Float);
  call.run("moe_route_topk_grad",
           [&](void* s) { return moe_route_topk_grad(ip, wp, dp, M, E, k, (float*)out.data_ptr(), s); });
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// Codes and scales of [rows, width], given or made here.
std::tuple<Tensor, Tensor> codes_of(Call& call, PyObject* codes, PyObject* scales, int64_t rows, int64_t width) {
  Tensor c, s;
  if (codes != Py_None) {
    c = tensor(codes, "codes");
    call.need(c, "codes", ScalarType::Char, {rows, width});
  }
  if (scales != Py_None) {
    s = tensor(scales, "scales");
    call.need(s, "scales", ScalarType::Float, {rows});
  }
  call.begin();
  if (!c.defined()) c = call.empty({rows, width}, ScalarType::Char);
  if (!s.defined()) s = call.empty({rows}, ScalarType::Float);
  return {c, s};
}

// x, codes, scales, stream
PyObject* quant_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 4);
  const Tensor& x = tensor(a[0], "x");
  TORCH_CHECK_VALUE(x.dim() == 2, "x must have shape (rows, K), got ", x.sizes());
  const int32_t M = size32(x.size(0)), K = size32(x.size(1));
  Call call(x, a[3]);
  const Matrix xm = call.matrix(x, "x", {ScalarType::BFloat16}, K);
  const auto [codes, scales] = codes_of(call, a[1], a[2], M, K);
  void *cp = codes.data_ptr(), *sp = scales.data_ptr();
  call.run("moe_quant_int8",
           [&](void* s) { return moe_quant_int8(xm.p, xm.stride, M, K, (int8_t*)cp, (float*)sp, s); });
  return tuple({wrap(codes), wrap(scales)});
  END_HANDLE_TH_ERRORS
}

// gu, row_weight, num_rows, codes, scales, stream
PyObject* swiglu_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 6);
  const Tensor& gu = tensor(a[0], "gu");
  TORCH_CHECK_VALUE(gu.dim() == 2 && gu.size(1) % 2 == 0, "gu must have shape (rows, 2*I), got ", gu.sizes());
  const int32_t R = size32(gu.size(0)), I = size32(gu.size(1) / 2);
  Call call(gu, a[5]);
  const Matrix gm = call.matrix(gu, "gu", {ScalarType::BFloat16}, 2 * (int64_t)I);
  const auto* wp = (const float*)call.optional(a[1], "row_weight", ScalarType::Float, {R});
  const auto* np = (const int32_t*)call.optional(a[2], "num_rows", ScalarType::Int, {1});
  const auto [codes, scales] = codes_of(call, a[3], a[4], R, I);
  void *cp = codes.data_ptr(), *sp = scales.data_ptr();
  call.run("moe_swiglu_int8",
           [&](void* s) { return moe_swiglu_int8(gm.p, gm.stride, wp, R, I, np, (int8_t*)cp, (float*)sp, s); });
  return tuple({wrap(codes), wrap(scales)});
  END_HANDLE_TH_ERRORS
}

// a, w, w_scale, offsets, out, a_scale, a_rows, a_div, out_rows, out_dtype, stream
PyObject* grouped_gemm_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 11);
  const Tensor &in = tensor(a[0], "input"), &w = tensor(a[1], "w");
  TORCH_CHECK_VALUE(w.dim() == 3, "the weights must be a tensor [E, N, K]");
  TORCH_CHECK_VALUE(in.dim() == 2, "input must be a [rows, K] tensor");
  moe_grouped_int8_args_t g = {};
  g.E = size32(w.size(0));
  g.N = size32(w.size(1));
  g.K = size32(w.size(2));
  const bool coded = in.scalar_type() == ScalarType::Char;
  TORCH_CHECK_VALUE(!coded || a[5] != Py_None, "int8 rows need a_scale");
  TORCH_CHECK_VALUE(coded || a[5] == Py_None, "a_scale goes with int8 rows");
  Call call(in, a[10]);
  // an operand's rows, chosen by ids
  auto rows_of = [&](const Tensor& t, const char* name, std::initializer_list<ScalarType> types, int64_t width,
                     PyObject* ids, int32_t div, int64_t R) {
    const Matrix m = call.matrix(t, name, types, width);
    moe_rows_t r = {m.p, m.stride, (int32_t)t.size(0), 1, nullptr};
    if (ids != Py_None) r.ids = (const int32_t*)call.need(ids, "the row ids", ScalarType::Int, {R});
    if (r.ids) r.div = div;
    return r;
  };
  g.R = size32(a[6] == Py_None ? in.size(0) : tensor(a[6], "a_rows").numel());
  const int32_t div = integer(a[7], "a_div");
  g.in = rows_of(in, "input", {coded ? ScalarType::Char : ScalarType::BFloat16}, g.K, a[6], div, g.R);
  if (coded) {
    g.in_scale = (const float*)call.need(a[5], "a_scale", ScalarType::Float, {in.size(0)});
    if (!g.in_scale) g.in_scale = (const float*)16;  // no rows at all
  }
  g.offsets = (const int32_t*)call.need(a[3], "offsets", ScalarType::Int, {g.E + (int64_t)1});
  g.w = (const int8_t*)call.need(w, "w", ScalarType::Char, {g.E, g.N, g.K});
  g.w_scale = (const float*)call.need(a[2], "w_scale", ScalarType::Float, {g.E, g.N});
  Tensor out;
  ScalarType type;
  if (a[4] != Py_None) {
    out = tensor(a[4], "out");
    type = out.scalar_type();
  } else {
    type = dtype(a[9], "out_dtype");
  }
  g.out_type = out_type(type, "out_dtype");
  if (out.defined()) g.out = rows_of(out, "out", {type}, g.N, a[8], 1, g.R);
  call.begin();
  if (!out.defined()) {
    out = call.empty({g.R, g.N}, type);
    g.out = rows_of(out, "out", {type}, g.N, a[8], 1, g.R);
  }
  Tensor workspace;
  if (!coded) {
    g.workspace_bytes = moe_grouped_int8_workspace_size(g.R, g.E, g.N, g.K, g.in.rows);
    if (g.workspace_bytes) {
      workspace = call.empty({(int64_t)g.workspace_bytes}, ScalarType::Byte, true);
      g.workspace = workspace.data_ptr();
    }
  }
  call.run("moe_grouped_gemm_int8", [&](void* s) { return moe_grouped_gemm_int8(&g, s); });
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// _stream, _empty, MoEError, the current stream of a device index.  The argument
// structs here are those of this version's header.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 4);
  TORCH_CHECK(moe_abi_version() == MOE_ABI_VERSION, "libmoe_mi355x.so has ABI version ", moe_abi_version(),
              ", the binding's compiled part is of version ", MOE_ABI_VERSION, ": rebuild them");
  PyObject** const at[4] = {&py_stream, &py_empty, &py_error, &py_current};
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*at[i], a[i]);
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define CALL(name) {#name, (PyCFunction)(void (*)())name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(init), CALL(dispatch), CALL(combine), CALL(combine_grad), CALL(route_topk_grad),
                         CALL(quant_int8), CALL(swiglu_int8), CALL(grouped_gemm_int8), {nullptr, nullptr, 0, nullptr}};
#undef CALL

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
