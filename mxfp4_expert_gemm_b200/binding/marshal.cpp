// Tensor arguments of the norms and 16-bit products, checked and handed to the C library.
//
// These calls take 2-10 us on the GPU at serving sizes; in Python their checks and allocations took
// as long again (a product 11.5 us a call, 4.7 of them in the library).  The rest of the binding
// stays in Python.  Functions take positional arguments from the wrappers in __init__.py and return
// (status, outputs ...).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "moe_mxfp4.h"

namespace {

// Addresses in the library that is in use (set by bind()).
struct Calls {
  decltype(&moe_norm) norm = nullptr;
  decltype(&moe_norm_backward) norm_backward = nullptr;
  decltype(&moe_norm_workspace_bytes) norm_workspace = nullptr;
  decltype(&moe_linear) linear = nullptr;
  decltype(&moe_linear_backward) linear_backward = nullptr;
  decltype(&moe_grouped_linear) grouped = nullptr;
  decltype(&moe_grouped_linear_backward) grouped_backward = nullptr;
  decltype(&moe_linear_workspace_bytes) workspace = nullptr;
} g_calls;

struct Bad {   // an argument error: a Python exception of this type
  PyObject* type;
  std::string text;
};

std::string str(const char* s) { return s; }

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Bad{PyExc_TypeError, str(name) + ": a CUDA tensor is required"};
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw Bad{PyExc_TypeError, str(name) + ": a CUDA tensor is required"};
  if (t.requires_grad() && c10::GradMode::is_enabled())
    TORCH_WARN_ONCE(name, " requires a gradient, but this call records no graph: its gradient comes from the _backward "
                    "call of the same name (with gradients off, as under torch.no_grad(), there is no such warning)");
  return t;
}

const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType type, int dev) {
  const at::Tensor& t = cuda_tensor(o, name);
  if (t.scalar_type() != type)
    throw Bad{PyExc_TypeError, str(name) + ": dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type)};
  if (t.get_device() != dev)
    throw Bad{PyExc_ValueError, str(name) + ": on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" + std::to_string(dev)};
  return t;
}

// The call's first tensor [rows, cols]; its device has to be the current one.
const at::Tensor& first_tensor(PyObject* o, const char* name) {
  const at::Tensor& t = cuda_tensor(o, name);
  const int now = c10::cuda::current_device();
  if (t.get_device() != now)
    throw Bad{PyExc_ValueError, str(name) + ": on cuda:" + std::to_string(t.get_device()) + ", but the current device is cuda:" +
                                    std::to_string(now)};
  if (t.dim() != 2 || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
    throw Bad{PyExc_ValueError, str(name) + ": shape " + shape_of(t) + ", expected [rows, columns]"};
  return t;
}

// Row stride of a [rows, cols] tensor whose columns are contiguous.
int64_t row_stride(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    throw Bad{PyExc_ValueError, str(name) + ": shape " + shape_of(t) + ", expected (" + std::to_string(rows) + ", " + std::to_string(cols) + ")"};
  if (t.stride(1) != 1 && cols != 1) throw Bad{PyExc_ValueError, str(name) + ": the columns of a row must be contiguous"};
  const int64_t ld = t.stride(0);
  return rows <= 1 && ld < cols ? cols : ld;
}

// Address of a contiguous tensor of the given shape (NULL for None).
void* flat(PyObject* o, const char* name, at::ScalarType type, int dev, at::IntArrayRef shape) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = checked(o, name, type, dev);
  if (t.sizes() != shape) throw Bad{PyExc_ValueError, str(name) + ": shape " + shape_of(t) + " is not the expected one"};
  if (!t.is_contiguous()) throw Bad{PyExc_ValueError, str(name) + ": must be contiguous"};
  return t.data_ptr();
}

struct Rows {   // a [rows, cols] operand: given, or made here
  at::Tensor t;
  void* p = nullptr;
  int64_t ld = 0;
  void make(const at::Tensor& like, int64_t rows, int64_t cols) {
    t = at::empty({rows, cols}, like.options());
    p = t.data_ptr();
    ld = cols;
  }
};
Rows rows_arg(PyObject* o, const char* name, at::ScalarType type, int dev, int64_t rows, int64_t cols) {
  Rows r;
  if (o == Py_None) return r;
  r.t = checked(o, name, type, dev);
  r.ld = row_stride(r.t, name, rows, cols);
  r.p = r.t.data_ptr();
  return r;
}

// The call's stream: the current one (None) or a given one, which then is torch's current stream while
// the call's outputs and scratch are made.  A block of another stream's pool may still be in use by
// kernels that this one does not wait for, and would go back there while this one still writes it.
struct Stream {
  void* raw = nullptr;
  c10::cuda::OptionalCUDAStreamGuard guard;
  Stream(PyObject* o, int dev) {
    if (o == Py_None) {
      raw = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    raw = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw python_error();
    guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), (c10::DeviceIndex)dev));
  }
};

struct Scratch {
  at::Tensor t;   // given (undefined: made here)
  void* p = nullptr;
  size_t n = 0;
  void take(size_t bytes, const at::Tensor& like) {
    if (!t.defined()) t = at::empty({(int64_t)((bytes + 3) / 4)}, like.options().dtype(at::kFloat));
    p = t.data_ptr();
    n = t.nbytes();
  }
};
Scratch scratch_arg(PyObject* o, int dev) {
  Scratch s;
  if (o == Py_None) return s;
  s.t = cuda_tensor(o, "ws");
  if (s.t.get_device() != dev || !s.t.is_contiguous())
    throw Bad{PyExc_ValueError, "ws: a contiguous tensor on cuda:" + std::to_string(dev) + " is required"};
  return s;
}

int32_t* status_of(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = checked(o, "status_word", at::kInt, dev);
  if (!t.is_contiguous()) throw Bad{PyExc_ValueError, "status_word: must be contiguous"};
  return static_cast<int32_t*>(t.data_ptr());
}

// Other Python threads run while this one allocates and launches: either may wait (for the driver, or
// for room in the stream's queue).  Nothing of Python is touched in its scope.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

int dtype_of(const at::Tensor& x, bool fp32) {
  switch (x.scalar_type()) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_F16;
    case at::kFloat:
      if (fp32) return MOE_DTYPE_F32;
    default: throw Bad{PyExc_TypeError, str("x: dtype ") + c10::toString(x.scalar_type()) + (fp32 ? "" : ": the products take bf16 or fp16 tensors")};
  }
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// (status, outputs): an output that was given is returned as it came.
PyObject* result(int status, std::initializer_list<std::pair<PyObject*, const at::Tensor*>> outs) {
  PyObject* r = PyTuple_New(1 + (Py_ssize_t)outs.size());
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (auto& o : outs) {
    PyObject* v;
    if (o.first && o.first != Py_None) v = Py_NewRef(o.first);
    else v = wrap(*o.second);
    PyTuple_SET_ITEM(r, i++, v);
  }
  return r;
}

float* f32_of(const at::Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; }

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v == 1;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw python_error();
  return v;
}
int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) throw python_error();
  return v;
}

#define BEGIN(count)                                                       \
  HANDLE_TH_ERRORS                                                         \
  if (n != count) {                                                        \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");         \
    return nullptr;                                                        \
  }                                                                        \
  if (!g_calls.workspace) {                                                \
    PyErr_SetString(PyExc_RuntimeError, "not bound to a library");         \
    return nullptr;                                                        \
  }                                                                        \
  try {
#define END                                                                \
  } catch (const Bad& b) {                                                 \
    PyErr_SetString(b.type, b.text.c_str());                               \
    return nullptr;                                                        \
  }                                                                        \
  END_HANDLE_TH_ERRORS

// x, w, b, kind, eps, y, want_stats, stream -> (status, y, mean, rstd)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(8)
  const at::Tensor& x = first_tensor(a[0], "x");
  const int dev = x.get_device(), dt = dtype_of(x, true), kind = (int)whole(a[3]);
  const int64_t T = x.size(0), d = x.size(1), ldx = row_stride(x, "x", T, d);
  const Stream stream(a[7], dev);
  float* w = static_cast<float*>(flat(a[1], "w", at::kFloat, dev, {d}));
  float* b = static_cast<float*>(flat(a[2], "b", at::kFloat, dev, {d}));
  Rows y = rows_arg(a[5], "y", x.scalar_type(), dev, T, d);
  const bool make_y = a[5] == Py_None, stats = truth(a[6]);
  const float eps = (float)number(a[4]);
  const auto call = g_calls.norm;
  at::Tensor mean, rstd;
  int st;
  {
    NoGil free;
    if (make_y) y.make(x, T, d);
    if (stats) {
      const auto o = x.options().dtype(at::kFloat);
      rstd = at::empty({T}, o);
      if (kind == MOE_NORM_LAYER) mean = at::empty({T}, o);
    }
    st = call(kind, dt, (int32_t)T, (int32_t)d, x.data_ptr(), ldx, w, b, eps, y.p, y.ld, f32_of(mean), f32_of(rstd),
              stream.raw);
  }
  return result(st, {{a[5], &y.t}, {nullptr, &mean}, {nullptr, &rstd}});
  END
}

// dy, x, w, mean, rstd, kind, dres, dx, need_dw, need_db, ws, stream -> (status, dx, dw, db)
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(12)
  const at::Tensor& x = first_tensor(a[1], "x");
  const auto type = x.scalar_type();
  const int dev = x.get_device(), dt = dtype_of(x, true), kind = (int)whole(a[5]);
  const int64_t T = x.size(0), d = x.size(1), ldx = row_stride(x, "x", T, d);
  if (a[0] == Py_None) throw Bad{PyExc_TypeError, "dy: a CUDA tensor is required"};
  const Stream stream(a[11], dev);
  const Rows dy = rows_arg(a[0], "dy", type, dev, T, d), dres = rows_arg(a[6], "dres", type, dev, T, d);
  float* w = static_cast<float*>(flat(a[2], "w", at::kFloat, dev, {d}));
  float* mean = static_cast<float*>(flat(a[3], "mean", at::kFloat, dev, {T}));
  float* rstd = static_cast<float*>(flat(a[4], "rstd", at::kFloat, dev, {T}));
  Rows dx = rows_arg(a[7], "dx", type, dev, T, d);
  const bool make_dx = a[7] == Py_None, need_dw = truth(a[8]), need_db = truth(a[9]);
  Scratch ws;
  if (need_dw || need_db) ws = scratch_arg(a[10], dev);
  const auto call = g_calls.norm_backward;
  const auto bytes = g_calls.norm_workspace;
  at::Tensor dw, db;
  int st;
  {
    NoGil free;
    const auto f32 = x.options().dtype(at::kFloat);
    if (make_dx) dx.make(x, T, d);
    if (need_dw) dw = at::empty({d}, f32);
    if (need_db) db = at::empty({d}, f32);
    if (need_dw || need_db) ws.take(bytes((int32_t)T, (int32_t)d), x);
    st = call(kind, dt, (int32_t)T, (int32_t)d, dy.p, dy.ld, x.data_ptr(), ldx, w, mean, rstd, dres.p, dres.ld, dx.p,
              dx.ld, f32_of(dw), f32_of(db), ws.p, ws.n, stream.raw);
  }
  return result(st, {{a[7], &dx.t}, {nullptr, &dw}, {nullptr, &db}});
  END
}

// The operands that both directions of a product have: x [rows, K], w [N, K] ([E, N, K] with offsets).
struct Product {
  const at::Tensor& x;
  const at::Tensor& w;
  int dev;
  int64_t rows, ldx, N, No;
  bool grouped;
  moe_linear_dims dims;
};
Product product_of(PyObject* xo, PyObject* wo, bool grouped, int fn, double limit) {
  const at::Tensor& x = first_tensor(xo, "x");
  const int dev = x.get_device(), dt = dtype_of(x, false);
  const at::Tensor& w = checked(wo, "w", x.scalar_type(), dev);
  const int64_t rows = x.size(0), K = x.size(1), ldx = row_stride(x, "x", rows, K);
  if (w.dim() != (grouped ? 3 : 2) || w.size(-1) != K)
    throw Bad{PyExc_ValueError, str("x [rows, K] and w ") + (grouped ? "[E, N, K]" : "[N, K]") + " are required"};
  if (!w.is_contiguous()) throw Bad{PyExc_ValueError, "w: must be contiguous"};
  const int64_t N = w.size(-2), E = grouped ? w.size(0) : 1, most = INT32_MAX;
  if (rows > most || K > most || N > most || E > most) throw Bad{PyExc_ValueError, "a dimension is beyond 2^31"};
  return Product{x, w, dev, rows, ldx, N, fn == MOE_FN_SWIGLU ? N / 2 : N, grouped,
                 moe_linear_dims{(int32_t)K, (int32_t)N, (int32_t)E, dt, fn, (float)limit}};
}

// x, w, offsets, bias, fn, limit, residual, y, z, want_z, status_word, stream -> (status, y, z)
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(12)
  const Product p = product_of(a[0], a[1], a[2] != Py_None, (int)whole(a[4]), number(a[5]));
  const auto type = p.x.scalar_type();
  const Stream stream(a[11], p.dev);
  const Rows res = rows_arg(a[6], "residual", type, p.dev, p.rows, p.No);
  Rows y = rows_arg(a[7], "y", type, p.dev, p.rows, p.No);
  void* zp = flat(a[8], "z", type, p.dev, {p.rows, p.N});
  const bool make_y = a[7] == Py_None, make_z = a[8] == Py_None && truth(a[9]);
  int32_t* status = status_of(a[10], p.dev);
  const int64_t E = p.dims.E;
  const float* bias = static_cast<float*>(p.grouped ? flat(a[3], "bias", at::kFloat, p.dev, {E, p.N})
                                                    : flat(a[3], "bias", at::kFloat, p.dev, {p.N}));
  const int32_t* off = p.grouped ? static_cast<int32_t*>(flat(a[2], "offsets", at::kInt, p.dev, {E + 1})) : nullptr;
  const Calls calls = g_calls;
  at::Tensor z;
  int st;
  {
    NoGil free;
    if (make_y) y.make(p.x, p.rows, p.No);
    if (make_z) {
      z = at::empty({p.rows, p.N}, p.x.options());
      zp = z.data_ptr();
    }
    st = p.grouped ? calls.grouped(&p.dims, (int32_t)p.rows, p.x.data_ptr(), p.ldx, p.w.data_ptr(), off, bias, y.p, y.ld,
                                   zp, status, stream.raw)
                   : calls.linear(&p.dims, (int32_t)p.rows, p.x.data_ptr(), p.ldx, p.w.data_ptr(), bias, res.p, res.ld,
                                  y.p, y.ld, zp, status, stream.raw);
  }
  return result(st, {{a[7], &y.t}, {a[8], &z}});
  END
}

// dy, x, w, offsets, z, fn, limit, dx, dw, need_dx, need_dw, need_db, ws, status_word, stream
// -> (status, dx, dw, db)
PyObject* product_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(15)
  const int fn = (int)whole(a[5]);
  const Product p = product_of(a[1], a[2], a[3] != Py_None, fn, number(a[6]));
  const auto type = p.x.scalar_type();
  if (a[0] == Py_None) throw Bad{PyExc_TypeError, "dy: a CUDA tensor is required"};
  const Stream stream(a[14], p.dev);
  const Rows dy = rows_arg(a[0], "dy", type, p.dev, p.rows, p.No);
  void* zp = nullptr;
  if (fn != MOE_FN_NONE) {
    if (a[4] == Py_None) throw Bad{PyExc_ValueError, "z: the forward pass's pre-activation is required with this fn"};
    zp = flat(a[4], "z", type, p.dev, {p.rows, p.N});
  }
  Rows dx = rows_arg(a[7], "dx", type, p.dev, p.rows, p.dims.K);
  void* dwp = flat(a[8], "dw", type, p.dev, p.w.sizes());
  const bool make_dx = a[7] == Py_None && truth(a[9]), make_dw = a[8] == Py_None && truth(a[10]);
  const bool want_db = truth(a[11]), want_ws = fn != MOE_FN_NONE || want_db;
  Scratch ws;
  if (want_ws) ws = scratch_arg(a[12], p.dev);
  int32_t* status = status_of(a[13], p.dev);
  const int32_t* off =
      p.grouped ? static_cast<int32_t*>(flat(a[3], "offsets", at::kInt, p.dev, {(int64_t)p.dims.E + 1})) : nullptr;
  const Calls calls = g_calls;
  at::Tensor dw, db;
  int st;
  {
    NoGil free;
    if (make_dx) dx.make(p.x, p.rows, p.dims.K);
    if (make_dw) {
      dw = at::empty(p.w.sizes(), p.w.options());
      dwp = dw.data_ptr();
    }
    if (want_db) db = at::empty(p.w.sizes().slice(0, p.w.dim() - 1), p.x.options().dtype(at::kFloat));
    if (want_ws) ws.take(calls.workspace(&p.dims, (int32_t)p.rows), p.x);
    st = p.grouped ? calls.grouped_backward(&p.dims, (int32_t)p.rows, dy.p, dy.ld, p.x.data_ptr(), p.ldx, p.w.data_ptr(),
                                            off, zp, dx.p, dx.ld, dwp, f32_of(db), ws.p, ws.n, status, stream.raw)
                   : calls.linear_backward(&p.dims, (int32_t)p.rows, dy.p, dy.ld, p.x.data_ptr(), p.ldx,
                                           p.w.data_ptr(), zp, dx.p, dx.ld, dwp, f32_of(db), ws.p, ws.n, status,
                                           stream.raw);
  }
  return result(st, {{a[7], &dx.t}, {a[8], &dw}, {nullptr, &db}});
  END
}

// The eight addresses of Calls, in order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    if (!p[i]) {
      PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  g_calls.norm = reinterpret_cast<decltype(g_calls.norm)>(p[0]);
  g_calls.norm_backward = reinterpret_cast<decltype(g_calls.norm_backward)>(p[1]);
  g_calls.norm_workspace = reinterpret_cast<decltype(g_calls.norm_workspace)>(p[2]);
  g_calls.linear = reinterpret_cast<decltype(g_calls.linear)>(p[3]);
  g_calls.linear_backward = reinterpret_cast<decltype(g_calls.linear_backward)>(p[4]);
  g_calls.grouped = reinterpret_cast<decltype(g_calls.grouped)>(p[5]);
  g_calls.grouped_backward = reinterpret_cast<decltype(g_calls.grouped_backward)>(p[6]);
  g_calls.workspace = reinterpret_cast<decltype(g_calls.workspace)>(p[7]);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm)), METH_FASTCALL, nullptr},
    {"norm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm_backward)), METH_FASTCALL, nullptr},
    {"product", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(product)), METH_FASTCALL, nullptr},
    {"product_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(product_backward)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
