// Native half of the MX4 binding (block_diagonal_linear_b200/mx4.py): checks the tensors of a call, takes its
// outputs and workspace from torch's allocator on the current stream and calls the C entry point.  A decoding
// step's kernels take a few microseconds, so what a call costs on the host is what a step costs; in Python
// the same checks took 3 us longer (one token through 4096 -> 4096: 8.3 us a call, 5.3 from here; an odd
// backward 25.0 and 16.3).
//
// Every function runs on its tensors' device and that device's current stream.  A quantised tensor comes as
// the bytes of a Quantised (mx4.py keeps its memory alive).  Wrong tensors raise ValueError, error codes of the
// library MonarchError (through the callable given to init).
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "../../include/monarch.h"

namespace {

struct Quantised {
  int64_t codes, scales;  // addresses
  int64_t rows, nblocks, cols, by_block, dtype;
  int64_t device;
};

// Addresses of the library's entry points, in the order that mx4.py gives them.
struct Library {
  size_t (*code_bytes)(const monarch_mx4_dims*);
  size_t (*scale_bytes)(const monarch_mx4_dims*);
  int (*quantise)(const void*, const monarch_mx4_dims*, void*, void*, void*);
  int (*dequantise)(const void*, const void*, const monarch_mx4_dims*, void*, void*);
  size_t (*wfwd_bytes)(const monarch_mx4_linear_dims*);
  size_t (*bwd_bytes)(const monarch_mx4_linear_dims*);
  int (*fwd)(const void*, const void*, const void*, const void*, const void*, const monarch_mx4_linear_dims*, void*, void*);
  int (*wfwd)(const void*, const void*, const void*, const void*, const monarch_mx4_linear_dims*, void*, void*, size_t, void*);
  int (*bwd)(const void*, const void*, const void*, const void*, const void*, const monarch_mx4_linear_dims*, void*, void*, void*,
             void*, size_t, void*);
  size_t (*monarch_bytes)(const monarch_dims*);
  int (*monarch_fwd)(const void*, const void*, const void*, const void*, const void*, const monarch_dims*, void*, void*, size_t, void*);
};
Library lib;
PyObject* check = nullptr;  // check(name, code): raises MonarchError for a code other than 0

[[noreturn]] void bad(const std::string& what) { throw c10::ValueError({__func__, __FILE__, (uint32_t)__LINE__}, what); }

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}
at::ScalarType torch_type(int64_t dtype) { return dtype == MONARCH_BF16 ? at::kBFloat16 : at::kFloat; }
const char* type_name(at::ScalarType t) { return t == at::kBFloat16 ? "bfloat16" : "float32"; }

// A contiguous CUDA tensor.
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || !t.is_contiguous()) bad("Monarch kernels take contiguous CUDA tensors");
  return t;
}
int64_t dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return MONARCH_BF16;
  if (t.scalar_type() == at::kFloat) return MONARCH_F32;
  bad(std::string(name) + " is neither bfloat16 nor float32");
}
void expect(const at::Tensor& t, const char* name, at::IntArrayRef shape, int64_t dtype, int64_t device) {
  if (t.sizes() != shape || t.scalar_type() != torch_type(dtype))
    bad(std::string(name) + " must be " + type_name(torch_type(dtype)) + " of shape " + shape_of(shape) + ", its shape is " + shape_of(t.sizes()));
  if (t.get_device() != device)
    bad(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", not cuda:" + std::to_string(device) + ": one call takes one device's");
}
const Quantised& quantised(PyObject* o, const char* name) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != sizeof(Quantised)) bad(std::string(name) + " must be an Mx4");
  const Quantised& q = *(const Quantised*)PyBytes_AS_STRING(o);
  if (q.device < 0) bad(std::string(name) + " is not on a CUDA device");
  return q;
}
void on_device(const Quantised& q, const char* name, int64_t device) {
  if (q.device != device)
    bad(std::string(name) + " is not on cuda:" + std::to_string(device) + ": one call takes one device's");
}
// The caller's tensor, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, int64_t dtype, int64_t device) {
  if (o == Py_None)
    return at::empty(shape, at::TensorOptions().dtype(torch_type(dtype)).device(at::kCUDA, (c10::DeviceIndex)device));
  const at::Tensor& t = tensor(o, name);
  expect(t, name, shape, dtype, device);
  return t;
}
at::Tensor bytes_on(int64_t n, int64_t device) {
  return at::empty({n}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)device));
}
struct Workspace {
  at::Tensor hold;
  void* p = nullptr;
  size_t n = 0;
  Workspace(PyObject* o, size_t need, int64_t device) {
    if (o == Py_None) {
      if (need == 0) return;
      hold = bytes_on((int64_t)need, device);
    } else {
      hold = tensor(o, "workspace");
      if (hold.get_device() != device) bad("the workspace is on another device");
    }
    p = hold.data_ptr();
    n = (size_t)hold.nbytes();
  }
};
bool truth(PyObject* o, const char* name) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) {
    PyErr_Clear();
    bad(std::string(name) + " must be true or false");
  }
  return r == 1;
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// f(stream) with `device` the current one, without the interpreter lock; raises on an error code.
template <class F>
void call(const char* name, int64_t device, F&& f) {
  int rc;
  {
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != device) guard.set_index((c10::DeviceIndex)device);
    void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    Py_BEGIN_ALLOW_THREADS;
    rc = f(stream);
    Py_END_ALLOW_THREADS;
  }
  if (rc != 0) {
    PyObject* r = PyObject_CallFunction(check, "si", name, rc);
    Py_XDECREF(r);
    throw python_error();
  }
}
void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) bad("wrong number of arguments");
}
monarch_mx4_dims dims_of(const Quantised& q, int64_t dtype) {
  return monarch_mx4_dims{q.rows, (int32_t)q.nblocks, (int32_t)q.cols, (int32_t)q.by_block, (int32_t)dtype};
}
int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) bad(std::string(name) + " is too large");
  return (int32_t)v;
}

// init(addresses, check)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 2);
  constexpr Py_ssize_t count = sizeof(Library) / sizeof(void*);
  if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != count) bad("init needs the library's addresses");
  for (Py_ssize_t i = 0; i < count; ++i) ((void**)&lib)[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
  if (PyErr_Occurred()) throw python_error();
  Py_INCREF(a[1]);
  Py_XDECREF(check);
  check = a[1];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// quantise(X, nblocks or None) -> (memory, bytes of the Quantised, code bytes, scale bytes)
PyObject* quantise(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 2);
  if (!THPVariable_Check(a[0])) bad("X must be a tensor");
  const at::Tensor& X = THPVariable_Unpack(a[0]);
  Quantised q;
  q.dtype = dtype_of(X, "X");
  const bool given = a[1] != Py_None;
  const int64_t nb = given ? PyLong_AsLongLong(a[1]) : 1;
  if (PyErr_Occurred()) throw python_error();
  q.by_block = X.dim() == 3;
  if (X.dim() == 3) {
    q.nblocks = X.size(0);
    q.rows = X.size(1);
    q.cols = X.size(2);
    if (given && nb != q.nblocks) bad("X has " + std::to_string(q.nblocks) + " blocks, nblocks is " + std::to_string(nb));
  } else if (X.dim() == 2) {
    q.nblocks = nb;
    q.rows = X.size(0);
    if (q.nblocks <= 0 || X.size(1) % q.nblocks) bad(std::to_string(X.size(1)) + " columns do not divide into " + std::to_string(q.nblocks) + " blocks");
    q.cols = X.size(1) / q.nblocks;
  } else {
    bad("X must have 2 or 3 dimensions, got " + std::to_string(X.dim()));
  }
  tensor(a[0], "X");
  q.device = X.get_device();
  size32(q.nblocks, "nblocks");
  size32(q.cols, "a block");
  const monarch_mx4_dims d = dims_of(q, q.dtype);
  const int64_t codes = (int64_t)lib.code_bytes(&d), scales = (int64_t)lib.scale_bytes(&d), at = (codes + 511) & ~int64_t(511);
  // both buffers in one piece of memory; sizes that the library does not take have none, and fail below
  const at::Tensor hold = bytes_on(at + scales, q.device);
  q.codes = (int64_t)hold.data_ptr();
  q.scales = q.codes + at;
  void* x = X.data_ptr();
  call("monarch_mx4_quantise", q.device, [&](void* s) { return lib.quantise(x, &d, (void*)q.codes, (void*)q.scales, s); });
  PyObject* h = THPVariable_Wrap(hold);
  if (h == nullptr) throw python_error();
  return Py_BuildValue("(Ny#LL)", h, (const char*)&q, (Py_ssize_t)sizeof(q), (long long)codes, (long long)scales);
  END_HANDLE_TH_ERRORS
}

// dequantise(q, dtype, out or None) -> out
PyObject* dequantise(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 3);
  const Quantised& q = quantised(a[0], "q");
  const int64_t dtype = PyLong_AsLongLong(a[1]);
  if (PyErr_Occurred()) throw python_error();
  const int64_t by_block[3] = {q.nblocks, q.rows, q.cols}, plain[2] = {q.rows, q.nblocks * q.cols};
  const at::Tensor out = output(a[2], "out", q.by_block ? at::IntArrayRef(by_block, 3) : at::IntArrayRef(plain, 2), dtype, q.device);
  const monarch_mx4_dims d = dims_of(q, dtype);
  void* p = out.data_ptr();
  call("monarch_mx4_dequantise", q.device, [&](void* s) { return lib.dequantise((void*)q.codes, (void*)q.scales, &d, p, s); });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

monarch_mx4_linear_dims layer_of(const Quantised& w, int64_t rows, bool bias, int64_t dtype) {
  return monarch_mx4_linear_dims{rows, (int32_t)w.nblocks, (int32_t)w.cols, size32(w.rows, "out_blk"), bias ? 1 : 0, (int32_t)dtype};
}

// linear_plain(X, W, bias or None, Y or None, workspace or None) -> Y
PyObject* linear_plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const Quantised& w = quantised(a[1], "W");
  if (!THPVariable_Check(a[0])) bad("X must be a tensor or an Mx4");
  const at::Tensor& X = THPVariable_Unpack(a[0]);
  const int64_t dtype = dtype_of(X, "X"), rows = X.dim() > 0 ? X.size(0) : 0, n_out = w.nblocks * w.rows;
  if (X.dim() != 2 || X.size(1) != w.nblocks * w.cols)
    bad("X must have shape " + shape_of({rows, w.nblocks * w.cols}) + ", its shape is " + shape_of(X.sizes()));
  tensor(a[0], "X");
  const int64_t device = X.get_device();
  on_device(w, "W", device);
  const at::Tensor bias = a[2] == Py_None ? at::Tensor() : output(a[2], "bias", {n_out}, dtype, device);
  const at::Tensor Y = output(a[3], "Y", {rows, n_out}, dtype, device);
  const monarch_mx4_linear_dims d = layer_of(w, rows, bias.defined(), dtype);
  const Workspace ws(a[4], lib.wfwd_bytes(&d), device);
  void *x = X.data_ptr(), *b = ptr(bias), *y = Y.data_ptr();
  call("monarch_mx4_linear_wfwd", device, [&](void* s) { return lib.wfwd(x, (void*)w.codes, (void*)w.scales, b, &d, y, ws.p, ws.n, s); });
  return THPVariable_Wrap(Y);
  END_HANDLE_TH_ERRORS
}

// linear_mx4(X, W, dtype, bias or None, Y or None) -> Y
PyObject* linear_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const Quantised &x = quantised(a[0], "X"), &w = quantised(a[1], "W");
  const int64_t dtype = PyLong_AsLongLong(a[2]), n_out = w.nblocks * w.rows;
  if (PyErr_Occurred()) throw python_error();
  const int64_t device = x.device;
  on_device(w, "W", device);
  const at::Tensor bias = a[3] == Py_None ? at::Tensor() : output(a[3], "bias", {n_out}, dtype, device);
  const at::Tensor Y = output(a[4], "Y", {x.rows, n_out}, dtype, device);
  const monarch_mx4_linear_dims d = layer_of(w, x.rows, bias.defined(), dtype);
  void *b = ptr(bias), *y = Y.data_ptr();
  call("monarch_mx4_linear_fwd", device,
       [&](void* s) { return lib.fwd((void*)x.codes, (void*)x.scales, (void*)w.codes, (void*)w.scales, b, &d, y, s); });
  return THPVariable_Wrap(Y);
  END_HANDLE_TH_ERRORS
}

// linear_bwd(dY, X or None, W, want dX, want dbias, dX, dW, dbias, workspace: each a tensor or None) -> (dX, dW, dbias)
PyObject* linear_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const bool want_x = truth(a[3], "need_dX"), want_b = truth(a[4], "bias");
  if (a[1] == Py_None && a[6] != Py_None) bad("dW needs X");
  if (!want_x && a[5] != Py_None) bad("dX is given, and need_dX is false");
  if (!want_b && a[7] != Py_None) bad("dbias is given, and bias is false");
  const Quantised& w = quantised(a[2], "W");
  const Quantised* x = a[1] == Py_None ? nullptr : &quantised(a[1], "X");
  if (!THPVariable_Check(a[0])) bad("dY must be a tensor");
  const at::Tensor& dY = THPVariable_Unpack(a[0]);
  const int64_t dtype = dtype_of(dY, "dY"), rows = dY.dim() > 0 ? dY.size(0) : 0, n_in = w.nblocks * w.cols, n_out = w.nblocks * w.rows;
  if (dY.dim() != 2 || dY.size(1) != n_out) bad("dY must have shape " + shape_of({rows, n_out}) + ", its shape is " + shape_of(dY.sizes()));
  if (x != nullptr && x->rows != rows) bad("X has " + std::to_string(x->rows) + " rows, dY " + std::to_string(rows));
  tensor(a[0], "dY");
  const int64_t device = dY.get_device();
  on_device(w, "W", device);
  if (x != nullptr) on_device(*x, "X", device);
  const at::Tensor dX = want_x ? output(a[5], "dX", {rows, n_in}, dtype, device) : at::Tensor();
  const at::Tensor dW = x != nullptr ? output(a[6], "dW", {w.nblocks, w.rows, w.cols}, dtype, device) : at::Tensor();
  const at::Tensor db = want_b ? output(a[7], "dbias", {n_out}, dtype, device) : at::Tensor();
  const monarch_mx4_linear_dims d = layer_of(w, rows, want_b, dtype);
  const Workspace ws(a[8], lib.bwd_bytes(&d), device);
  void *dy = dY.data_ptr(), *px = ptr(dX), *pw = ptr(dW), *pb = ptr(db);
  call("monarch_mx4_linear_bwd", device, [&](void* s) {
    return lib.bwd(dy, x ? (void*)x->codes : nullptr, x ? (void*)x->scales : nullptr, (void*)w.codes, (void*)w.scales, &d, px, pw, pb, ws.p,
                   ws.n, s);
  });
  auto wrap = [](const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_INCREF(Py_None);
    return Py_None;
  };
  return Py_BuildValue("(NNN)", wrap(dX), wrap(dW), wrap(db));
  END_HANDLE_TH_ERRORS
}

// monarch(X, R, L, (nb1, in1, out1, nb2, in2, out2, out_transpose), Y or None, workspace or None) -> Y
PyObject* monarch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const Quantised &r = quantised(a[1], "R"), &l = quantised(a[2], "L");
  if (!PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 7) bad("the dims must be seven numbers");
  int64_t v[7];
  for (int i = 0; i < 7; ++i) v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a[3], i));
  if (PyErr_Occurred()) throw python_error();
  if (!THPVariable_Check(a[0])) bad("X must be a tensor");
  const at::Tensor& X = THPVariable_Unpack(a[0]);
  if (r.nblocks != v[0] || r.cols != v[1] || r.rows != v[2])
    bad("R has shape " + shape_of({r.nblocks, r.rows, r.cols}) + ", the dims need " + shape_of({v[0], v[2], v[1]}));
  if (l.nblocks != v[3] || l.cols != v[4] || l.rows != v[5])
    bad("L has shape " + shape_of({l.nblocks, l.rows, l.cols}) + ", the dims need " + shape_of({v[3], v[5], v[4]}));
  const int64_t dtype = dtype_of(X, "X"), rows = X.dim() > 0 ? X.size(0) : 0;
  if (X.dim() != 2 || X.size(1) != v[0] * v[1]) bad("X must have shape " + shape_of({rows, v[0] * v[1]}) + ", its shape is " + shape_of(X.sizes()));
  tensor(a[0], "X");
  const int64_t device = X.get_device();
  on_device(r, "R", device);
  on_device(l, "L", device);
  const at::Tensor Y = output(a[4], "Y", {rows, v[3] * v[5]}, dtype, device);
  const monarch_dims d = {rows,          (int32_t)v[0], (int32_t)v[1],       size32(v[2], "out1"),       (int32_t)v[3],
                          (int32_t)v[4], size32(v[5], "out2"), v[6] ? 1 : 0, (int32_t)dtype};
  const Workspace ws(a[5], lib.monarch_bytes(&d), device);
  void *x = X.data_ptr(), *y = Y.data_ptr();
  call("monarch_mx4_fwd", device, [&](void* s) {
    return lib.monarch_fwd(x, (void*)r.codes, (void*)r.scales, (void*)l.codes, (void*)l.scales, &d, y, ws.p, ws.n, s);
  });
  return THPVariable_Wrap(Y);
  END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init),         FAST(quantise),   FAST(dequantise), FAST(linear_plain), FAST(linear_mx4),
                         FAST(linear_bwd),   FAST(monarch),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mx4_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx4_native() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "key", MX4_NATIVE_KEY) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
