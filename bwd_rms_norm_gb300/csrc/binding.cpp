// The usual calls of the block norm and of the gradient norm and clip, from
// Python straight to the C entry points: a short call costs what it costs on
// the host (8 x 4096: 20 us through ctypes, 6.3 here; with outputs given 4.4, of
// which the kernel takes 4.2).
//
// Argument marshalling only, and only of arguments that need no second look:
// plain contiguous CUDA tensors of one device, the current one, with matching
// types and shapes, the current stream.  Every function returns None for
// anything else, and for arguments that the C entry refuses; the Python
// functions then take their own way, with their checks and messages.  A CUDA
// error raises RMSNormError from here: what was enqueued before it must not run
// twice.  No C++ exception leaves this file.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "rms_norm.h"

namespace {

struct Entries {
  decltype(&rms_norm_block_fwd) block_fwd;
  decltype(&rms_norm_block_bwd) block_bwd;
  decltype(&rms_norm_block_bwd_workspace_size) block_ws;
  decltype(&rms_norm_grad_norm) grad_norm;
  decltype(&rms_norm_grad_clip) grad_clip;
  decltype(&rms_norm_grad_workspace_size) grad_ws;
} entry;

int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return RMSN_F32;
    case at::kBFloat16: return RMSN_BF16;
    case at::kHalf: return RMSN_F16;
    default: return -1;
  }
}

// A tensor argument, or none (Py_None), that needs no second look.
struct Arg {
  const at::Tensor* t = nullptr;
  bool usual = true;
  explicit Arg(PyObject* o) {
    if (o == Py_None) return;
    usual = THPVariable_CheckExact(o);
    if (!usual) return;
    t = &THPVariable_Unpack(o);
    usual = t->is_cuda() && t->is_contiguous() && code_of(*t) >= 0;
  }
  explicit operator bool() const { return t != nullptr; }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
  // of this type and these sizes, on this device; or none
  bool fits(at::ScalarType type, at::IntArrayRef sizes, int device) const {
    return usual &&
           (!t || (t->scalar_type() == type && t->sizes() == sizes && t->get_device() == device));
  }
};

struct Call {
  int64_t rows = 0, hidden = 0, gate_rows = 0;
  int device = 0, dtype = 0, stream_dtype = 0;
  at::IntArrayRef sizes, row_sizes;
};

// What the block norm's calls share: x, the residual stream, the weights.
bool usual_call(const Arg& x, const Arg& res, const Arg& post, const Arg& gate, const Arg& next,
                Call* c) {
  if (!x || !res || !x.usual || !res.usual || (!post && !next) || x.t->dim() < 1) return false;
  c->hidden = x.t->size(-1);
  if (x.t->numel() == 0) return false;
  c->rows = x.t->numel() / c->hidden;
  c->device = x.t->get_device();
  c->dtype = code_of(*x.t);
  c->stream_dtype = code_of(*res.t);
  c->sizes = x.t->sizes();
  c->row_sizes = c->sizes.slice(0, c->sizes.size() - 1);
  const at::ScalarType type = x.t->scalar_type();
  if (c->stream_dtype != c->dtype && c->stream_dtype != RMSN_F32) return false;
  if (!res.fits(res.t->scalar_type(), c->sizes, c->device)) return false;
  if (!post.fits(type, {c->hidden}, c->device) || !next.fits(type, {c->hidden}, c->device))
    return false;
  if (gate) {
    if (!gate.fits(type, gate.t->sizes(), c->device) || gate.t->dim() < 1 ||
        gate.t->size(-1) != c->hidden)
      return false;
    c->gate_rows = gate.t->numel() / c->hidden;
    if (c->gate_rows < 1 || c->rows % c->gate_rows != 0) return false;
    // rows for runs of x's rows for certain (a gate may broadcast otherwise)
    const int64_t nx = x.t->dim(), ng = gate.t->dim();
    if (c->gate_rows > 1 && nx != 2 &&
        !(nx == 3 && ng == 3 && gate.t->size(0) == x.t->size(0)) &&
        !(nx == 3 && ng == 2 && gate.t->size(0) != x.t->size(1)))
      return false;
  } else if (!gate.usual) {
    return false;
  }
  return c10::cuda::current_device() == c->device;
}

// A new tensor, without the dispatcher (8 x 4096 forward 7.3 -> 6.1 us): on the current
// device, which every call's is, from the current stream's memory.
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, int device) {
  return at::Tensor(at::detail::empty_cuda(
      sizes, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt));
}

at::Tensor bytes(size_t n, int device) {
  return empty({(int64_t)(n < 16 ? 16 : n)}, at::kByte, device);
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

bool numbers(PyObject* const* a, int n, double* out) {
  for (int i = 0; i < n; ++i) {
    out[i] = PyFloat_AsDouble(a[i]);
    if (out[i] == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
  }
  return true;
}

// Sets RMSNormError(fn, RMSN_ERR_CUDA).
void set_cuda_error(const char* fn) {
  PyObject* package = PyImport_ImportModule("bwd_rms_norm_gb300");
  PyObject* type = package ? PyObject_GetAttrString(package, "RMSNormError") : nullptr;
  PyObject* error = type ? PyObject_CallFunction(type, "si", fn, (int)RMSN_ERR_CUDA) : nullptr;
  if (error) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(package);
}

// The body of a call of the C entry `fn`: None where it is not a usual one, or
// throws.  f(st) leaves the entry's status in st, once it has called it.
template <typename F>
PyObject* guarded(const char* fn, F f) {
  int st = RMSN_OK;
  try {
    PyObject* r = f(st);
    if (r) return r;
  } catch (...) {
  }
  if (PyErr_Occurred()) PyErr_Clear();
  if (st == RMSN_ERR_CUDA) {
    set_cuda_error(fn);
    return nullptr;
  }
  Py_RETURN_NONE;
}

// Other threads of Python run while one of these lives: allocations may free
// memory and launches may wait for room in their queue.  Nothing of Python's is
// touched meanwhile; the arguments are held by the caller, or by a List.
class Unlocked {
  PyThreadState* state_ = PyEval_SaveThread();

 public:
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state_); }
};

// An output of a call: the tensor given as argument i, or a new one (`make`,
// which Unlocked allows).
struct Output {
  at::Tensor t;
  at::IntArrayRef sizes;
  at::ScalarType type = at::kFloat;
  int device = 0;
  bool wanted = false, usual = true;
  Output() = default;
  Output(PyObject* const* a, Py_ssize_t n, int i, at::IntArrayRef s, at::ScalarType ty, int dev)
      : sizes(s), type(ty), device(dev), wanted(true) {
    if (i >= n || a[i] == Py_None) return;
    const Arg o(a[i]);
    usual = o.fits(type, sizes, device);
    if (usual) t = *o.t;
  }
  void make() {
    if (wanted && !t.defined()) t = empty(sizes, type, device);
  }
  void* ptr() const { return t.defined() ? t.data_ptr() : nullptr; }
};

// Counts a version of a tensor that a call wrote: autograd's check of what it
// has saved.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The same for the output that was given as argument i, if one was.
void written(PyObject* const* a, Py_ssize_t n, int i) {
  if (i < n && a[i] != Py_None) written(THPVariable_Unpack(a[i]));
}

// block_fwd(x, residual, post, gate, next, eps, offset, residual_scale, branch_scale[,
//           residual_out, y, rstd_post, rstd_next])
PyObject* block_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_block_fwd", [&](int& st) -> PyObject* {
    if (n != 9 && n != 13) return nullptr;
    const Arg x(a[0]), res(a[1]), post(a[2]), gate(a[3]), next(a[4]);
    Call c;
    double v[4];
    if (!usual_call(x, res, post, gate, next, &c) || !numbers(a + 5, 4, v)) return nullptr;
    if (v[1] != 0.0 && v[1] != 1.0) return nullptr;
    Output out(a, n, 9, c.sizes, res.t->scalar_type(), c.device), y, r1, r2;
    if (post) r1 = Output(a, n, 11, c.row_sizes, at::kFloat, c.device);
    if (next) {
      y = Output(a, n, 10, c.sizes, x.t->scalar_type(), c.device);
      r2 = Output(a, n, 12, c.row_sizes, at::kFloat, c.device);
    }
    if (!out.usual || !y.usual || !r1.usual || !r2.usual) return nullptr;
    {
      const Unlocked unlocked;
      for (Output* o : {&out, &y, &r1, &r2}) o->make();
      st = entry.block_fwd(
          x.ptr(), res.ptr(), post.ptr(), gate.ptr(), c.gate_rows, next.ptr(), out.ptr(), y.ptr(),
          static_cast<float*>(r1.ptr()), static_cast<float*>(r2.ptr()), c.rows, c.hidden,
          (float)v[2], (float)v[3], (float)v[0], (int)v[1], c.dtype, c.stream_dtype,
          c10::cuda::getCurrentCUDAStream(c.device).stream());
    }
    if (st != RMSN_OK) return nullptr;
    written(a, n, 9);
    if (post) written(a, n, 11);
    if (next) written(a, n, 10), written(a, n, 12);
    return tuple_of({out.t, y.t, r1.t, r2.t});
  });
}

// block_bwd(dy, dresidual_out, x, residual_out, rstd_post, rstd_next, post, gate, next, offset,
//           residual_scale, branch_scale, with_dgate[, dx, dresidual, workspace])
PyObject* block_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_block_bwd", [&](int& st) -> PyObject* {
    if (n != 13 && n != 16) return nullptr;
    const Arg dy(a[0]), dr(a[1]), x(a[2]), res(a[3]), r1(a[4]), r2(a[5]), post(a[6]), gate(a[7]),
        next(a[8]);
    Call c;
    double v[4];
    if (!usual_call(x, res, post, gate, next, &c) || !numbers(a + 9, 4, v)) return nullptr;
    if (v[0] != 0.0 && v[0] != 1.0) return nullptr;
    if ((next && (!dy || !r2)) || (!next && !dr) || (post && !r1)) return nullptr;
    if (!dy.fits(x.t->scalar_type(), c.sizes, c.device) ||
        !dr.fits(res.t->scalar_type(), c.sizes, c.device) ||
        !r1.fits(at::kFloat, c.row_sizes, c.device) || !r2.fits(at::kFloat, c.row_sizes, c.device))
      return nullptr;
    Output dx(a, n, 13, c.sizes, x.t->scalar_type(), c.device);
    Output dres(a, n, 14, c.sizes, res.t->scalar_type(), c.device);
    if (!dx.usual || !dres.usual) return nullptr;
    at::Tensor dpost, dgate, dnext, ws;
    if (n > 15 && a[15] != Py_None) {
      if (!THPVariable_CheckExact(a[15])) return nullptr;
      ws = THPVariable_Unpack(a[15]);
      if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != c.device) return nullptr;
    }
    {
      const Unlocked unlocked;
      dx.make();
      dres.make();
      if (post) dpost = empty({c.hidden}, at::kFloat, c.device);
      if (next) dnext = empty({c.hidden}, at::kFloat, c.device);
      if (gate && v[3] != 0.0) dgate = empty(gate.t->sizes(), at::kFloat, c.device);
      if (!ws.defined()) ws = bytes(entry.block_ws(c.rows, c.hidden, c.gate_rows), c.device);
      st = entry.block_bwd(
          next ? dy.ptr() : nullptr, dr.ptr(), x.ptr(), res.ptr(), post.ptr(), gate.ptr(),
          c.gate_rows, next.ptr(), static_cast<float*>(r1.ptr()), static_cast<float*>(r2.ptr()),
          dx.ptr(), dres.ptr(), static_cast<float*>(ptr(dpost)), static_cast<float*>(ptr(dgate)),
          static_cast<float*>(ptr(dnext)), c.rows, c.hidden, (float)v[1], (float)v[2], (int)v[0],
          c.dtype, c.stream_dtype, ptr(ws), (size_t)ws.nbytes(),
          c10::cuda::getCurrentCUDAStream(c.device).stream());
    }
    if (st != RMSN_OK) return nullptr;
    written(a, n, 13);
    written(a, n, 14);
    return tuple_of({dx.t, dres.t, dpost, dgate, dnext});
  });
}

// A list of tensors, as it was when it was read: it holds them, since the
// caller's list may change while other threads run.
struct List {
  std::vector<void*> ptrs;
  std::vector<int64_t> numels;
  std::vector<int> codes;
  PyObject* held = nullptr;  // a tuple
  List() = default;
  List(const List&) = delete;
  ~List() { Py_XDECREF(held); }
  const at::Tensor& tensor(Py_ssize_t i) const {
    return THPVariable_Unpack(PyTuple_GET_ITEM(held, i));
  }
  // A list or tuple of usual tensors on one device, `device` if that is >= 0.
  bool read(PyObject* o, int device) {
    if (!PyList_CheckExact(o) && !PyTuple_CheckExact(o)) return false;
    held = PySequence_Tuple(o);
    if (!held) return false;
    const Py_ssize_t n = PyTuple_GET_SIZE(held);
    if (n == 0) return false;
    ptrs.reserve(n);
    numels.reserve(n);
    codes.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      if (!THPVariable_CheckExact(PyTuple_GET_ITEM(held, i))) return false;
      const at::Tensor& t = tensor(i);
      const int code = code_of(t);
      if (code < 0 || !t.is_cuda() || !t.is_contiguous()) return false;
      if (device < 0) device = t.get_device();
      if (t.get_device() != device) return false;
      ptrs.push_back(t.data_ptr());
      numels.push_back(t.numel());
      codes.push_back(code);
    }
    return c10::cuda::current_device() == device;
  }
};

// grad_norm(grads)
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_grad_norm", [&](int& st) -> PyObject* {
    List g;
    if (n != 1 || !g.read(a[0], -1)) return nullptr;
    const int64_t count = (int64_t)g.ptrs.size();
    const int device = (int)g.tensor(0).get_device();
    at::Tensor norm, ws;
    {
      const Unlocked unlocked;
      norm = empty({}, at::kFloat, device);
      ws = bytes(entry.grad_ws(count), device);
      st = entry.grad_norm(g.ptrs.data(), g.numels.data(), g.codes.data(), count,
                           static_cast<float*>(norm.data_ptr()), ws.data_ptr(), (size_t)ws.numel(),
                           c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    }
    return st == RMSN_OK ? wrap(norm) : nullptr;
  });
}

// grad_clip(grads, max_norm, eps, out or None, total_norm or None)
PyObject* grad_clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_grad_clip", [&](int& st) -> PyObject* {
    List g, o;
    double v[2];
    if (n != 5 || !g.read(a[0], -1) || !numbers(a + 1, 2, v)) return nullptr;
    const int device = (int)g.tensor(0).get_device();
    const int64_t count = (int64_t)g.ptrs.size();
    const bool in_place = a[3] == Py_None;
    if (!in_place) {
      if (!o.read(a[3], device) || o.numels != g.numels) return nullptr;
      for (int64_t i = 0; i < count; ++i)
        if (o.codes[i] != g.codes[i] && o.codes[i] != RMSN_F32) return nullptr;
    }
    const Arg total(a[4]);
    if (!total.usual || (total && (total.t->scalar_type() != at::kFloat || total.t->numel() != 1 ||
                                   total.t->get_device() != device)))
      return nullptr;
    const List& out = in_place ? g : o;
    at::Tensor norm, ws;
    {
      const Unlocked unlocked;
      norm = empty({}, at::kFloat, device);
      if (!total) ws = bytes(entry.grad_ws(count), device);
    }
    PyObject* result = wrap(norm);  // before the call: in place there is no second one
    if (!result) return nullptr;
    {
      const Unlocked unlocked;
      st = entry.grad_clip(
          g.ptrs.data(), g.numels.data(), g.codes.data(), out.ptrs.data(), out.codes.data(), count,
          (float)v[0], (float)v[1], static_cast<const float*>(total.ptr()),
          static_cast<float*>(norm.data_ptr()), ptr(ws), ws.defined() ? (size_t)ws.numel() : 0,
          c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    }
    if (st != RMSN_OK) {
      Py_DECREF(result);
      return nullptr;
    }
    for (int64_t i = 0; i < count; ++i) written(out.tensor((Py_ssize_t)i));
    return result;
  });
}

template <typename F>
bool address(PyObject* o, F* f) {
  *f = reinterpret_cast<F>(PyLong_AsVoidPtr(o));
  return *f != nullptr && !PyErr_Occurred();
}

// init(addresses of the C entry points, in the order of Entries)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !address(a[0], &entry.block_fwd) || !address(a[1], &entry.block_bwd) ||
      !address(a[2], &entry.block_ws) || !address(a[3], &entry.grad_norm) ||
      !address(a[4], &entry.grad_clip) || !address(a[5], &entry.grad_ws)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "six addresses expected");
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"init", FAST(init), nullptr},
                         {"block_fwd", FAST(block_fwd), nullptr},
                         {"block_bwd", FAST(block_bwd), nullptr},
                         {"grad_norm", FAST(grad_norm), nullptr},
                         {"grad_clip", FAST(grad_clip), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
