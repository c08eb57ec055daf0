// The usual calls of the block norm, of the gradient norm and clip, of the head
// norm with rotation and of the embedding, from Python straight to the C entry
// points: a short call costs what it costs on
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
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
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

struct MoreEntries {
  decltype(&rms_norm_rotary_fwd) rotary_fwd;
  decltype(&rms_norm_rotary_bwd) rotary_bwd;
  decltype(&rms_norm_rotary_bwd_workspace_size) rotary_ws;
  decltype(&rms_norm_embedding_fwd) embedding_fwd;
  decltype(&rms_norm_embedding_bwd) embedding_bwd;
  decltype(&rms_norm_embedding_bwd_workspace_size) embedding_ws;
} more;

int code_of(at::ScalarType type) {
  switch (type) {
    case at::kFloat: return RMSN_F32;
    case at::kBFloat16: return RMSN_BF16;
    case at::kHalf: return RMSN_F16;
    default: return -1;
  }
}

int code_of(const at::Tensor& t) { return code_of(t.scalar_type()); }

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

// A tensor argument of any strides and type, or none.
const at::Tensor* tensor_of(PyObject* o, bool* usual) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_CheckExact(o)) {
    *usual = false;
    return nullptr;
  }
  const at::Tensor* t = &THPVariable_Unpack(o);
  if (!t->is_cuda()) *usual = false;
  return t;
}

// A tensor of heads of these sizes, its last dimension contiguous.
bool heads_fit(const at::Tensor* t, at::ScalarType type, at::IntArrayRef sizes, int device) {
  return t && t->scalar_type() == type && t->sizes() == sizes && t->get_device() == device &&
         (t->size(-1) == 1 || t->stride(-1) == 1);
}

rmsn_heads heads_of(const at::Tensor& t) {
  return {t.data_ptr(), t.dim() == 4 ? t.stride(0) : 0, t.stride(-3), t.stride(-2)};
}

// A new tensor like torch.empty_like's.
at::Tensor heads_like(const at::Tensor& t, int device) {
  int64_t last = 0;
  bool in_order = true;
  for (int64_t i = t.dim() - 1; i >= 0 && in_order; --i) {
    if (t.size(i) == 1) continue;
    in_order = t.stride(i) >= last;
    last = t.stride(i);
  }
  if (in_order) return empty(t.sizes(), t.scalar_type(), device);
  if (!t.is_non_overlapping_and_dense()) return at::empty_like(t);
  return at::Tensor(at::detail::empty_strided_cuda(
      t.sizes(), t.strides(), t.scalar_type(), at::Device(at::kCUDA, (c10::DeviceIndex)device)));
}

// What the head norm's calls share.
struct RotaryCall {
  const at::Tensor *q, *k, *freq, *pos;
  int64_t batch, tokens, hq, hk = 0, dim, rotary = 0, pos_stride = 0;
  int device, dtype;
  double offset, interleaved;
  const void *qg, *kg, *freq_p, *pos_p;
  int freq_64, pos_64;
  bool usual = true;
  // a: q, k, q_gamma, k_gamma; b: inv_freq, positions
  RotaryCall(PyObject* const* a, PyObject* const* b) {
    q = tensor_of(a[0], &usual);
    k = tensor_of(a[1], &usual);
    const Arg g0(a[2]), g1(a[3]);
    freq = tensor_of(b[0], &usual);
    pos = tensor_of(b[1], &usual);
    usual = usual && q && g0 && g0.usual && g1.usual && !k == !g1 && take(g0, g1);
  }
  bool take(const Arg& g0, const Arg& g1) {
    if (q->dim() != 3 && q->dim() != 4) return false;
    const at::ScalarType type = q->scalar_type();
    device = q->get_device();
    dtype = code_of(type);
    dim = q->size(-1), hq = q->size(-2), tokens = q->size(-3);
    batch = q->dim() == 4 ? q->size(0) : 1;
    if (dtype < 0 || q->numel() == 0 || !heads_fit(q, type, q->sizes(), device)) return false;
    if (!g0.fits(type, {dim}, device) || !g1.fits(type, {dim}, device)) return false;
    if (k) {
      hk = k->dim() == q->dim() ? k->size(-2) : 0;
      if (hk < 1 || !heads_fit(k, type, k->sizes(), device)) return false;
      for (int64_t i = 0; i < q->dim(); ++i)
        if (i != q->dim() - 2 && k->size(i) != q->size(i)) return false;
    }
    qg = g0.ptr(), kg = g1.ptr();
    freq_p = pos_p = nullptr;
    freq_64 = pos_64 = 0;
    if (freq) {
      const at::ScalarType f = freq->scalar_type();
      if ((f != at::kFloat && f != at::kDouble) || freq->dim() != 1 || !freq->is_contiguous() ||
          freq->get_device() != device || 2 * freq->numel() > dim)
        return false;
      rotary = 2 * freq->numel();
      freq_64 = f == at::kDouble;
      if (rotary) freq_p = freq->data_ptr();
    }
    if (pos) {
      const at::ScalarType f = pos->scalar_type();
      if ((f != at::kInt && f != at::kLong) || pos->get_device() != device) return false;
      const bool shared = pos->sizes() == at::IntArrayRef(tokens);
      if (!shared && pos->sizes() != q->sizes().slice(0, q->dim() - 2)) return false;
      if (tokens > 1 && pos->stride(-1) != 1) return false;
      pos_stride = pos->dim() == 2 ? pos->stride(0) : 0;
      pos_64 = f == at::kLong;
      pos_p = pos->data_ptr();
    }
    return c10::cuda::current_device() == device;
  }
};

// An output of heads: the tensor given as argument i, or one to be made like `like`.
bool given_heads(PyObject* const* a, Py_ssize_t n, int i, const at::Tensor* like, at::Tensor* t) {
  if (i >= n || a[i] == Py_None) return true;
  bool usual = true;
  const at::Tensor* g = tensor_of(a[i], &usual);
  if (!usual || !like || !heads_fit(g, like->scalar_type(), like->sizes(), like->get_device()))
    return false;
  *t = *g;
  return true;
}

// rotary_fwd(q, k, q_gamma, k_gamma, inv_freq, positions, eps, offset, interleaved, with_rstd[,
//            q_out, k_out, rstd_q, rstd_k])
PyObject* rotary_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_rotary_fwd", [&](int& st) -> PyObject* {
    if (n != 10 && n != 14) return nullptr;
    const RotaryCall c(a, a + 4);
    double v[4];
    if (!c.usual || !numbers(a + 6, 4, v)) return nullptr;
    for (int i = 1; i < 4; ++i)
      if (v[i] != 0.0 && v[i] != 1.0) return nullptr;
    at::Tensor qo, ko;
    if (!given_heads(a, n, 10, c.q, &qo) || !given_heads(a, n, 11, c.k, &ko)) return nullptr;
    const bool stats = v[3] != 0.0;
    if (n > 12 && !stats && (a[12] != Py_None || a[13] != Py_None)) return nullptr;
    if (n > 13 && !c.k && a[13] != Py_None) return nullptr;
    Output rq, rk;
    if (stats) rq = Output(a, n, 12, c.q->sizes().slice(0, c.q->dim() - 1), at::kFloat, c.device);
    if (stats && c.k)
      rk = Output(a, n, 13, c.k->sizes().slice(0, c.k->dim() - 1), at::kFloat, c.device);
    if (!rq.usual || !rk.usual) return nullptr;
    {
      const Unlocked unlocked;
      if (!qo.defined()) qo = heads_like(*c.q, c.device);
      if (!ko.defined() && c.k) ko = heads_like(*c.k, c.device);
      rq.make();
      rk.make();
      const rmsn_heads q = heads_of(*c.q), q_out = heads_of(qo);
      rmsn_heads k{}, k_out{};
      if (c.k) k = heads_of(*c.k), k_out = heads_of(ko);
      st = more.rotary_fwd(&q, c.k ? &k : nullptr, c.qg, c.kg, c.freq_p, c.freq_64, c.pos_p,
                           c.pos_64, c.pos_stride, &q_out, c.k ? &k_out : nullptr,
                           static_cast<float*>(rq.ptr()), static_cast<float*>(rk.ptr()), c.batch,
                           c.tokens, c.hq, c.hk, c.dim, c.rotary, (int)v[2], (float)v[0],
                           (int)v[1], c.dtype,
                           c10::cuda::getCurrentCUDAStream(c.device).stream());
    }
    if (st != RMSN_OK) return nullptr;
    for (int i = 10; i < 14; ++i) written(a, n, i);
    return tuple_of({qo, ko, rq.t, rk.t});
  });
}

// rotary_bwd(dq_out, dk_out, q, k, q_gamma, k_gamma, rstd_q, rstd_k, inv_freq, positions, offset,
//            interleaved[, dq, dk, workspace])
PyObject* rotary_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_rotary_bwd", [&](int& st) -> PyObject* {
    if (n != 12 && n != 15) return nullptr;
    const RotaryCall c(a + 2, a + 8);
    double v[2];
    if (!c.usual || !numbers(a + 10, 2, v)) return nullptr;
    for (double x : v)
      if (x != 0.0 && x != 1.0) return nullptr;
    bool usual = true;
    const at::Tensor *uq = tensor_of(a[0], &usual), *uk = tensor_of(a[1], &usual);
    const Arg rq(a[6]), rk(a[7]);
    const at::ScalarType type = c.q->scalar_type();
    if (!usual || !heads_fit(uq, type, c.q->sizes(), c.device) || !rq ||
        !rq.fits(at::kFloat, c.q->sizes().slice(0, c.q->dim() - 1), c.device))
      return nullptr;
    if (c.k ? !heads_fit(uk, type, c.k->sizes(), c.device) || !rk ||
                  !rk.fits(at::kFloat, c.k->sizes().slice(0, c.k->dim() - 1), c.device)
            : uk || !rk.usual || rk)
      return nullptr;
    at::Tensor dq, dk, dgq, dgk, ws;
    if (!given_heads(a, n, 12, c.q, &dq) || !given_heads(a, n, 13, c.k, &dk)) return nullptr;
    if (n > 14 && a[14] != Py_None) {
      if (!THPVariable_CheckExact(a[14])) return nullptr;
      ws = THPVariable_Unpack(a[14]);
      if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != c.device) return nullptr;
    }
    {
      const Unlocked unlocked;
      if (!dq.defined()) dq = heads_like(*c.q, c.device);
      if (!dk.defined() && c.k) dk = heads_like(*c.k, c.device);
      dgq = empty({c.dim}, at::kFloat, c.device);
      if (c.k) dgk = empty({c.dim}, at::kFloat, c.device);
      const size_t need = more.rotary_ws(c.batch, c.tokens, c.hq, c.hk, c.dim);
      if (need > 0 && !ws.defined()) ws = bytes(need, c.device);
      const rmsn_heads q = heads_of(*c.q), up_q = heads_of(*uq), out_q = heads_of(dq);
      rmsn_heads k{}, up_k{}, out_k{};
      if (c.k) k = heads_of(*c.k), up_k = heads_of(*uk), out_k = heads_of(dk);
      const auto given = [&](const rmsn_heads& h) { return c.k ? &h : nullptr; };
      st = more.rotary_bwd(
          &up_q, given(up_k), &q, given(k), c.qg, c.kg, static_cast<const float*>(rq.ptr()),
          static_cast<const float*>(rk.ptr()), c.freq_p, c.freq_64, c.pos_p, c.pos_64,
          c.pos_stride, &out_q, given(out_k), static_cast<float*>(ptr(dgq)),
          static_cast<float*>(ptr(dgk)), c.batch, c.tokens, c.hq, c.hk, c.dim, c.rotary, (int)v[1],
          (int)v[0], c.dtype, ptr(ws), ws.defined() ? (size_t)ws.nbytes() : 0,
          c10::cuda::getCurrentCUDAStream(c.device).stream());
    }
    if (st != RMSN_OK) return nullptr;
    written(a, n, 12);
    written(a, n, 13);
    return tuple_of({dq, dk, dgq, dgk});
  });
}

// The scalar type that a dtype argument names, `otherwise` for None.
bool type_of(PyObject* o, at::ScalarType otherwise, at::ScalarType* type) {
  *type = otherwise;
  if (o == Py_None) return true;
  if (!THPDtype_Check(o)) return false;
  *type = reinterpret_cast<THPDtype*>(o)->scalar_type;
  return true;
}

bool is_ids(const at::Tensor* t) {
  return t && (t->scalar_type() == at::kInt || t->scalar_type() == at::kLong) &&
         t->is_contiguous() && t->numel() > 0;
}

// Of one type, or one of them fp32.
bool types_match(at::ScalarType a, at::ScalarType b) {
  return code_of(a) >= 0 && code_of(b) >= 0 && (a == b || a == at::kFloat || b == at::kFloat);
}

bool whole(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// embedding_fwd(ids, weight, scale, dtype or None[, y])
PyObject* embedding_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_embedding_fwd", [&](int& st) -> PyObject* {
    if (n != 4 && n != 5) return nullptr;
    bool usual = true;
    const at::Tensor* ids = tensor_of(a[0], &usual);
    const Arg w(a[1]);
    double scale;
    at::ScalarType type;
    if (!usual || !is_ids(ids) || !w || !w.usual || w.t->dim() != 2 || w.t->numel() == 0 ||
        !numbers(a + 2, 1, &scale))
      return nullptr;
    const bool given = n > 4 && a[4] != Py_None;
    const Arg y(given ? a[4] : Py_None);
    if (!y.usual || !type_of(a[3], y ? y.t->scalar_type() : w.t->scalar_type(), &type) ||
        !types_match(w.t->scalar_type(), type))
      return nullptr;
    const int device = (int)ids->get_device();
    const int64_t vocab = w.t->size(0), hidden = w.t->size(1);
    c10::SmallVector<int64_t, 6> sizes(ids->sizes().begin(), ids->sizes().end());
    sizes.push_back(hidden);
    if (w.t->get_device() != device || c10::cuda::current_device() != device ||
        !y.fits(type, sizes, device))
      return nullptr;
    at::Tensor out;
    {
      const Unlocked unlocked;
      out = y ? *y.t : empty(sizes, type, device);
      st = more.embedding_fwd(ids->data_ptr(), ids->scalar_type() == at::kLong, w.ptr(),
                              out.data_ptr(), ids->numel(), vocab, hidden, (float)scale,
                              code_of(*w.t), code_of(type),
                              c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    }
    if (st != RMSN_OK) return nullptr;
    written(a, n, 4);
    return wrap(out);
  });
}

// embedding_bwd(dy, ids, vocab, scale, padding_idx or None, dtype or None, dweight or None,
//               accumulate[, workspace])
PyObject* embedding_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rms_norm_embedding_bwd", [&](int& st) -> PyObject* {
    if (n != 8 && n != 9) return nullptr;
    bool usual = true;
    const Arg dy(a[0]), dw(a[6]);
    const at::Tensor* ids = tensor_of(a[1], &usual);
    int64_t vocab, pad = -1;
    double scale, accumulate;
    at::ScalarType type;
    if (!usual || !dy || !dy.usual || !dw.usual || !is_ids(ids) || !whole(a[2], &vocab) ||
        !numbers(a + 3, 1, &scale) || !numbers(a + 7, 1, &accumulate) || vocab < 1 ||
        vocab > RMSN_EMBEDDING_MAX_VOCAB)
      return nullptr;
    if (a[4] != Py_None && (!whole(a[4], &pad) || pad < 0 || pad >= vocab)) return nullptr;
    if ((accumulate != 0.0 && accumulate != 1.0) || (accumulate != 0.0 && !dw)) return nullptr;
    if (!type_of(a[5], dw ? dw.t->scalar_type() : at::kFloat, &type) ||
        !types_match(dy.t->scalar_type(), type))
      return nullptr;
    const int device = (int)dy.t->get_device();
    if (dy.t->dim() < 1 || dy.t->numel() == 0 ||
        dy.t->sizes().slice(0, dy.t->dim() - 1) != ids->sizes() || ids->get_device() != device ||
        c10::cuda::current_device() != device)
      return nullptr;
    const int64_t hidden = dy.t->size(-1), tokens = ids->numel();
    if (!dw.fits(type, {vocab, hidden}, device)) return nullptr;
    at::Tensor out, ws;
    if (n > 8 && a[8] != Py_None) {
      if (!THPVariable_CheckExact(a[8])) return nullptr;
      ws = THPVariable_Unpack(a[8]);
      if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != device) return nullptr;
    }
    {
      const Unlocked unlocked;
      out = dw ? *dw.t : empty({vocab, hidden}, type, device);
      const size_t need = more.embedding_ws(tokens, vocab, hidden);
      if (need > 0 && !ws.defined()) ws = bytes(need, device);
      st = more.embedding_bwd(dy.ptr(), ids->data_ptr(), ids->scalar_type() == at::kLong,
                              out.data_ptr(), tokens, vocab, hidden, (float)scale, pad,
                              (int)accumulate, code_of(*dy.t), code_of(type), ptr(ws),
                              ws.defined() ? (size_t)ws.nbytes() : 0,
                              c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    }
    if (st != RMSN_OK) return nullptr;
    written(a, n, 6);
    return wrap(out);
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

// init_more(addresses of the C entry points, in the order of MoreEntries)
PyObject* init_more(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !address(a[0], &more.rotary_fwd) || !address(a[1], &more.rotary_bwd) ||
      !address(a[2], &more.rotary_ws) || !address(a[3], &more.embedding_fwd) ||
      !address(a[4], &more.embedding_bwd) || !address(a[5], &more.embedding_ws)) {
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
                         {"init_more", FAST(init_more), nullptr},
                         {"rotary_fwd", FAST(rotary_fwd), nullptr},
                         {"rotary_bwd", FAST(rotary_bwd), nullptr},
                         {"embedding_fwd", FAST(embedding_fwd), nullptr},
                         {"embedding_bwd", FAST(embedding_bwd), nullptr},
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
