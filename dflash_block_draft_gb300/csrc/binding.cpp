// binding.cpp -- Python entry of the serving operators: checks the tensors and
// calls the C ABI.
//
// These calls take a few microseconds on the device, and a checked call through
// ctypes took 17 to 34 on the host (Grace).  Reading the tensors in C++, rotation, append
// and verification take 4 to 8; attention and the gradients, which allocate a workspace
// besides their results, 16 to 24.  Each function takes the arguments of its Python function in order, all of
// them, and returns the results, or the status as an int where it is not 0.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <utility>
#include <vector>

#include "dflash_attn.h"

namespace {

struct Refusal {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refusal{PyExc_ValueError, what}; }
struct PythonError {};  // one is set already

using Shape = std::initializer_list<int64_t>;

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return &THPVariable_Unpack(o);
}
const at::Tensor& required(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return *t;
}
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v != (int)v) throw Refusal{PyExc_OverflowError, "an integer argument does not fit 32 bits"};
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return (float)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}
int narrow(int64_t v) {
  if (v != (int)v) refuse("a dimension does not fit 32 bits");
  return (int)v;
}

std::string list(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

bool lies_on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

void common(const at::Tensor& t, const char* name, int dev, at::ScalarType type) {
  if (!lies_on(t, dev))
    refuse(std::string(name) + " must be a CUDA tensor" + (dev >= 0 ? " on device " + std::to_string(dev) : ""));
  if (t.scalar_type() != type)
    throw Refusal{PyExc_TypeError, std::string(name) + " must be " + at::toString(type) + ", got " + at::toString(t.scalar_type())};
}
void shaped(const at::Tensor& t, const char* name, Shape shape) {
  if (t.sizes() != at::IntArrayRef(shape))
    refuse(std::string(name) + " must be " + list(at::IntArrayRef(shape)) + ", got " + list(t.sizes()));
}

// Data pointer of a contiguous tensor, checked; null for None.
void* flat(const at::Tensor* t, const char* name, int dev, at::ScalarType type) {
  if (!t) return nullptr;
  common(*t, name, dev, type);
  if (!t->is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t->data_ptr();
}
void* flat(const at::Tensor* t, const char* name, int dev, at::ScalarType type, Shape shape) {
  if (!t) return nullptr;
  common(*t, name, dev, type);
  shaped(*t, name, shape);
  if (!t->is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t->data_ptr();
}
// Of [tokens, heads, D] whose tokens are each contiguous; their stride goes to *stride.
void* tokens(const at::Tensor& t, const char* name, int dev, at::ScalarType type, int64_t T, int64_t H, int64_t D,
             int64_t* stride) {
  common(t, name, dev, type);
  shaped(t, name, {T, H, D});
  // (the strides of a tensor without elements mean nothing)
  if (t.numel() > 0 && ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D) || (T > 1 && t.stride(0) < H * D)))
    refuse(std::string("the heads of a token of ") + name + " must be contiguous");
  *stride = T > 1 && t.numel() > 0 ? t.stride(0) : 0;
  return t.data_ptr();
}
// Of [pages, page_size, H_kv, D] whose pages are each contiguous, the last four axes of t.
void* pages(const at::Tensor& t, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape,
            int64_t* stride) {
  common(t, name, dev, type);
  if (t.sizes() != shape) refuse(std::string(name) + " must be " + list(shape) + ", got " + list(t.sizes()));
  const at::IntArrayRef s = shape.slice(shape.size() - 4), st = t.strides().slice(shape.size() - 4);
  const int64_t n = s[0], P = s[1], H = s[2], D = s[3];
  if (t.numel() > 0 && ((D > 1 && st[3] != 1) || (H > 1 && st[2] != D) || (P > 1 && st[1] != H * D) ||
                        (n > 1 && st[0] < P * H * D)))
    refuse(std::string("the pages of ") + name + " must be contiguous");
  *stride = n > 1 && t.numel() > 0 ? st[0] : 0;
  return t.data_ptr();
}

dflash_dtype_t code_of(at::ScalarType t) {
  if (t == at::kBFloat16) return DFLASH_BF16;
  if (t == at::kFloat) return DFLASH_FP32;
  throw Refusal{PyExc_TypeError, std::string("unsupported dtype ") + at::toString(t) + " (bf16 or fp32)"};
}

at::Tensor fresh(const at::Tensor& like, Shape shape, at::ScalarType type) {
  return at::empty(at::IntArrayRef(shape), like.options().dtype(type));
}

// Makes the inputs' device and the call's stream (a stream object, a plain handle, or
// None: the device's current one) current, before anything is allocated, so that
// workspaces and results come from the memory of the stream that uses them.
class On {
 public:
  On(int dev, PyObject* stream) {
    if (c10::cuda::current_device() != dev) device_.emplace((c10::DeviceIndex)dev);
    if (stream == Py_None) {
      handle_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
    if (!h) {
      PyErr_Clear();
      h = Py_NewRef(stream);
    }
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw PythonError{};
    handle_ = (cudaStream_t)p;
    stream_.emplace(p ? c10::cuda::getStreamFromExternal(handle_, (c10::DeviceIndex)dev)
                      : c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)dev));
  }
  dflash_stream_t stream() const { return (dflash_stream_t)handle_; }

 private:
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_;
  cudaStream_t handle_;
};

struct Workspace {
  at::Tensor own;
  void* ptr;
};
Workspace workspace(PyObject* given, size_t bytes, const at::Tensor& like) {
  Workspace w;
  if (const at::Tensor* t = tensor(given, "workspace")) {
    if (!lies_on(*t, like.get_device()) || !t->is_contiguous()) refuse("workspace must be a contiguous CUDA tensor on the inputs' device");
    if (t->nbytes() < bytes) refuse("workspace too small: need " + std::to_string(bytes) + " bytes");
    w.ptr = t->data_ptr();
  } else {
    w.own = fresh(like, {(int64_t)(bytes ? bytes : 1)}, at::kByte);
    w.ptr = w.own.data_ptr();
  }
  return w;
}

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (!r) throw PythonError{};
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(t)), ...);
  return r;
}
PyObject* status(dflash_status_t st) { return PyLong_FromLong(st); }

// Runs a body with its argument count checked and every C++ exception turned into Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  try {
    if (n != want) throw Refusal{PyExc_TypeError, "expected " + std::to_string(want) + " arguments"};
    return body();
  } catch (const PythonError&) {
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (!type) PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// What norm and rotation share: q and k (either None), positions, cos_sin.
struct Rope {
  const at::Tensor *q, *k, *one;
  at::ScalarType type;
  int dev;
  int64_t T, Hq, Hk, D;
  const float* cs;
  const int32_t* pos;
  const void *qp, *kp;
  dflash_rope_dims_t d;
};
Rope rope(PyObject* q, PyObject* k, PyObject* positions, PyObject* cos_sin, PyObject* eps, PyObject* interleaved) {
  Rope r = {};
  r.q = tensor(q, "q");
  r.k = tensor(k, "k");
  r.one = r.q ? r.q : r.k;
  if (!r.one) refuse("q or k must be given");
  if ((r.q && r.q->dim() != 3) || (r.k && r.k->dim() != 3)) refuse("q and k must be [tokens, heads, D]");
  r.type = r.one->scalar_type();
  code_of(r.type);
  r.dev = r.one->get_device();
  r.T = r.one->size(0);
  r.D = r.one->size(2);
  r.Hq = r.q ? r.q->size(1) : 0;
  r.Hk = r.k ? r.k->size(1) : 0;
  if (r.q) r.qp = tokens(*r.q, "q", r.dev, r.type, r.T, r.Hq, r.D, &r.d.q_stride);
  if (r.k) r.kp = tokens(*r.k, "k", r.dev, r.type, r.T, r.Hk, r.D, &r.d.k_stride);
  if (const at::Tensor* t = tensor(cos_sin, "cos_sin")) {
    if (t->dim() != 2 || positions == Py_None) refuse("cos_sin must be [max_pos, rot_dim] and comes with positions");
    r.cs = (const float*)flat(t, "cos_sin", r.dev, at::kFloat);
    r.d.max_pos = narrow(t->size(0));
    r.d.rot_dim = narrow(t->size(1));
    r.pos = (const int32_t*)flat(tensor(positions, "positions"), "positions", r.dev, at::kInt, {r.T});
  }
  r.d.T = narrow(r.T);
  r.d.H_q = narrow(r.Hq);
  r.d.H_kv = narrow(r.Hk);
  r.d.D = narrow(r.D);
  r.d.eps = real(eps);
  r.d.interleaved = truth(interleaved);
  return r;
}
at::Tensor given_or(PyObject* o, const char* name, const at::Tensor& like, Shape shape, at::ScalarType type) {
  const at::Tensor* t = tensor(o, name);
  return t ? *t : fresh(like, shape, type);
}

// (q, k, positions, cos_sin, q_norm, k_norm, eps, interleaved, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Rope r = rope(a[0], a[1], a[2], a[3], a[6], a[7]);
    const void* wq = flat(tensor(a[4], "q_norm"), "q_norm", r.dev, r.type, {r.D});
    const void* wk = flat(tensor(a[5], "k_norm"), "k_norm", r.dev, r.type, {r.D});
    const On on(r.dev, a[10]);
    at::Tensor qo, ko;
    void *qop = nullptr, *kop = nullptr;
    if (r.q) {
      qo = given_or(a[8], "q_out", *r.q, {r.T, r.Hq, r.D}, r.type);
      qop = flat(&qo, "q_out", r.dev, r.type, {r.T, r.Hq, r.D});
    }
    if (r.k) {
      ko = given_or(a[9], "k_out", *r.k, {r.T, r.Hk, r.D}, r.type);
      kop = flat(&ko, "k_out", r.dev, r.type, {r.T, r.Hk, r.D});
    }
    const dflash_status_t st = dflash_qk_norm_rope(&r.d, code_of(r.type), r.qp, r.kp, wq, wk, r.cs, r.pos, qop, kop,
                                                   on.stream());
    return st ? status(st) : tuple(qo, ko);
  });
}

// (q, k, positions, cos_sin, dq_out, dk_out, q_norm, k_norm, eps, interleaved, dq, dk, dq_norm, dk_norm, workspace, stream)
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const Rope r = rope(a[0], a[1], a[2], a[3], a[8], a[9]);
    const void* wq = flat(tensor(a[6], "q_norm"), "q_norm", r.dev, r.type, {r.D});
    const void* wk = flat(tensor(a[7], "k_norm"), "k_norm", r.dev, r.type, {r.D});
    const On on(r.dev, a[15]);
    const void *gq = nullptr, *gk = nullptr;
    at::Tensor dq, dk, dwq, dwk;
    void *dqp = nullptr, *dkp = nullptr, *dwqp = nullptr, *dwkp = nullptr;
    if (r.q) {
      gq = flat(&required(a[4], "dq_out"), "dq_out", r.dev, r.type, {r.T, r.Hq, r.D});
      dq = given_or(a[10], "dq", *r.q, {r.T, r.Hq, r.D}, r.type);
      dqp = flat(&dq, "dq", r.dev, r.type, {r.T, r.Hq, r.D});
    }
    if (r.k) {
      gk = flat(&required(a[5], "dk_out"), "dk_out", r.dev, r.type, {r.T, r.Hk, r.D});
      dk = given_or(a[11], "dk", *r.k, {r.T, r.Hk, r.D}, r.type);
      dkp = flat(&dk, "dk", r.dev, r.type, {r.T, r.Hk, r.D});
    }
    if (wq) {
      dwq = given_or(a[12], "dq_norm", *r.one, {r.D}, at::kFloat);
      dwqp = flat(&dwq, "dq_norm", r.dev, at::kFloat, {r.D});
    }
    if (wk) {
      dwk = given_or(a[13], "dk_norm", *r.one, {r.D}, at::kFloat);
      dwkp = flat(&dwk, "dk_norm", r.dev, at::kFloat, {r.D});
    }
    const size_t bytes = dflash_qk_norm_rope_workspace_size(&r.d);
    const Workspace ws = workspace(a[14], bytes, *r.one);
    const dflash_status_t st =
        dflash_qk_norm_rope_backward(&r.d, code_of(r.type), r.qp, r.kp, wq, wk, r.cs, r.pos, gq, gk, dqp, dkp,
                                     (float*)dwqp, (float*)dwkp, ws.ptr, bytes, on.stream());
    return st ? status(st) : tuple(dq, dk, dwq, dwk);
  });
}

// A paged batch: caches, table, lengths, offsets.
struct Paged {
  void *kc, *vc;
  const int32_t *table, *lens, *off;
  int64_t Hk, D;
  dflash_paged_dims_t d;
};
Paged paged(PyObject* k_cache, PyObject* v_cache, PyObject* table, PyObject* lens, PyObject* off, int dev,
            at::ScalarType type) {
  Paged p = {};
  const at::Tensor& k = required(k_cache, "k_cache");
  if (k.dim() != 4) refuse("k_cache and v_cache must be [num_pages, page_size, H_kv, D]");
  p.kc = pages(k, "k_cache", dev, type, k.sizes(), &p.d.k_page_stride);
  p.vc = pages(required(v_cache, "v_cache"), "v_cache", dev, type, k.sizes(), &p.d.v_page_stride);
  const at::Tensor &t = required(table, "page_table"), &o = required(off, "q_offsets");
  if (t.dim() != 2 || o.dim() != 1) refuse("page_table must be [R, max_pages] and q_offsets [R + 1]");
  const int64_t R = t.size(0);
  p.table = (const int32_t*)flat(&t, "page_table", dev, at::kInt);
  p.lens = (const int32_t*)flat(&required(lens, "kv_lens"), "kv_lens", dev, at::kInt, {R});
  p.off = (const int32_t*)flat(&o, "q_offsets", dev, at::kInt, {R + 1});
  p.Hk = k.size(2);
  p.D = k.size(3);
  p.d.R = narrow(R);
  p.d.H_kv = narrow(p.Hk);
  p.d.D = narrow(p.D);
  p.d.num_pages = narrow(k.size(0));
  p.d.page_size = narrow(k.size(1));
  p.d.max_pages = narrow(t.size(1));
  return p;
}

// (k, v, k_cache, v_cache, page_table, kv_lens, q_offsets, q, cos_sin, q_norm, k_norm, eps, interleaved, q_out, stream)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const at::Tensor &k = required(a[0], "k"), &v = required(a[1], "v");
    const at::ScalarType type = k.scalar_type();
    const dflash_dtype_t code = code_of(type);
    const int dev = k.get_device();
    Paged p = paged(a[2], a[3], a[4], a[5], a[6], dev, type);
    if (k.dim() != 3) refuse("k and v must be [total_q, H_kv, D]");
    const int64_t T = k.size(0);
    dflash_rope_dims_t d = {};
    int64_t vs = 0;
    const void* kp = tokens(k, "k", dev, type, T, p.Hk, p.D, &d.k_stride);
    const void* vp = tokens(v, "v", dev, type, T, p.Hk, p.D, &vs);
    const On on(dev, a[14]);
    const at::Tensor* q = tensor(a[7], "q");
    int64_t Hq = p.Hk;
    const void* qp = nullptr;
    void* qop = nullptr;
    at::Tensor qo;
    if (q) {
      if (q->dim() != 3) refuse("q must be [total_q, H_q, D]");
      Hq = q->size(1);
      qp = tokens(*q, "q", dev, type, T, Hq, p.D, &d.q_stride);
      qo = given_or(a[13], "q_out", *q, {T, Hq, p.D}, type);
      qop = flat(&qo, "q_out", dev, type, {T, Hq, p.D});
    }
    const float* cs = nullptr;
    if (const at::Tensor* t = tensor(a[8], "cos_sin")) {
      if (t->dim() != 2) refuse("cos_sin must be [max_pos, rot_dim]");
      cs = (const float*)flat(t, "cos_sin", dev, at::kFloat);
      d.max_pos = narrow(t->size(0));
      d.rot_dim = narrow(t->size(1));
    }
    const void* wq = flat(tensor(a[9], "q_norm"), "q_norm", dev, type, {p.D});
    const void* wk = flat(tensor(a[10], "k_norm"), "k_norm", dev, type, {p.D});
    d.eps = real(a[11]);
    d.interleaved = truth(a[12]);
    p.d.H_q = narrow(Hq);
    p.d.total_q = narrow(T);
    const dflash_status_t st = dflash_cache_append(&p.d, &d, code, qp, kp, vp, vs, wq, wk, cs, p.table, p.lens, p.off,
                                                   qop, p.kc, p.vc, on.stream());
    return st ? status(st) : wrap(qo);
  });
}

// Attention over the pages; parents is null for dflash_attn_paged.
PyObject* attend(PyObject* const* a, PyObject* parents, PyObject* max_q_len, int causal, PyObject* const* rest) {
  const at::Tensor& q = required(a[0], "q");
  const at::ScalarType type = q.scalar_type();
  const dflash_dtype_t code = code_of(type);
  if (q.dim() != 3) refuse("q must be [total_q, H_q, D]");
  const int dev = q.get_device();
  Paged p = paged(a[1], a[2], a[3], a[4], a[5], dev, type);
  const int64_t T = q.size(0), Hq = q.size(1);
  const void* qp = flat(&q, "q", dev, type, {T, Hq, p.D});
  const int32_t* up =
      parents ? (const int32_t*)flat(&required(parents, "parents"), "parents", dev, at::kInt, {T}) : nullptr;
  const On on(dev, rest[4]);
  const at::Tensor out = given_or(rest[0], "out", q, {T, Hq, p.D}, type);
  void* op = flat(&out, "out", dev, type, {T, Hq, p.D});
  float* lse = (float*)flat(tensor(rest[1], "lse"), "lse", dev, at::kFloat, {Hq, T});
  p.d.H_q = narrow(Hq);
  p.d.total_q = narrow(T);
  p.d.max_q_len = (int)integer(max_q_len);
  const float scale = rest[2] == Py_None ? 0.f : real(rest[2]);
  const size_t bytes = dflash_attn_paged_workspace_size(&p.d, code);
  const Workspace ws = workspace(rest[3], bytes, q);
  const dflash_status_t st =
      parents ? dflash_attn_tree(&p.d, code, qp, p.kc, p.vc, p.table, p.lens, p.off, up, scale, op, lse, ws.ptr, bytes,
                                 on.stream())
              : dflash_attn_paged(&p.d, code, qp, p.kc, p.vc, p.table, p.lens, p.off, causal, scale, op, lse, ws.ptr,
                                  bytes, on.stream());
  return st ? status(st) : wrap(out);
}

// (q, k_cache, v_cache, page_table, kv_lens, q_offsets, max_q_len, causal, out, lse, scale, workspace, stream)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* { return attend(a, nullptr, a[6], truth(a[7]), a + 8); });
}

// (q, k_cache, v_cache, page_table, kv_lens, q_offsets, parents, max_q_len, out, lse, scale, workspace, stream)
PyObject* attn_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* { return attend(a, a[6], a[7], 1, a + 8); });
}

// (target_probs, draft_probs, draft_tokens, draft_offsets, accept_u, sample_u, max_draft, out_tokens, num_accepted, stream)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &p = required(a[0], "target_probs"), &tok = required(a[2], "draft_tokens"),
                     &off = required(a[3], "draft_offsets");
    const at::Tensor* q = tensor(a[1], "draft_probs");
    if (p.dim() != 2 || (p.size(1) > 1 && p.stride(1) != 1) || tok.dim() != 1 || off.dim() != 1 || off.size(0) < 1)
      refuse("target_probs must be [rows, V] with contiguous rows, draft_tokens [total_draft], draft_offsets [R + 1]");
    const int dev = p.get_device();
    const int64_t rows = p.size(0), V = p.size(1), T = tok.size(0), R = off.size(0) - 1;
    // (a broadcast row, whose stride is 0, would read as contiguous ones)
    if ((rows > 1 && p.stride(0) < V) || (q && q->dim() == 2 && T > 1 && q->stride(0) < V))
      refuse("the rows of target_probs and draft_probs must not overlap");
    if (rows < T + R) refuse("target_probs needs a row for every drafted token and one more for every request");
    common(p, "target_probs", dev, at::kFloat);
    dflash_verify_dims_t d = {};
    const void* qp = nullptr;
    if (q) {
      common(*q, "draft_probs", dev, at::kFloat);
      shaped(*q, "draft_probs", {T, V});
      if (T > 0) {
        if (V > 1 && q->stride(1) != 1) refuse("draft_probs must have contiguous rows");
        qp = q->data_ptr();
        d.draft_stride = T > 1 ? q->stride(0) : 0;
      }
    }
    d.R = narrow(R);
    d.V = narrow(V);
    d.total_draft = narrow(T);
    d.max_draft = (int)integer(a[6]);
    d.target_stride = rows > 1 ? p.stride(0) : 0;
    if (d.max_draft < 0) refuse("max_draft must not be negative");
    const int64_t N = (int64_t)d.max_draft + 1;
    const int32_t* tp = (const int32_t*)flat(&tok, "draft_tokens", dev, at::kInt);
    const int32_t* fp = (const int32_t*)flat(&off, "draft_offsets", dev, at::kInt);
    const float* u = (const float*)flat(&required(a[4], "accept_u"), "accept_u", dev, at::kFloat, {T});
    const float* su = (const float*)flat(&required(a[5], "sample_u"), "sample_u", dev, at::kFloat, {R});
    const On on(dev, a[9]);
    const at::Tensor out = given_or(a[7], "out_tokens", p, {R, N}, at::kInt);
    const at::Tensor acc = given_or(a[8], "num_accepted", p, {R}, at::kInt);
    int32_t* op = (int32_t*)flat(&out, "out_tokens", dev, at::kInt, {R, N});
    int32_t* ap = (int32_t*)flat(&acc, "num_accepted", dev, at::kInt, {R});
    const dflash_status_t st = dflash_verify(&d, (const float*)p.data_ptr(), (const float*)qp, tp, fp, u, su, op, ap,
                                             on.stream());
    return st ? status(st) : tuple(out, acc);
  });
}

// Several int32 results in one allocation (each costs 1.2 us of a call that takes 2 besides):
// views of one buffer, 256 bytes apart.  Those that the caller gives are taken as they are.
class Ints {
 public:
  explicit Ints(const at::Tensor& like) : like_(like) {}
  // A result of this shape, which make() allocates: at(0) for the first, and so on.
  void want(PyObject* given, const char* name, std::vector<int64_t> shape) {
    const at::Tensor* t = tensor(given, name);
    parts_.push_back({t ? *t : at::Tensor(), name, std::move(shape), used_});
    if (t) return;
    int64_t n = 1;
    for (const int64_t d : parts_.back().shape) n *= d;
    used_ += (n + 63) / 64 * 64;
    any_ = true;
  }
  void make(int dev) {
    at::Tensor block;
    if (any_) block = fresh(like_, {used_}, at::kInt);
    for (Part& p : parts_) {
      if (!p.t.defined()) {
        p.t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(), block.dtype());
        p.t.unsafeGetTensorImpl()->set_sizes_contiguous(p.shape);
        p.t.unsafeGetTensorImpl()->set_storage_offset(p.offset);
      }
      common(p.t, p.name, dev, at::kInt);
      if (p.t.sizes() != at::IntArrayRef(p.shape))
        refuse(std::string(p.name) + " must be " + list(p.shape) + ", got " + list(p.t.sizes()));
      if (!p.t.is_contiguous()) refuse(std::string(p.name) + " must be contiguous");
    }
  }
  const at::Tensor& at(int i) const { return parts_[i].t; }
  int32_t* ptr(int i) const { return (int32_t*)parts_[i].t.data_ptr(); }

 private:
  struct Part {
    at::Tensor t;
    const char* name;
    std::vector<int64_t> shape;
    int64_t offset;
  };
  const at::Tensor& like_;
  std::vector<Part> parts_;
  int64_t used_ = 0;
  bool any_ = false;
};

// (logits, u, temperature, top_k, top_p, min_p, probs, tokens, stream)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& x = required(a[0], "logits");
    const at::ScalarType type = x.scalar_type();
    const dflash_dtype_t code = code_of(type);
    const int dev = x.get_device();
    if (x.dim() != 2) refuse("logits must be [N, V]");
    const int64_t N = x.size(0), V = x.size(1);
    common(x, "logits", dev, type);
    dflash_sample_dims_t d = {};
    d.N = narrow(N);
    d.V = narrow(V);
    // rows of [N, V] that are each contiguous and do not overlap
    auto rows = [&](const at::Tensor& t, const char* name) -> int64_t {
      if (t.numel() > 0 && ((V > 1 && t.stride(1) != 1) || (N > 1 && t.stride(0) < V)))
        refuse(std::string("the rows of ") + name + " must be contiguous and must not overlap");
      return N > 1 && t.numel() > 0 ? t.stride(0) : 0;
    };
    d.logits_stride = rows(x, "logits");
    const float* u = (const float*)flat(&required(a[1], "u"), "u", dev, at::kFloat, {N});
    const float* t = (const float*)flat(tensor(a[2], "temperature"), "temperature", dev, at::kFloat, {N});
    const int32_t* k = (const int32_t*)flat(tensor(a[3], "top_k"), "top_k", dev, at::kInt, {N});
    const float* p = (const float*)flat(tensor(a[4], "top_p"), "top_p", dev, at::kFloat, {N});
    const float* m = (const float*)flat(tensor(a[5], "min_p"), "min_p", dev, at::kFloat, {N});
    float* probs = nullptr;
    if (const at::Tensor* o = tensor(a[6], "probs")) {
      common(*o, "probs", dev, at::kFloat);
      shaped(*o, "probs", {N, V});
      d.probs_stride = rows(*o, "probs");
      probs = (float*)o->data_ptr();
    }
    const On on(dev, a[8]);
    const at::Tensor tokens = given_or(a[7], "tokens", x, {N}, at::kInt);
    int32_t* tp = (int32_t*)flat(&tokens, "tokens", dev, at::kInt, {N});
    const dflash_status_t st = dflash_sample(&d, code, x.data_ptr(), u, t, k, p, m, tp, probs, on.stream());
    return st ? status(st) : wrap(tokens);
  });
}

// (sampled, tokens, parents, q_offsets, max_path, path, out_tokens, num_accepted, stream)
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor &smp = required(a[0], "sampled"), &off = required(a[3], "q_offsets");
    if (smp.dim() != 1 || off.dim() != 1 || off.size(0) < 1) refuse("sampled must be [total] and q_offsets [R + 1]");
    const int dev = smp.get_device();
    const int64_t T = smp.size(0), R = off.size(0) - 1;
    dflash_accept_dims_t d = {narrow(R), narrow(T), (int)integer(a[4])};
    if (d.max_path <= 0) refuse("max_path must be positive");
    const int64_t M = d.max_path;
    const int32_t* sp = (const int32_t*)flat(&smp, "sampled", dev, at::kInt);
    const int32_t* tp = (const int32_t*)flat(&required(a[1], "tokens"), "tokens", dev, at::kInt, {T});
    const int32_t* up = (const int32_t*)flat(&required(a[2], "parents"), "parents", dev, at::kInt, {T});
    const int32_t* fp = (const int32_t*)flat(&off, "q_offsets", dev, at::kInt);
    const On on(dev, a[8]);
    Ints r(smp);
    r.want(a[5], "path", {R, M});
    r.want(a[6], "out_tokens", {R, M});
    r.want(a[7], "num_accepted", {R});
    r.make(dev);
    const dflash_status_t st = dflash_tree_accept(&d, sp, tp, up, fp, r.ptr(0), r.ptr(1), r.ptr(2), on.stream());
    return st ? status(st) : tuple(r.at(0), r.at(1), r.at(2));
  });
}

// A cache with or without an axis of layers in front.
struct Cache {
  void *kc, *vc;
  int64_t R;
  at::ScalarType type;
  int dev;
  dflash_paged_dims_t d;
  dflash_layers_t l;
};
void* layered(const at::Tensor& t, const char* name, int dev, at::ScalarType type, at::IntArrayRef shape,
              int64_t* page, int64_t* layer) {
  void* p = pages(t, name, dev, type, shape, page);
  const bool many = t.dim() == 5 && t.size(0) > 1 && t.numel() > 0;
  *layer = many ? t.stride(0) : 0;
  if (many && *layer <= 0) refuse(std::string("the layers of ") + name + " must not overlap");
  return p;
}
Cache cache(PyObject* k_cache, PyObject* v_cache) {
  Cache c = {};
  const at::Tensor& k = required(k_cache, "k_cache");
  if (k.dim() != 4 && k.dim() != 5)
    refuse("k_cache and v_cache must be [num_pages, page_size, H_kv, D] or [L, num_pages, page_size, H_kv, D]");
  c.type = k.scalar_type();
  code_of(c.type);
  c.dev = k.get_device();
  c.kc = layered(k, "k_cache", c.dev, c.type, k.sizes(), &c.d.k_page_stride, &c.l.k_layer_stride);
  c.vc = layered(required(v_cache, "v_cache"), "v_cache", c.dev, c.type, k.sizes(), &c.d.v_page_stride,
                 &c.l.v_layer_stride);
  const at::IntArrayRef s = k.sizes().slice(k.dim() - 4);
  c.l.L = k.dim() == 5 ? narrow(k.size(0)) : 1;
  c.d.num_pages = narrow(s[0]);
  c.d.page_size = narrow(s[1]);
  c.d.H_q = c.d.H_kv = narrow(s[2]);
  c.d.D = narrow(s[3]);
  return c;
}

// (k_cache, v_cache, page_table, kv_lens, q_offsets, path, num_accepted, new_lens, stream)
PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Cache c = cache(a[0], a[1]);
    const at::Tensor &t = required(a[2], "page_table"), &lens = required(a[3], "kv_lens"), &path = required(a[5], "path");
    if (t.dim() != 2 || path.dim() != 2) refuse("page_table must be [R, max_pages] and path [R, max_path]");
    const int64_t R = t.size(0);
    const int32_t* tp = (const int32_t*)flat(&t, "page_table", c.dev, at::kInt);
    const int32_t* lp = (const int32_t*)flat(&lens, "kv_lens", c.dev, at::kInt, {R});
    const int32_t* fp = (const int32_t*)flat(&required(a[4], "q_offsets"), "q_offsets", c.dev, at::kInt, {R + 1});
    const int32_t* pp = (const int32_t*)flat(&path, "path", c.dev, at::kInt, {R, path.size(1)});
    const int32_t* np = (const int32_t*)flat(&required(a[6], "num_accepted"), "num_accepted", c.dev, at::kInt, {R});
    const On on(c.dev, a[8]);
    const at::Tensor out = given_or(a[7], "new_lens", lens, {R}, at::kInt);
    int32_t* op = (int32_t*)flat(&out, "new_lens", c.dev, at::kInt, {R});
    if (R > 0 && op == lp) refuse("new_lens must not be kv_lens");
    c.d.R = narrow(R);
    c.d.max_pages = narrow(t.size(1));
    c.d.total_q = INT32_MAX;  // the packed axis itself is not read
    const dflash_status_t st = dflash_cache_compact(&c.d, &c.l, code_of(c.type), tp, lp, fp, pp, narrow(path.size(1)), np,
                                                    c.kc, c.vc, op, on.stream());
    return st ? status(st) : wrap(out);
  });
}

// (k_cache, v_cache, src_pages, dst_pages, rows, stream)
PyObject* cache_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const Cache c = cache(a[0], a[1]);
    const at::Tensor& src = required(a[2], "src_pages");
    if (src.dim() != 1) refuse("src_pages must be [n]");
    const int64_t N = src.size(0);
    const int32_t* sp = (const int32_t*)flat(&src, "src_pages", c.dev, at::kInt);
    const int32_t* dp = (const int32_t*)flat(&required(a[3], "dst_pages"), "dst_pages", c.dev, at::kInt, {N});
    const int32_t* rp = (const int32_t*)flat(tensor(a[4], "rows"), "rows", c.dev, at::kInt, {N});
    const On on(c.dev, a[5]);
    const dflash_status_t st =
        dflash_cache_copy(&c.d, &c.l, code_of(c.type), narrow(N), sp, dp, rp, c.kc, c.vc, on.stream());
    return st ? status(st) : Py_NewRef(Py_None);
  });
}

// A pool: page table and the pages' counts.
struct Pool {
  int32_t *table, *refs;
  int dev;
  dflash_pool_dims_t d;
};
Pool pool(PyObject* page_table, PyObject* refs, PyObject* page_size) {
  Pool p = {};
  const at::Tensor &t = required(page_table, "page_table"), &c = required(refs, "refs");
  if (t.dim() != 2 || c.dim() != 1) refuse("page_table must be [R, max_pages] and refs [num_pages]");
  p.dev = t.get_device();
  p.table = (int32_t*)flat(&t, "page_table", p.dev, at::kInt);
  p.refs = (int32_t*)flat(&c, "refs", p.dev, at::kInt);
  p.d.R = narrow(t.size(0));
  p.d.max_pages = narrow(t.size(1));
  p.d.num_pages = narrow(c.size(0));
  p.d.page_size = (int)integer(page_size);
  return p;
}

// (page_table, old_lens, new_lens, refs, page_size, missing, workspace, stream)
PyObject* pages_resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Pool p = pool(a[0], a[3], a[4]);
    const at::Tensor& old = required(a[1], "old_lens");
    const int32_t* op = (const int32_t*)flat(&old, "old_lens", p.dev, at::kInt, {p.d.R});
    const int32_t* np = (const int32_t*)flat(&required(a[2], "new_lens"), "new_lens", p.dev, at::kInt, {p.d.R});
    const On on(p.dev, a[7]);
    const at::Tensor missing = given_or(a[5], "missing", old, {1}, at::kInt);
    int32_t* mp = (int32_t*)flat(&missing, "missing", p.dev, at::kInt, {1});
    const size_t bytes = dflash_pages_workspace_size(&p.d);
    const Workspace ws = workspace(a[6], bytes, old);
    const dflash_status_t st = dflash_pages_resize(&p.d, p.table, op, np, p.refs, mp, ws.ptr, bytes, on.stream());
    return st ? status(st) : wrap(missing);
  });
}

// (page_table, lens, src, dst, refs, page_size, copy_src, copy_dst, copy_rows, missing, workspace, stream)
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Pool p = pool(a[0], a[4], a[5]);
    const at::Tensor& src = required(a[2], "src");
    if (src.dim() != 1) refuse("src must be [n]");
    const int64_t N = src.size(0);
    int32_t* lp = (int32_t*)flat(&required(a[1], "lens"), "lens", p.dev, at::kInt, {p.d.R});
    const int32_t* sp = (const int32_t*)flat(&src, "src", p.dev, at::kInt);
    const int32_t* dp = (const int32_t*)flat(&required(a[3], "dst"), "dst", p.dev, at::kInt, {N});
    const On on(p.dev, a[11]);
    const size_t bytes = dflash_pages_workspace_size(&p.d);
    const Workspace ws = workspace(a[10], bytes, src);
    Ints r(src);
    r.want(a[6], "copy_src", {N});
    r.want(a[7], "copy_dst", {N});
    r.want(a[8], "copy_rows", {N});
    r.want(a[9], "missing", {1});
    r.make(p.dev);
    const dflash_status_t st = dflash_pages_fork(&p.d, p.table, lp, narrow(N), sp, dp, p.refs, r.ptr(0), r.ptr(1), r.ptr(2),
                                                 r.ptr(3), ws.ptr, bytes, on.stream());
    return st ? status(st) : tuple(r.at(0), r.at(1), r.at(2), r.at(3));
  });
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(qk_norm_rope), METHOD(qk_norm_rope_backward), METHOD(cache_append), METHOD(attn_paged),
                         METHOD(attn_tree), METHOD(verify), METHOD(sample), METHOD(tree_accept), METHOD(cache_compact),
                         METHOD(cache_copy), METHOD(pages_resize), METHOD(pages_fork), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dflash_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dflash_binding() { return PyModule_Create(&module); }
