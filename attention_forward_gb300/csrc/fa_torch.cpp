// fa_torch.cpp -- the calls on 16-bit paged caches and latent attention, from torch
// tensors: what fa.py's functions of these names do for the plain call, on the current
// stream with outputs and workspace of its own, in compiled code.  Whatever is not that,
// or not as it should be, comes back as NotImplemented, and fa.py goes through it: it
// refuses what is wrong, by name, and serves other devices, streams, captures and given
// outputs.  (On a Grace host a call of fa_fwd_paged takes 18 us through ctypes: 5 for the
// launches, 4 for two output tensors, the rest for checks and arguments.)
//
// It calls the library by the addresses that bind() is given.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>

#include "../../include/fa.h"

namespace {

struct Library {
  decltype(&fa_paged_write) paged_write;
  decltype(&fa_paged_read) paged_read;
  decltype(&fa_fwd_paged) fwd_paged;
  decltype(&fa_latent_write) latent_write;
  decltype(&fa_latent_read) latent_read;
  decltype(&fa_fwd_latent) fwd_latent;
  decltype(&fa_fwd_expanded) fwd_expanded;
} lib;

constexpr int64_t kLatent = 512, kRope = 64, kRow = kLatent + kRope, kNope = 128;
const double kLatentScale = std::pow(192.0, -0.5);

PyObject* not_taken() { Py_RETURN_NOTIMPLEMENTED; }

// The tensor behind an argument; null where it is none of torch's own.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

// A tensor's memory.  Throws where it has none: its address would be taken for that of an
// argument left out (a tensor under torch.func.functionalize is at 0).
void* memory(const at::Tensor& t) {
  void* at = t.data_ptr();
  if (!at && t.numel() > 0) throw std::invalid_argument("a tensor without memory");
  return at;
}

// A contiguous tensor of that type, device and shape.
bool is(const at::Tensor* t, c10::ScalarType type, int dev, at::IntArrayRef shape) {
  return t && t->is_cuda() && t->scalar_type() == type && t->get_device() == dev &&
         t->sizes() == shape && t->is_contiguous();
}

// The first tensor of a call: contiguous, 16 bits, of so many dimensions, on the current
// device, whose current stream is not being captured.
bool leads(const at::Tensor* t, int64_t dims) {
  return t && t->is_cuda() && t->dim() == dims &&
         (t->scalar_type() == at::kHalf || t->scalar_type() == at::kBFloat16) && t->is_contiguous() &&
         t->get_device() == c10::cuda::current_device() &&
         c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None;
}

int dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? FA_BF16 : FA_F16; }

fa_stream_t stream_of(const at::Tensor& t) {
  return reinterpret_cast<fa_stream_t>(
      c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(t.get_device())).stream());
}

// An optional [n] tensor's pointer; false where it is something else.
template <class T>
bool optional(PyObject* o, c10::ScalarType type, int dev, int64_t n, const T** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!is(t, type, dev, {n})) return false;
  *out = static_cast<const T*>(memory(*t));
  return true;
}

bool number(PyObject* o, double* out) {
  if (PyFloat_CheckExact(o)) {
    *out = PyFloat_AS_DOUBLE(o);
    return true;
  }
  if (!PyLong_CheckExact(o)) return false;
  *out = PyLong_AsDouble(o);
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// A pair's items (a tuple's or a list's).
bool pair(PyObject* o, PyObject** a, PyObject** b) {
  if (!(PyTuple_CheckExact(o) || PyList_CheckExact(o)) || PySequence_Fast_GET_SIZE(o) != 2) return false;
  *a = PySequence_Fast_GET_ITEM(o, 0);
  *b = PySequence_Fast_GET_ITEM(o, 1);
  return true;
}

// An int argument of the library.
bool fits(int64_t n) { return n >= 0 && n <= 0x7fffffff; }
bool all_fit(const at::Tensor& t) {
  for (int64_t n : t.sizes())
    if (!fits(n)) return false;
  return true;
}

struct Pages {
  const int *table, *start, *count;
  int num, size, max;
};

// page_table [B, n], and start and count where they are given.
bool places(PyObject* table, PyObject* start, PyObject* count, int dev, int64_t B, Pages* p) {
  const at::Tensor* t = tensor(table);
  if (!t || t->dim() != 2 || !is(t, at::kInt, dev, {B, t->size(1)}) || !all_fit(*t)) return false;
  p->table = static_cast<const int*>(memory(*t));
  p->max = static_cast<int>(t->size(1));
  return optional(start, at::kInt, dev, B, &p->start) && optional(count, at::kInt, dev, B, &p->count);
}

// (k_pages, v_pages) of Hkv heads of D channels.
bool pools(PyObject* cache, const at::Tensor& like, int64_t Hkv, int64_t D, void** k, void** v, Pages* p) {
  PyObject *a, *b;
  if (!pair(cache, &a, &b)) return false;
  const at::Tensor *kp = tensor(a), *vp = tensor(b);
  if (!kp || kp->dim() != 4 || !all_fit(*kp)) return false;
  const int64_t shape[4] = {kp->size(0), Hkv, kp->size(2), D};
  const int dev = like.get_device();
  if (!is(kp, like.scalar_type(), dev, shape) || !is(vp, like.scalar_type(), dev, shape)) return false;
  *k = memory(*kp);
  *v = memory(*vp);
  p->num = static_cast<int>(shape[0]);
  p->size = static_cast<int>(shape[2]);
  return true;
}

bool latent_pool(PyObject* cache, const at::Tensor& like, void** pool, Pages* p) {
  const at::Tensor* t = tensor(cache);
  if (!t || t->dim() != 3 || !all_fit(*t) ||
      !is(t, like.scalar_type(), like.get_device(), {t->size(0), t->size(1), kRow}))
    return false;
  *pool = memory(*t);
  p->num = static_cast<int>(t->size(0));
  p->size = static_cast<int>(t->size(1));
  return true;
}

// c [B, S, 512] and k_rope [B, S, 64].
bool latent_rows(const at::Tensor* c, const at::Tensor* r) {
  return leads(c, 3) && all_fit(*c) && c->size(2) == kLatent &&
         is(r, c->scalar_type(), c->get_device(), {c->size(0), c->size(1), kRope});
}

// The interpreter's lock given up, and back however the scope is left.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// A call of the library without the interpreter's lock; true where its work is in the
// stream.  The arguments are evaluated by the caller, under the lock: a tensor without
// storage (under torch.vmap and the like) throws where its address is asked for.
template <class Call, class... Args>
bool launched(Call call, Args... args) {
  Unlocked unlocked;
  return call(args...) == FA_OK;
}

// Torch's errors (no memory, tensors without storage) are fa.py's to meet again.
template <class Body>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, Body body) {
  if (n != want) return not_taken();
  try {
    return body();
  } catch (...) {
    PyErr_Clear();
    return not_taken();
  }
}

PyObject* outputs(const at::Tensor& o, const at::Tensor& lse) {
  PyObject *a = THPVariable_Wrap(o), *b = a ? THPVariable_Wrap(lse) : nullptr;
  PyObject* r = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

int n32(int64_t n) { return static_cast<int>(n); }

// (q, cache, page_table, length, scale, softcap, slopes) -> (o, lse)
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor* q = tensor(a[0]);
    if (!leads(q, 4) || !all_fit(*q)) return not_taken();
    const int64_t B = q->size(0), H = q->size(1), Sq = q->size(2), D = q->size(3);
    const int dev = q->get_device();
    PyObject *first, *second;
    const at::Tensor* kp = pair(a[1], &first, &second) ? tensor(first) : nullptr;
    if (!kp || kp->dim() != 4) return not_taken();
    const int64_t Hkv = kp->size(1);
    Pages p{};
    void *k, *v;
    const float* slopes;
    double scale, cap;
    if (Hkv < 1 || H % Hkv != 0 || !pools(a[1], *q, Hkv, D, &k, &v, &p) ||
        !places(a[2], a[3], Py_None, dev, B, &p) || !p.start || !number(a[5], &cap) ||
        !optional(a[6], at::kFloat, dev, H, &slopes))
      return not_taken();
    if (a[4] == Py_None)
      scale = std::pow(static_cast<double>(D), -0.5);
    else if (!number(a[4], &scale))
      return not_taken();
    at::Tensor o = at::empty_like(*q), lse = at::empty({B, H, Sq}, q->options().dtype(at::kFloat));
    const bool ok = launched(lib.fwd_paged, memory(*q), k, v, p.table, p.start, memory(o),
                             static_cast<float*>(memory(lse)), n32(B), n32(H), n32(Hkv), n32(Sq), n32(D),
                             p.num, p.size, p.max, static_cast<float>(scale), dtype_of(*q),
                             static_cast<float>(cap), slopes, nullptr, 0, stream_of(*q));
    return ok ? outputs(o, lse) : not_taken();
  });
}

// (q, cache, page_table, length, scale) -> (o, lse)
PyObject* fwd_latent(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor* q = tensor(a[0]);
    if (!leads(q, 4) || !all_fit(*q) || q->size(3) != kRow) return not_taken();
    const int64_t B = q->size(0), H = q->size(1), Sq = q->size(2);
    Pages p{};
    void* pool;
    double scale = kLatentScale;
    if (!latent_pool(a[1], *q, &pool, &p) || !places(a[2], a[3], Py_None, q->get_device(), B, &p) ||
        !p.start || (a[4] != Py_None && !number(a[4], &scale)))
      return not_taken();
    at::Tensor o = at::empty({B, H, Sq, kLatent}, q->options());
    at::Tensor lse = at::empty({B, H, Sq}, q->options().dtype(at::kFloat));
    const bool ok = launched(lib.fwd_latent, memory(*q), pool, p.table, p.start, memory(o),
                             static_cast<float*>(memory(lse)), n32(B), n32(H), n32(Sq), p.num, p.size,
                             p.max, static_cast<float>(scale), dtype_of(*q), nullptr, 0, stream_of(*q));
    return ok ? outputs(o, lse) : not_taken();
  });
}

// (q, kv, k_rope, causal, scale) -> (o, lse)
PyObject* fwd_expanded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor *q = tensor(a[0]), *kv = tensor(a[1]), *r = tensor(a[2]);
    if (!leads(q, 4) || !all_fit(*q) || q->size(3) != kNope + kRope || !kv || kv->dim() != 4 || !all_fit(*kv))
      return not_taken();
    const int64_t B = q->size(0), H = q->size(1), Sq = q->size(2), Skv = kv->size(2);
    const int dev = q->get_device();
    double scale = kLatentScale;
    if (!is(kv, q->scalar_type(), dev, {B, H, Skv, 2 * kNope}) ||
        !is(r, q->scalar_type(), dev, {B, Skv, kRope}) || !PyBool_Check(a[3]) ||
        (a[4] != Py_None && !number(a[4], &scale)))
      return not_taken();
    at::Tensor o = at::empty({B, H, Sq, kNope}, q->options());
    at::Tensor lse = at::empty({B, H, Sq}, q->options().dtype(at::kFloat));
    const bool ok = launched(lib.fwd_expanded, memory(*q), memory(*kv), memory(*r), memory(o),
                             static_cast<float*>(memory(lse)), n32(B), n32(H), n32(Sq), n32(Skv),
                             static_cast<float>(scale), a[3] == Py_True, dtype_of(*q), nullptr, 0,
                             stream_of(*q));
    return ok ? outputs(o, lse) : not_taken();
  });
}

// (k, v, cache, page_table, start, count, freqs, interleaved, q, q_out) -> None; q and
// q_out are both given, or both None
PyObject* paged_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]);
    if (!leads(k, 4) || !all_fit(*k)) return not_taken();
    const int64_t B = k->size(0), Hkv = k->size(1), S = k->size(2), D = k->size(3);
    const int dev = k->get_device();
    Pages p{};
    void *kp, *vp;
    if (!is(v, k->scalar_type(), dev, k->sizes()) || !pools(a[2], *k, Hkv, D, &kp, &vp, &p) ||
        !places(a[3], a[4], a[5], dev, B, &p) || !PyBool_Check(a[7]))
      return not_taken();
    const float* freqs = nullptr;
    int64_t rotary = 0;
    if (a[6] != Py_None) {
      const at::Tensor* f = tensor(a[6]);
      if (!f || f->dim() != 1 || f->size(0) > 1024 || !optional(a[6], at::kFloat, dev, f->size(0), &freqs))
        return not_taken();
      rotary = 2 * f->size(0);
    }
    const void* q = nullptr;
    void* q_out = nullptr;
    int64_t H = Hkv;
    if ((a[8] == Py_None) != (a[9] == Py_None)) return not_taken();
    if (a[8] != Py_None) {
      const at::Tensor *t = tensor(a[8]), *o = tensor(a[9]);
      if (!t || t->dim() != 4 || !all_fit(*t)) return not_taken();
      H = t->size(1);
      if (Hkv < 1 || H % Hkv != 0 || !is(t, k->scalar_type(), dev, {B, H, S, D}) ||
          !is(o, k->scalar_type(), dev, t->sizes()))
        return not_taken();
      q = memory(*t);
      q_out = memory(*o);
    }
    const bool ok = launched(lib.paged_write, q, memory(*k), memory(*v), q_out, kp, vp, p.table,
                             p.start, p.count, freqs, n32(rotary), a[7] == Py_True, n32(B), n32(H),
                             n32(Hkv), n32(S), n32(D), p.num, p.size, p.max, dtype_of(*k), stream_of(*k));
    if (!ok) return not_taken();
    Py_RETURN_NONE;
  });
}

// (cache, page_table, start, count, out) -> None
PyObject* paged_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    PyObject *first, *second;
    if (!pair(a[4], &first, &second)) return not_taken();
    const at::Tensor *k = tensor(first), *v = tensor(second);
    if (!leads(k, 4) || !all_fit(*k)) return not_taken();
    const int64_t B = k->size(0), Hkv = k->size(1), S = k->size(2), D = k->size(3);
    const int dev = k->get_device();
    Pages p{};
    void *kp, *vp;
    if (!is(v, k->scalar_type(), dev, k->sizes()) || !pools(a[0], *k, Hkv, D, &kp, &vp, &p) ||
        !places(a[1], a[2], a[3], dev, B, &p))
      return not_taken();
    const bool ok = launched(lib.paged_read, kp, vp, p.table, p.start, p.count, memory(*k),
                             memory(*v), n32(B), n32(Hkv), n32(S), n32(D), p.num, p.size, p.max,
                             dtype_of(*k), stream_of(*k));
    if (!ok) return not_taken();
    Py_RETURN_NONE;
  });
}

// (c, k_rope, cache, page_table, start, count, freqs, interleaved, q_rope, q) -> None
PyObject* latent_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor *c = tensor(a[0]), *r = tensor(a[1]);
    if (!latent_rows(c, r)) return not_taken();
    const int64_t B = c->size(0), S = c->size(1);
    const int dev = c->get_device();
    Pages p{};
    void* pool;
    const float* freqs;
    if (!latent_pool(a[2], *c, &pool, &p) || !places(a[3], a[4], a[5], dev, B, &p) ||
        !optional(a[6], at::kFloat, dev, kRope / 2, &freqs) || !PyBool_Check(a[7]) ||
        (a[8] == Py_None) != (a[9] == Py_None))
      return not_taken();
    const void* q_rope = nullptr;
    void* q = nullptr;
    int64_t H = 0, width = 0;
    if (a[9] != Py_None) {
      const at::Tensor *t = tensor(a[8]), *o = tensor(a[9]);
      if (!o || o->dim() != 4 || !all_fit(*o)) return not_taken();
      H = o->size(1);
      width = o->size(3);
      if (!is(o, c->scalar_type(), dev, {B, H, S, width}) || !is(t, c->scalar_type(), dev, {B, H, S, kRope}))
        return not_taken();
      q_rope = memory(*t);
      q = memory(*o);
    }
    const bool ok = launched(lib.latent_write, memory(*c), memory(*r), pool, q_rope, q, p.table,
                             p.start, p.count, freqs, a[7] == Py_True, n32(B), n32(H), n32(S), n32(width),
                             p.num, p.size, p.max, dtype_of(*c), stream_of(*c));
    if (!ok) return not_taken();
    Py_RETURN_NONE;
  });
}

// (cache, page_table, start, count, out) -> None
PyObject* latent_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    PyObject *first, *second;
    if (!pair(a[4], &first, &second)) return not_taken();
    const at::Tensor *c = tensor(first), *r = tensor(second);
    if (!latent_rows(c, r)) return not_taken();
    Pages p{};
    void* pool;
    if (!latent_pool(a[0], *c, &pool, &p) || !places(a[1], a[2], a[3], c->get_device(), c->size(0), &p))
      return not_taken();
    const bool ok = launched(lib.latent_read, pool, p.table, p.start, p.count, memory(*c), memory(*r),
                             n32(c->size(0)), n32(c->size(1)), p.num, p.size, p.max, dtype_of(*c),
                             stream_of(*c));
    if (!ok) return not_taken();
    Py_RETURN_NONE;
  });
}

// The addresses of the library's functions, in the order of Library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  lib.paged_write = reinterpret_cast<decltype(lib.paged_write)>(at[0]);
  lib.paged_read = reinterpret_cast<decltype(lib.paged_read)>(at[1]);
  lib.fwd_paged = reinterpret_cast<decltype(lib.fwd_paged)>(at[2]);
  lib.latent_write = reinterpret_cast<decltype(lib.latent_write)>(at[3]);
  lib.latent_read = reinterpret_cast<decltype(lib.latent_read)>(at[4]);
  lib.fwd_latent = reinterpret_cast<decltype(lib.fwd_latent)>(at[5]);
  lib.fwd_expanded = reinterpret_cast<decltype(lib.fwd_expanded)>(at[6]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"paged_write", fast(paged_write), METH_FASTCALL, nullptr},
                         {"paged_read", fast(paged_read), METH_FASTCALL, nullptr},
                         {"fwd_paged", fast(fwd_paged), METH_FASTCALL, nullptr},
                         {"latent_write", fast(latent_write), METH_FASTCALL, nullptr},
                         {"latent_read", fast(latent_read), METH_FASTCALL, nullptr},
                         {"fwd_latent", fast(fwd_latent), METH_FASTCALL, nullptr},
                         {"fwd_expanded", fast(fwd_expanded), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
