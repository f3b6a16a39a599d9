// cache_binding.cpp - the short way from tensors to the cache's C ABI.
//
// A call of a few microseconds on the device is soon outweighed by checking
// its tensors in Python, so the common form of each call (outputs and
// workspace not given, the current stream) is checked and made here.  A
// function returns None, before it does anything, when a call is not of that
// form or a check fails: cache.py then takes it and says what is wrong.
// Otherwise it returns (status code, outputs...).  The entry points' addresses
// come from the loaded library through bind().
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <vector>

#include "psi_verify.h"

namespace {

using at::Tensor;

decltype(&psi_cache_append) call_append;
decltype(&psi_attend_block_workspace_bytes) call_attend_bytes;
decltype(&psi_attend_block) call_attend;
decltype(&psi_cache_commit) call_commit;
decltype(&psi_cache_resize) call_resize;
decltype(&psi_cache_fork_workspace_bytes) call_fork_bytes;
decltype(&psi_cache_fork) call_fork;

// The tensors of one call: each must be a plain CUDA tensor of the current
// device.
struct Call {
  int device = -1;
  bool ok = true;

  const Tensor *tensor(PyObject *o) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) {
      ok = false;
    } else if (device < 0) {
      device = t.get_device();
      ok = ok && device == c10::cuda::current_device();
    } else if (t.get_device() != device) {
      ok = false;
    }
    return &t;
  }
  const Tensor *optional(PyObject *o) { return o == Py_None ? nullptr : tensor(o); }

  psi_stream_t stream() const {
    return reinterpret_cast<psi_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
  }
};

bool is_int32(const Tensor &t, at::IntArrayRef shape) {
  return t.scalar_type() == at::kInt && t.sizes() == shape && t.is_contiguous();
}

// The pools' layout: [P, S, H, D] of one layer, or [L, P, S, H, D].
bool layout_of(const Tensor &k, const Tensor &v, bool layered, psi_cache_layout *c) {
  const int64_t dims = layered ? 5 : 4, at = layered ? 1 : 0;
  if (k.dim() != dims || v.dim() != dims || k.sizes() != v.sizes() || k.strides() != v.strides() ||
      k.scalar_type() != v.scalar_type() || k.stride(-1) != 1)
    return false;
  if (k.scalar_type() == at::kBFloat16)
    c->dtype = PSI_DTYPE_BF16;
  else if (k.scalar_type() == at::kFloat)
    c->dtype = PSI_DTYPE_F32;
  else
    return false;
  const auto size = [&](int64_t d) { return (int32_t)k.size(d); };
  const auto stride = [&](int64_t d) { return k.size(d) == 1 ? 0 : k.stride(d); };
  for (int64_t d = 0; d < dims; ++d)
    if (k.size(d) > INT32_MAX) return false;
  c->layers = layered ? size(0) : 1;
  c->num_pages = size(at);
  c->page_size = size(at + 1);
  c->kv_heads = size(at + 2);
  c->head_dim = size(at + 3);
  c->layer_stride = layered ? stride(0) : 0;
  c->page_stride = stride(at);
  c->slot_stride = stride(at + 1);
  c->head_stride = stride(at + 2);
  return true;
}

// A [N, R, heads, D] tensor with evenly spaced rows.
bool heads_of(const Tensor &t, int64_t N, int64_t R, int64_t heads, int64_t D, at::ScalarType dtype,
              int64_t *row, int64_t *head) {
  if (t.dim() != 4 || t.scalar_type() != dtype || t.size(0) != N || t.size(1) != R ||
      t.size(2) != heads || t.size(3) != D || t.stride(3) != 1)
    return false;
  *row = R > 1 ? t.stride(1) : N > 1 ? t.stride(0) : 0;
  *head = heads > 1 ? t.stride(2) : 0;
  return !(N > 1 && R > 1 && t.stride(0) != R * *row);
}

bool block_of(const Tensor &q, const Tensor &table, const Tensor &lens, const Tensor *parents) {
  if (q.dim() != 4 || table.dim() != 2 || q.size(0) > INT32_MAX || q.size(1) > INT32_MAX ||
      table.size(1) > INT32_MAX || q.size(2) > INT32_MAX)
    return false;
  const int64_t N = q.size(0), R = q.size(1);
  return is_int32(table, {N, table.size(1)}) && is_int32(lens, {N}) &&
         (!parents || is_int32(*parents, {N, R - 1}));
}

Tensor empty(at::IntArrayRef shape, const Tensor &like) { return at::empty(shape, like.options()); }
Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, int device) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, device));
}

// Status words, zeroed many at a time on the stream that uses them; each is
// handed out once, to a later call on that stream.  Two kinds of call get one
// of their own: one that is being captured (its graph zeroes it on every
// replay), and one on a stream that is not torch's, whose handle may be
// another stream's by the next call.
Tensor new_status(const Call &c) {
  const auto zeros = [&](int64_t n) {
    return at::zeros({n}, at::TensorOptions().dtype(at::kInt).device(at::kCUDA, c.device));
  };
  // (a stream from outside is known by its handle)
  const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream(c.device);
  const bool outside = s.id() != 0 && s.id() == reinterpret_cast<int64_t>(s.stream());
  if (outside || c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    return zeros(1);
  static auto *words = new std::map<std::pair<int, void *>, std::vector<Tensor>>;
  std::vector<Tensor> &w = (*words)[{c.device, (void *)s.stream()}];
  if (w.empty()) {
    // later calls may be made outside the inference mode that this one is in
    c10::InferenceMode normal(false);
    w = zeros(256).split(1);
  }
  Tensor t = std::move(w.back());
  w.pop_back();
  return t;
}

template <typename T>
T *ptr(const Tensor *t) {
  return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}
template <typename T>
T *ptr(const Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

PyObject *result(psi_status st, std::initializer_list<const Tensor *> outs) {
  PyObject *r = PyTuple_New(1 + (Py_ssize_t)outs.size());
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
  Py_ssize_t i = 1;
  for (const Tensor *t : outs) {
    PyObject *o = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Exceptions of the allocator and the like become Python's.
template <typename F>
PyObject *guarded(F &&f) {
  try {
    return f();
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

bool number(PyObject *o, double *x) {
  *x = PyFloat_AsDouble(o);
  if (*x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool whole(PyObject *o, int32_t *x) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (over || v < INT32_MIN || v > INT32_MAX) return false;
  *x = (int32_t)v;
  return true;
}

// (q, k, v, k_pages, v_pages, table, lens, q_weight, k_weight, eps, inv_freq,
//  interleaved, rope_scale, parents) -> (status, q, status word)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    Call c;
    const Tensor *q = c.tensor(a[0]), *k = c.tensor(a[1]), *v = c.tensor(a[2]), *kp = c.tensor(a[3]),
                 *vp = c.tensor(a[4]), *table = c.tensor(a[5]), *lens = c.tensor(a[6]),
                 *qw = c.optional(a[7]), *kw = c.optional(a[8]), *freq = c.optional(a[10]),
                 *parents = c.optional(a[13]);
    double eps, scale;
    if (!c.ok || !number(a[9], &eps) || !number(a[12], &scale)) Py_RETURN_NONE;
    psi_cache_layout lay;
    if (!block_of(*q, *table, *lens, parents) || !layout_of(*kp, *vp, false, &lay)) Py_RETURN_NONE;
    const int64_t N = q->size(0), R = q->size(1), Hq = q->size(2), D = lay.head_dim;
    const at::ScalarType dt = kp->scalar_type();
    int64_t s[6];
    if (!heads_of(*q, N, R, Hq, D, dt, s, s + 1) || !heads_of(*k, N, R, lay.kv_heads, D, dt, s + 2, s + 3) ||
        !heads_of(*v, N, R, lay.kv_heads, D, dt, s + 4, s + 5))
      Py_RETURN_NONE;
    for (const Tensor *w : {qw, kw})
      if (w && (w->scalar_type() != dt || w->dim() != 1 || w->size(0) != D || !w->is_contiguous()))
        Py_RETURN_NONE;
    if (freq && (freq->scalar_type() != at::kDouble || freq->dim() != 1 || !freq->is_contiguous() ||
                 freq->size(0) > D))
      Py_RETURN_NONE;
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) return nullptr;
    const Tensor out = empty({N, R, Hq, D}, *q), status = new_status(c);
    const psi_status st = call_append(
        &lay, kp->data_ptr(), vp->data_ptr(), ptr<int32_t>(table), (int32_t)table->size(1),
        ptr<int32_t>(lens), (int32_t)N, (int32_t)R, (int32_t)Hq, q->data_ptr(), s[0], s[1],
        k->data_ptr(), s[2], s[3], v->data_ptr(), s[4], s[5], ptr<void>(qw), ptr<void>(kw),
        (float)eps, ptr<double>(freq), freq ? (int32_t)(2 * freq->size(0)) : 0, interleaved,
        (float)scale, ptr<int32_t>(parents), out.data_ptr(), ptr<uint32_t>(status), c.stream());
    return result(st, {&out, &status});
  });
}

// (q, k_pages, v_pages, table, lens, parents, scale or None, want_lse)
// -> (status, o, lse, status word)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 8) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    Call c;
    const Tensor *q = c.tensor(a[0]), *kp = c.tensor(a[1]), *vp = c.tensor(a[2]), *table = c.tensor(a[3]),
                 *lens = c.tensor(a[4]), *parents = c.optional(a[5]);
    psi_cache_layout lay;
    if (!c.ok || !block_of(*q, *table, *lens, parents) || !layout_of(*kp, *vp, false, &lay))
      Py_RETURN_NONE;
    const int64_t N = q->size(0), R = q->size(1), Hq = q->size(2), D = lay.head_dim;
    int64_t row, head;
    if (!heads_of(*q, N, R, Hq, D, kp->scalar_type(), &row, &head)) Py_RETURN_NONE;
    double scale = 1.0 / std::sqrt((double)D);
    if (a[6] != Py_None && !number(a[6], &scale)) Py_RETURN_NONE;
    const int want_lse = PyObject_IsTrue(a[7]);
    if (want_lse < 0) return nullptr;
    const int32_t max_pages = (int32_t)table->size(1);
    const size_t bytes = call_attend_bytes(&lay, (int32_t)N, (int32_t)R, (int32_t)Hq, max_pages);
    if (bytes == 0) Py_RETURN_NONE;  // (sizes that the call refuses)
    const Tensor out = empty({N, R, Hq, D}, *q), status = new_status(c),
                 ws = empty({(int64_t)bytes}, at::kByte, c.device);
    const Tensor lse = want_lse ? empty({N, R, Hq}, at::kFloat, c.device) : Tensor();
    const psi_status st = call_attend(
        &lay, kp->data_ptr(), vp->data_ptr(), ptr<int32_t>(table), max_pages, ptr<int32_t>(lens),
        (int32_t)N, (int32_t)R, (int32_t)Hq, q->data_ptr(), row, head, ptr<int32_t>(parents),
        (float)scale, out.data_ptr(), want_lse ? ptr<float>(lse) : nullptr, ptr<uint32_t>(status),
        ws.data_ptr(), bytes, c.stream());
    return result(st, {&out, want_lse ? &lse : nullptr, &status});
  });
}

// (k_pages, v_pages, table, lens, path_nodes, path_len) -> (status, lens, status word)
PyObject *commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 6) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    Call c;
    const Tensor *kp = c.tensor(a[0]), *vp = c.tensor(a[1]), *table = c.tensor(a[2]), *lens = c.tensor(a[3]),
                 *nodes = c.tensor(a[4]), *steps = c.tensor(a[5]);
    psi_cache_layout lay;
    if (!c.ok || !layout_of(*kp, *vp, true, &lay) || table->dim() != 2 || nodes->dim() != 2 ||
        nodes->size(0) > INT32_MAX || nodes->size(1) > INT32_MAX || table->size(1) > INT32_MAX)
      Py_RETURN_NONE;
    const int64_t N = nodes->size(0), M = nodes->size(1);
    if (!is_int32(*table, {N, table->size(1)}) || !is_int32(*lens, {N}) || !is_int32(*nodes, {N, M}) ||
        !is_int32(*steps, {N}))
      Py_RETURN_NONE;
    const Tensor out = empty({N}, *lens), status = new_status(c);
    const psi_status st = call_commit(&lay, kp->data_ptr(), vp->data_ptr(), ptr<int32_t>(table),
                                      (int32_t)table->size(1), ptr<int32_t>(lens), (int32_t)N,
                                      (int32_t)M, ptr<int32_t>(nodes), ptr<int32_t>(steps),
                                      ptr<int32_t>(out), ptr<uint32_t>(status), c.stream());
    return result(st, {&out, &status});
  });
}

// A page state from its five tensors, and a new one of the same sizes.
struct State {
  const Tensor *t[5];  // table, counts, refs, free, n_free
  int64_t N = 0, max_pages = 0, P = 0;

  bool take(Call &c, PyObject *const *a) {
    for (int i = 0; i < 5; ++i) t[i] = c.tensor(a[i]);
    if (!c.ok || t[0]->dim() != 2) return false;
    N = t[0]->size(0);
    max_pages = t[0]->size(1);
    P = t[2]->numel();
    return N <= INT32_MAX && max_pages <= INT32_MAX && P <= INT32_MAX &&
           is_int32(*t[0], {N, max_pages}) && is_int32(*t[1], {N}) && is_int32(*t[2], {P}) &&
           is_int32(*t[3], {P}) && is_int32(*t[4], {1});
  }
  static psi_page_state ptrs(const Tensor *const *t) {
    return {ptr<int32_t>(t[0]), ptr<int32_t>(t[1]), ptr<int32_t>(t[2]), ptr<int32_t>(t[3]),
            ptr<int32_t>(t[4])};
  }
  // one allocation for all five
  std::vector<Tensor> like() const {
    const Tensor all = empty({N * max_pages + 2 * P + N + 1}, *t[0]);
    const int64_t at[5] = {0, N * max_pages + 2 * P, N * max_pages, N * max_pages + P,
                           N * max_pages + 2 * P + N};
    const int64_t len[5] = {N * max_pages, N, P, P, 1};
    std::vector<Tensor> r;
    for (int i = 0; i < 5; ++i)
      r.push_back(i == 0 ? all.as_strided({N, max_pages}, {max_pages, 1}, 0)
                         : all.as_strided({len[i]}, {1}, at[i]));
    return r;
  }
};

// (table, counts, refs, free, n_free, lens, extra, page_size)
// -> (status, table, counts, refs, free, n_free, status word)
PyObject *resize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 8) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    Call c;
    State s;
    int32_t extra, page_size;
    if (!s.take(c, a) || !whole(a[6], &extra) || !whole(a[7], &page_size)) Py_RETURN_NONE;
    const Tensor *lens = c.tensor(a[5]);
    if (!c.ok || !is_int32(*lens, {s.N})) Py_RETURN_NONE;
    const std::vector<Tensor> o = s.like();
    const Tensor *outs[5] = {&o[0], &o[1], &o[2], &o[3], &o[4]};
    const Tensor status = new_status(c);
    const psi_page_state in = State::ptrs(s.t), out = State::ptrs(outs);
    const psi_status st = call_resize((int32_t)s.N, (int32_t)s.max_pages, (int32_t)s.P, page_size,
                                      ptr<int32_t>(lens), extra, &in, &out, ptr<uint32_t>(status),
                                      c.stream());
    return result(st, {outs[0], outs[1], outs[2], outs[3], outs[4], &status});
  });
}

// (k_pages, v_pages, table, counts, refs, free, n_free, lens, src, dst)
// -> (status, table, counts, refs, free, n_free, lens, status word)
PyObject *fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 10) Py_RETURN_NONE;
  return guarded([&]() -> PyObject * {
    Call c;
    const Tensor *kp = c.tensor(a[0]), *vp = c.tensor(a[1]);
    State s;
    psi_cache_layout lay;
    if (!s.take(c, a + 2) || !layout_of(*kp, *vp, true, &lay) || s.P != lay.num_pages) Py_RETURN_NONE;
    const Tensor *lens = c.tensor(a[7]), *src = c.tensor(a[8]), *dst = c.tensor(a[9]);
    if (!c.ok || src->dim() != 1 || src->size(0) > INT32_MAX) Py_RETURN_NONE;
    const int64_t K = src->size(0);
    if (!is_int32(*lens, {s.N}) || !is_int32(*src, {K}) || !is_int32(*dst, {K})) Py_RETURN_NONE;
    const size_t bytes = call_fork_bytes((int32_t)K);
    if (bytes == 0) Py_RETURN_NONE;  // (sizes that the call refuses)
    const std::vector<Tensor> o = s.like();
    const Tensor *outs[5] = {&o[0], &o[1], &o[2], &o[3], &o[4]};
    const Tensor out_lens = empty({s.N}, *lens), status = new_status(c),
                 ws = empty({(int64_t)bytes}, at::kByte, c.device);
    const psi_page_state in = State::ptrs(s.t), out = State::ptrs(outs);
    const psi_status st = call_fork(&lay, kp->data_ptr(), vp->data_ptr(), (int32_t)s.N,
                                    (int32_t)s.max_pages, ptr<int32_t>(lens), ptr<int32_t>(out_lens),
                                    &in, &out, (int32_t)K, ptr<int32_t>(src), ptr<int32_t>(dst),
                                    ptr<uint32_t>(status), ws.data_ptr(), bytes, c.stream());
    return result(st, {outs[0], outs[1], outs[2], outs[3], outs[4], &out_lens, &status});
  });
}

// bind(addresses of the entry points, in the order below)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *p[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes 7 addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  call_append = reinterpret_cast<decltype(call_append)>(p[0]);
  call_attend_bytes = reinterpret_cast<decltype(call_attend_bytes)>(p[1]);
  call_attend = reinterpret_cast<decltype(call_attend)>(p[2]);
  call_commit = reinterpret_cast<decltype(call_commit)>(p[3]);
  call_resize = reinterpret_cast<decltype(call_resize)>(p[4]);
  call_fork_bytes = reinterpret_cast<decltype(call_fork_bytes)>(p[5]);
  call_fork = reinterpret_cast<decltype(call_fork)>(p[6]);
  Py_RETURN_NONE;
}

#define PSI_METHOD(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {PSI_METHOD(bind),   PSI_METHOD(append), PSI_METHOD(attend), PSI_METHOD(commit),
                         PSI_METHOD(resize), PSI_METHOD(fork),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, methods, nullptr, nullptr,
                      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding() { return PyModule_Create(&module); }
