// sdpa_binding.cpp -- the paged operators' calls from Python on torch tensors,
// compiled: a call of one token is as long as the host takes to look at its
// arguments, and reading twenty tensors' properties from Python is half of that.
//
// Each function takes what the Python function of its name was given, on the
// current device and stream, and answers Py_NotImplemented for everything that is
// not plainly in order (another device, a wrong type, shape or layout, a status of
// the C entry): the Python function then looks itself and names the error.
//
// Other Python threads run while a call allocates and launches, either of which may
// wait: for memory, for room in a full queue, for a kernel to be loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/sdpa.h"

namespace {

#define NEED(condition) \
  if (!(condition)) Py_RETURN_NOTIMPLEMENTED

// Gives the interpreter's lock up for as long as it lives (an exception takes it back
// on its way out).  What it spans touches no Python object; the arguments' tensors
// stay, the caller holds them.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The call's arguments, in order.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, at = 0;
  int64_t device = -1;
  bool ok = true;

  Args(PyObject* const* args, Py_ssize_t count) : a(args), n(count) {}
  PyObject* next() {
    if (at < n) return a[at++];
    ok = false;
    return Py_None;
  }
  // A CUDA tensor of the device with storage, or null for None.
  const at::Tensor* tensor() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || !t.has_storage() || t.get_device() != device) ok = false;
    return &t;
  }
  const at::Tensor* required() {
    const at::Tensor* t = tensor();
    if (!t) ok = false;
    return ok ? t : nullptr;
  }
  int64_t integer() {
    PyObject* o = next();
    int overflow = 0;
    if (!PyLong_Check(o)) {
      ok = false;
      return 0;
    }
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (overflow != 0) ok = false;
    return v;
  }
  bool truth() {
    PyObject* o = next();
    if (o != Py_True && o != Py_False) ok = false;
    return o == Py_True;
  }
  // NaN for None
  float real() {
    PyObject* o = next();
    if (o == Py_None) return NAN;
    if (!PyFloat_Check(o)) {
      ok = false;
      return 0.0f;
    }
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
  }
  const sdpa_paged_cache* cache() { return reinterpret_cast<const sdpa_paged_cache*>(integer()); }
  // The device that the tensors have to be on: the current one.
  bool on(int64_t d) {
    device = d;
    return d >= 0 && c10::cuda::current_device() == d;
  }
  bool all() const { return ok && at == n; }
};

bool ints(const at::Tensor* t, int64_t n) {
  return t->scalar_type() == at::kInt && t->dim() == 1 && t->size(0) == n && t->is_contiguous();
}
bool floats(const at::Tensor* t, int64_t n) {
  return t->scalar_type() == at::kFloat && t->dim() == 1 && t->size(0) == n && t->is_contiguous();
}
bool table(const at::Tensor* t) {
  return t->scalar_type() == at::kInt && t->dim() == 2 && (t->stride(1) == 1 || t->size(1) == 1);
}
// [tokens, heads, D] of a type with a last stride of 1.
bool rows(const at::Tensor* t, at::ScalarType type) {
  return t->scalar_type() == type && t->dim() == 3 && t->stride(2) == 1;
}
bool code(at::ScalarType type, int elem, sdpa_dtype* dt) {
  if (type != at::kBFloat16 && type != at::kHalf) return false;
  *dt = type == at::kBFloat16 ? SDPA_BF16 : SDPA_FP16;
  return elem < 0 || elem == SDPA_CACHE_E4M3 || elem == static_cast<int>(*dt);
}
bool angles(const at::Tensor* c, const at::Tensor* s) {
  if (!c && !s) return true;
  return c && s && c->scalar_type() == at::kFloat && s->scalar_type() == at::kFloat && c->dim() == 2 && c->sizes() == s->sizes() &&
         c->is_contiguous() && s->is_contiguous();
}
void* at_or_null(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <class T>
T* as(const at::Tensor* t) {
  return static_cast<T*>(at_or_null(t));
}
void* stream(int64_t device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
at::Tensor vector_of(const at::Tensor& like, int64_t n) { return at::empty({n}, like.options()); }

// (cache, device, k, v, page_table, kv_lens, cu_seqlens, cos, sin, interleaved, q, q_out, q_norm, k_norm, eps)
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  const sdpa_paged_cache* cache = a.cache();
  NEED(a.on(a.integer()));
  const at::Tensor *k = a.required(), *v = a.required(), *tab = a.required(), *lens = a.required(), *cu = a.tensor(), *cos = a.tensor(),
                   *sin = a.tensor();
  const bool interleaved = a.truth();
  const at::Tensor *q = a.tensor(), *q_out = a.tensor(), *qn = a.tensor(), *kn = a.tensor();
  const float eps = a.real();
  NEED(a.all());
  sdpa_dtype dt;
  const at::ScalarType type = k->scalar_type();
  NEED(code(type, cache->elem, &dt) && rows(k, type) && rows(v, type) && k->sizes() == v->sizes() && k->size(1) == cache->n_kv_heads &&
       k->size(2) == cache->head_dim && table(tab) && angles(cos, sin) && (q || (!q_out && !qn)));
  const int64_t seqs = tab->size(0), total = k->size(0);
  NEED(ints(lens, seqs) && (!cu || ints(cu, seqs + 1)));
  NEED((!qn || floats(qn, cache->head_dim)) && (!kn || floats(kn, cache->head_dim)));
  NEED(!q || (rows(q, type) && q->size(0) == total && q->size(2) == cache->head_dim));
  NEED(!q_out || (rows(q_out, type) && q_out->sizes() == q->sizes()));
  at::Tensor made;
  sdpa_status status;
  {
    Unlocked others;
    if (q && !q_out) {
      made = at::empty(q->sizes(), q->options());
      q_out = &made;
    }
    const int64_t ks[2] = {k->stride(0), k->stride(1)}, vs[2] = {v->stride(0), v->stride(1)};
    const int64_t qs[2] = {q ? q->stride(0) : 0, q ? q->stride(1) : 0}, os[2] = {q ? q_out->stride(0) : 0, q ? q_out->stride(1) : 0};
    status = sdpa_cache_append_norm(cache, k->data_ptr(), v->data_ptr(), dt, total, ks, vs, as<int32_t>(tab), tab->stride(0), tab->size(1),
                                    as<int32_t>(lens), as<int32_t>(cu), seqs, as<float>(cos), as<float>(sin), cos ? cos->size(0) : 0,
                                    cos ? 2 * cos->size(1) : 0, interleaved, at_or_null(q), at_or_null(q_out), q ? q->size(1) : 0, qs, os,
                                    as<float>(qn), as<float>(kn), eps, stream(a.device));
  }
  NEED(status == SDPA_OK);
  if (!q) Py_RETURN_NONE;
  return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[11]);
  END_HANDLE_TH_ERRORS
}

// (cache, device, q, page_table, kv_lens, cu_seqlens_q, max_seqlen_q, out, is_causal, window, sinks, scale, return_lse, lse);
// cu_seqlens_q None: max_seqlen_q is not used; window 0: none
PyObject* forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  const sdpa_paged_cache* cache = a.cache();
  NEED(a.on(a.integer()));
  const at::Tensor *q = a.required(), *tab = a.required(), *lens = a.required(), *cu = a.tensor();
  int64_t most = a.integer();
  const at::Tensor* out = a.tensor();
  const bool causal = a.truth();
  const int64_t window = a.integer(), sinks = a.integer();
  const float scale = a.real();
  const bool return_lse = a.truth();
  const at::Tensor* lse = a.tensor();
  NEED(a.all());
  sdpa_dtype dt;
  const at::ScalarType type = q->scalar_type();
  NEED(code(type, cache->elem, &dt) && rows(q, type) && q->size(2) == cache->head_dim && table(tab));
  const int64_t seqs = tab->size(0), total = q->size(0), heads = q->size(1);
  NEED(seqs >= 1 && total >= 1 && heads >= 1 && tab->size(1) >= 1 && heads % cache->n_kv_heads == 0);
  NEED(ints(lens, seqs) && (!cu || ints(cu, seqs + 1)) && (cu || total % seqs == 0));
  if (!cu) most = total / seqs;
  NEED(most >= 1 && (window == 0 ? sinks == 0 : causal && window >= 1 && sinks >= 0));
  if (most > total) most = total;
  const uint64_t size = sdpa_paged_workspace_bytes(cache->head_dim, heads, cache->n_kv_heads, most);
  NEED(size != 0);
  NEED(!out || (rows(out, type) && out->sizes() == q->sizes()));
  NEED(!lse || (lse->scalar_type() == at::kFloat && lse->dim() == 2 && lse->size(0) == total && lse->size(1) == heads));
  at::Tensor made, made_lse;
  sdpa_status status;
  {
    Unlocked others;
    if (!out) {
      made = at::empty(q->sizes(), q->options());
      out = &made;
    }
    if (!lse && return_lse) {
      made_lse = at::empty({total, heads}, q->options().dtype(at::kFloat));
      lse = &made_lse;
    }
    const at::Tensor work = at::empty({static_cast<int64_t>(size)}, q->options().dtype(at::kByte));
    const int64_t qs[2] = {q->stride(0), q->stride(1)}, os[2] = {out->stride(0), out->stride(1)};
    const int64_t ls[2] = {lse ? lse->stride(0) : 0, lse ? lse->stride(1) : 0};
    void* const st = stream(a.device);
    status = window == 0 ? sdpa_paged_forward(q->data_ptr(), out->data_ptr(), as<float>(lse), dt, cache, total, heads, qs, os, ls,
                                              as<int32_t>(tab), tab->stride(0), tab->size(1), as<int32_t>(lens), as<int32_t>(cu), seqs,
                                              most, causal, scale, work.data_ptr(), size, st)
                         : sdpa_paged_forward_window(q->data_ptr(), out->data_ptr(), as<float>(lse), dt, cache, total, heads, qs, os, ls,
                                                     as<int32_t>(tab), tab->stride(0), tab->size(1), as<int32_t>(lens), as<int32_t>(cu),
                                                     seqs, most, window, sinks, scale, work.data_ptr(), size, st);
  }
  NEED(status == SDPA_OK);
  PyObject* o = made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[7]);
  if (!lse) return o;
  PyObject* l = made_lse.defined() ? THPVariable_Wrap(made_lse) : Py_NewRef(args[13]);
  PyObject* both = PyTuple_Pack(2, o, l);
  Py_DECREF(o);
  Py_DECREF(l);
  return both;
  END_HANDLE_TH_ERRORS
}

// (device, q, k, positions, cos, sin, interleaved, q_norm, k_norm, eps, q_out, k_out)
PyObject* norm_rotate(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  NEED(a.on(a.integer()));
  const at::Tensor *q = a.required(), *k = a.tensor(), *pos = a.tensor(), *cos = a.tensor(), *sin = a.tensor();
  const bool interleaved = a.truth();
  const at::Tensor *qn = a.tensor(), *kn = a.tensor();
  const float eps = a.real();
  const at::Tensor *q_out = a.tensor(), *k_out = a.tensor();
  NEED(a.all());
  sdpa_dtype dt;
  const at::ScalarType type = q->scalar_type();
  NEED(code(type, -1, &dt) && rows(q, type) && (!k || rows(k, type)) && angles(cos, sin) && (k || (!kn && !k_out)));
  const int64_t total = q->size(0), dim = q->size(2);
  NEED((!k || (k->size(0) == total && k->size(2) == dim)) && (!pos || ints(pos, total)));
  NEED((!qn || floats(qn, dim)) && (!kn || floats(kn, dim)));
  NEED(!q_out || (rows(q_out, type) && q_out->sizes() == q->sizes()));
  NEED(!k_out || (rows(k_out, type) && k_out->sizes() == k->sizes()));
  at::Tensor made_q, made_k;
  sdpa_status status;
  {
    Unlocked others;
    if (!q_out) {
      made_q = at::empty(q->sizes(), q->options());
      q_out = &made_q;
    }
    if (k && !k_out) {
      made_k = at::empty(k->sizes(), k->options());
      k_out = &made_k;
    }
    const int64_t qs[2] = {q->stride(0), q->stride(1)}, qos[2] = {q_out->stride(0), q_out->stride(1)};
    const int64_t ks[2] = {k ? k->stride(0) : 0, k ? k->stride(1) : 0}, kos[2] = {k ? k_out->stride(0) : 0, k ? k_out->stride(1) : 0};
    status = sdpa_norm_rotate(q->data_ptr(), q_out->data_ptr(), q->size(1), qs, qos, at_or_null(k), at_or_null(k_out), k ? k->size(1) : 0,
                              ks, kos, dt, total, dim, as<int32_t>(pos), as<float>(cos), as<float>(sin), cos ? cos->size(0) : 0,
                              cos ? 2 * cos->size(1) : 0, interleaved, as<float>(qn), as<float>(kn), eps, stream(a.device));
  }
  NEED(status == SDPA_OK);
  PyObject* o = made_q.defined() ? THPVariable_Wrap(made_q) : Py_NewRef(args[10]);
  PyObject* l = made_k.defined() ? THPVariable_Wrap(made_k) : Py_NewRef(k ? args[11] : Py_None);
  PyObject* both = PyTuple_Pack(2, o, l);
  Py_DECREF(o);
  Py_DECREF(l);
  return both;
  END_HANDLE_TH_ERRORS
}

bool accounts(const at::Tensor* refs, const at::Tensor* tab) {
  return refs->scalar_type() == at::kInt && refs->dim() == 1 && refs->is_contiguous() && table(tab);
}

// (device, refs, page_table, from_lens, to_lens, page_size)
PyObject* take(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  NEED(a.on(a.integer()));
  const at::Tensor *refs = a.required(), *tab = a.required(), *lo = a.required(), *hi = a.required();
  const int64_t P = a.integer();
  NEED(a.all() && accounts(refs, tab) && ints(lo, tab->size(0)) && ints(hi, tab->size(0)));
  at::Tensor missing;
  sdpa_status status;
  {
    Unlocked others;
    missing = vector_of(*refs, 1);
    status = sdpa_pages_take(as<int32_t>(refs), refs->size(0), as<int32_t>(tab), tab->stride(0), tab->size(0), tab->size(1), P,
                             as<int32_t>(lo), as<int32_t>(hi), as<int32_t>(&missing), stream(a.device));
  }
  NEED(status == SDPA_OK);
  return THPVariable_Wrap(missing);
  END_HANDLE_TH_ERRORS
}

// (device, refs, page_table, kv_lens, src, dst, page_size, new_table); a tuple of four
PyObject* fork_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  NEED(a.on(a.integer()));
  const at::Tensor *refs = a.required(), *tab = a.required(), *lens = a.required(), *src = a.required(), *dst = a.required();
  const int64_t P = a.integer();
  const at::Tensor* to = a.tensor();
  NEED(a.all() && accounts(refs, tab) && ints(lens, tab->size(0)) && src->dim() == 1);
  if (!to) to = tab;
  const int64_t pairs = src->size(0);
  NEED(ints(src, pairs) && ints(dst, pairs) && table(to) && to->size(1) == tab->size(1));
  at::Tensor made[4];
  sdpa_status status;
  {
    Unlocked others;
    for (int i = 0; i < 4; ++i) made[i] = vector_of(*refs, i < 3 ? pairs : 1);
    status = sdpa_pages_fork(as<int32_t>(refs), refs->size(0), as<int32_t>(tab), tab->stride(0), tab->size(0), as<int32_t>(to),
                             to->stride(0), to->size(0), tab->size(1), P, as<int32_t>(lens), as<int32_t>(src), as<int32_t>(dst), pairs,
                             as<int32_t>(&made[0]), as<int32_t>(&made[1]), as<int32_t>(&made[2]), as<int32_t>(&made[3]),
                             stream(a.device));
  }
  NEED(status == SDPA_OK);
  PyObject* four = PyTuple_New(4);
  for (int i = 0; four && i < 4; ++i) PyTuple_SET_ITEM(four, i, THPVariable_Wrap(made[i]));
  return four;
  END_HANDLE_TH_ERRORS
}

// (device, refs, page_table, from_lens, to_lens, page_size, rows)
PyObject* release(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  NEED(a.on(a.integer()));
  const at::Tensor *refs = a.required(), *tab = a.required(), *lo = a.tensor(), *hi = a.tensor();
  const int64_t P = a.integer();
  const at::Tensor* which = a.tensor();
  NEED(a.all() && accounts(refs, tab) && (!which || which->dim() == 1));
  const int64_t count = which ? which->size(0) : tab->size(0);
  NEED((!which || ints(which, count)) && (!lo || ints(lo, count)) && (!hi || ints(hi, count)));
  sdpa_status status;
  {
    Unlocked others;
    status = sdpa_pages_release(as<int32_t>(refs), refs->size(0), as<int32_t>(tab), tab->stride(0), tab->size(0), tab->size(1), P,
                                as<int32_t>(which), as<int32_t>(lo), as<int32_t>(hi), count, stream(a.device));
  }
  NEED(status == SDPA_OK);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (cache, device, src, dst, rows)
PyObject* copy_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  const sdpa_paged_cache* cache = a.cache();
  NEED(a.on(a.integer()));
  const at::Tensor *src = a.required(), *dst = a.required(), *part = a.tensor();
  NEED(a.all() && src->dim() == 1);
  const int64_t count = src->size(0);
  NEED(ints(src, count) && ints(dst, count) && (!part || ints(part, count)));
  sdpa_status status;
  {
    Unlocked others;
    status = sdpa_cache_copy_pages(cache, as<int32_t>(src), as<int32_t>(dst), as<int32_t>(part), count, stream(a.device));
  }
  NEED(status == SDPA_OK);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (cache, device, page_table, kept, new_table, kept_lens)
PyObject* compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n);
  const sdpa_paged_cache* cache = a.cache();
  NEED(a.on(a.integer()));
  const at::Tensor *tab = a.required(), *kept = a.required(), *to = a.required(), *lens = a.tensor();
  NEED(a.all() && table(tab) && table(kept) && table(to));
  const int64_t seqs = tab->size(0);
  NEED(kept->size(0) == seqs && to->size(0) == seqs && (!lens || ints(lens, seqs)));
  sdpa_status status;
  {
    Unlocked others;
    status = sdpa_cache_compact(cache, as<int32_t>(tab), tab->stride(0), tab->size(1), as<int32_t>(kept), kept->stride(0), kept->size(1),
                                as<int32_t>(lens), as<int32_t>(to), to->stride(0), to->size(1), seqs, stream(a.device));
  }
  NEED(status == SDPA_OK);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("append", append),         ENTRY("forward", forward),       ENTRY("norm_rotate", norm_rotate),
                         ENTRY("take", take),             ENTRY("fork", fork_rows),        ENTRY("release", release),
                         ENTRY("copy_pages", copy_pages), ENTRY("compact", compact),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sdpa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sdpa_binding() { return PyModule_Create(&module); }
