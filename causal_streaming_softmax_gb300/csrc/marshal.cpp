// marshal.cpp - the serving calls of api.py from PyTorch tensors to the C ABI
// in one step, for the ordinary case: tensors of the current device, the
// current stream.
//
// A token step's kernels take a few microseconds, and looking at a call's
// tensors attribute by attribute from Python takes as long again (attn_paged_fwd
// 12 us a call that way).  These functions make the checks that api.py makes;
// where one fails, or the case is not the ordinary one, they return None
// without having done anything, and api.py's own path goes on from there: it
// names what is wrong, or handles the rest.
//
// The objects are read through PyTorch's headers: built_for names the PyTorch
// and Python that they belong to, and api.py binds the entry points only where
// those are the ones that run.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn.h"

namespace {

struct {
  decltype(&attn_packed_fwd) packed_fwd;
  decltype(&attn_paged_plan) paged_plan;
  decltype(&attn_paged_store) paged_store;
  decltype(&attn_paged_fwd) paged_fwd;
} entry;

enum Name {
  TOKENS, BATCH, HEADS, KV_HEADS, CAUSAL, SCALE, DTYPE, PAGE_SIZE, NUM_PAGES, TABLE_WIDTH, MAX_NEW,
  NAMES
};
const char* const kNames[NAMES] = {"tokens", "batch", "heads", "kv_heads", "causal", "scale",
                                   "dtype", "page_size", "num_pages", "table_width", "max_new"};
PyObject* names[NAMES];

// An int attribute of the shape that fits 32 bits.
bool get(PyObject* s, Name n, int32_t* out) {
  PyObject* v = PyObject_GetAttr(s, names[n]);
  if (!v) return false;
  const bool is_int = PyLong_Check(v);
  const long long x = is_int ? PyLong_AsLongLong(v) : 0;
  Py_DECREF(v);
  *out = static_cast<int32_t>(x);
  return is_int && !PyErr_Occurred() && x == *out;
}

bool get_scale(PyObject* s, float* out) {
  PyObject* v = PyObject_GetAttr(s, names[SCALE]);
  if (!v) return false;
  const double x = PyFloat_AsDouble(v);
  Py_DECREF(v);
  *out = static_cast<float>(x);
  return !PyErr_Occurred();
}

bool get_dtype(PyObject* s, at::ScalarType* type, int32_t* code) {
  PyObject* v = PyObject_GetAttr(s, names[DTYPE]);
  if (!v) return false;
  const bool ok = THPDtype_Check(v);
  if (ok) *type = reinterpret_cast<THPDtype*>(v)->scalar_type;
  Py_DECREF(v);
  *code = ok && *type == at::kBFloat16 ? ATTN_BF16 : ATTN_F16;
  return ok && (*type == at::kHalf || *type == at::kBFloat16);
}

// The common device of a call's tensors: the first one's, if it is current.
struct Call {
  int dev = -1;
  bool ok = true;

  const at::Tensor* tensor(PyObject* o, at::ScalarType type) {
    if (!ok) return nullptr;
    if (!THPVariable_Check(o)) return ok = false, nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || t.layout() != at::kStrided)
      return ok = false, nullptr;
    if (dev < 0) {
      dev = t.get_device();
      if (dev != c10::cuda::current_device()) ok = false;
    } else if (t.get_device() != dev) {
      ok = false;
    }
    return ok ? &t : nullptr;
  }

  // [d0][d1][64], any strides over the first two
  void* rows(PyObject* o, at::ScalarType type, int64_t d0, int64_t d1, int64_t* s0, int64_t* s1) {
    const at::Tensor* t = tensor(o, type);
    if (!t) return nullptr;
    const auto z = t->sizes(), s = t->strides();
    if (z.size() != 3 || z[0] != d0 || z[1] != d1 || z[2] != 64 || s[2] != 1)
      return ok = false, nullptr;
    *s0 = s[0];
    *s1 = s[1];
    return t->data_ptr();
  }

  // [pages][kv heads][page size][64], any strides over the first three
  void* pool(PyObject* o, at::ScalarType type, const attn_paged_shape& p, int64_t* s0, int64_t* s1,
             int64_t* s2) {
    const at::Tensor* t = tensor(o, type);
    if (!t) return nullptr;
    const auto z = t->sizes(), s = t->strides();
    if (z.size() != 4 || z[0] != p.num_pages || z[1] != p.kv_heads || z[2] != p.page_size ||
        z[3] != 64 || s[3] != 1)
      return ok = false, nullptr;
    *s0 = s[0];
    *s1 = s[1];
    *s2 = s[2];
    return t->data_ptr();
  }

  // a contiguous tensor [d0] or, with d1 >= 0, [d0][d1]
  void* dense(PyObject* o, at::ScalarType type, int64_t d0, int64_t d1 = -1) {
    const at::Tensor* t = tensor(o, type);
    if (!t) return nullptr;
    const auto z = t->sizes();
    if (static_cast<int64_t>(z.size()) != (d1 < 0 ? 1 : 2) || z[0] != d0 ||
        (d1 >= 0 && z[1] != d1) || !t->is_contiguous())
      return ok = false, nullptr;
    return t->data_ptr();
  }

  int32_t* ints(PyObject* o, int64_t d0, int64_t d1 = -1) {
    return static_cast<int32_t*>(dense(o, at::kInt, d0, d1));
  }

  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// The entry point's code as a Python int; other threads run meanwhile, as a full
// launch queue may hold the call up.
template <class F>
PyObject* launched(F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// Runs `call` (marshalling and launch), with any exception as "not here".
template <class F>
PyObject* guarded(F call) {
  try {
    return call();
  } catch (...) {
    return none();
  }
}

bool paged_shape(PyObject* s, attn_paged_shape* p, at::ScalarType* type) {
  *p = attn_paged_shape{};
  p->head_dim = 64;
  return get(s, BATCH, &p->batch) && get(s, TOKENS, &p->tokens) && get(s, HEADS, &p->heads) &&
         get(s, KV_HEADS, &p->kv_heads) && get(s, PAGE_SIZE, &p->page_size) &&
         get(s, NUM_PAGES, &p->num_pages) && get(s, TABLE_WIDTH, &p->table_width) &&
         get(s, MAX_NEW, &p->max_new) && get_dtype(s, type, &p->dtype) && get_scale(s, &p->scale);
}

// packed_fwd(shape, q, k, v, cu, o, lse)
PyObject* packed_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7 || !entry.packed_fwd) return none();
  return guarded([&]() -> PyObject* {
    attn_packed_shape p{};
    at::ScalarType type;
    p.head_dim = 64;
    PyObject* const causal = PyObject_GetAttr(a[0], names[CAUSAL]);
    const int truth = causal ? PyObject_IsTrue(causal) : -1;
    Py_XDECREF(causal);
    if (truth < 0 || !get(a[0], TOKENS, &p.tokens) || !get(a[0], BATCH, &p.batch) ||
        !get(a[0], HEADS, &p.heads) || !get(a[0], KV_HEADS, &p.kv_heads) ||
        !get_dtype(a[0], &type, &p.dtype) || !get_scale(a[0], &p.scale))
      return none();
    p.causal = truth;
    Call c;
    void* const q = c.rows(a[1], type, p.tokens, p.heads, &p.q_token, &p.q_head);
    void* const k = c.rows(a[2], type, p.tokens, p.kv_heads, &p.k_token, &p.k_head);
    void* const v = c.rows(a[3], type, p.tokens, p.kv_heads, &p.v_token, &p.v_head);
    int32_t* const cu = c.ints(a[4], p.batch + 1ll);
    void* const o = c.rows(a[5], type, p.tokens, p.heads, &p.o_token, &p.o_head);
    float* lse = nullptr;
    if (a[6] != Py_None) lse = static_cast<float*>(c.dense(a[6], at::kFloat, p.heads, p.tokens));
    if (!c.ok) return none();
    void* const stream = c.stream();
    return launched([&] { return entry.packed_fwd(&p, q, k, v, cu, o, lse, stream); });
  });
}

// paged_plan(shape, cached, fresh, ring, state, table, cu, lens, slots, next)
PyObject* paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10 || !entry.paged_plan) return none();
  return guarded([&]() -> PyObject* {
    attn_paged_shape p;
    at::ScalarType type;
    if (!paged_shape(a[0], &p, &type)) return none();
    Call c;
    int32_t* const cached = c.ints(a[1], p.batch);
    int32_t* const fresh = c.ints(a[2], p.batch);
    int32_t* const ring = c.ints(a[3], p.num_pages);
    int32_t* const state = c.ints(a[4], 4);
    int32_t* const table = c.ints(a[5], p.batch, p.table_width);
    int32_t* const cu = c.ints(a[6], p.batch + 1ll);
    int32_t* const lens = c.ints(a[7], p.batch);
    int32_t* const slots = c.ints(a[8], p.tokens);
    int32_t* const next = c.ints(a[9], 4);
    if (!c.ok) return none();
    void* const stream = c.stream();
    return launched([&] {
      return entry.paged_plan(&p, cached, fresh, ring, state, table, cu, lens, slots, next, stream);
    });
  });
}

// paged_store(shape, k, v, slots, k_cache, v_cache)
PyObject* paged_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !entry.paged_store) return none();
  return guarded([&]() -> PyObject* {
    attn_paged_shape p;
    at::ScalarType type;
    if (!paged_shape(a[0], &p, &type)) return none();
    Call c;
    void* const k = c.rows(a[1], type, p.tokens, p.kv_heads, &p.k_token, &p.k_head);
    void* const v = c.rows(a[2], type, p.tokens, p.kv_heads, &p.v_token, &p.v_head);
    int32_t* const slots = c.ints(a[3], p.tokens);
    void* const kc = c.pool(a[4], type, p, &p.kc_page, &p.kc_head, &p.kc_row);
    void* const vc = c.pool(a[5], type, p, &p.vc_page, &p.vc_head, &p.vc_row);
    if (!c.ok) return none();
    void* const stream = c.stream();
    return launched([&] { return entry.paged_store(&p, k, v, slots, kc, vc, stream); });
  });
}

// paged_fwd(shape, q, k_cache, v_cache, table, cu, lens, ws, o, lse)
PyObject* paged_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10 || !entry.paged_fwd) return none();
  return guarded([&]() -> PyObject* {
    attn_paged_shape p;
    at::ScalarType type;
    if (!paged_shape(a[0], &p, &type)) return none();
    Call c;
    void* const q = c.rows(a[1], type, p.tokens, p.heads, &p.q_token, &p.q_head);
    void* const kc = c.pool(a[2], type, p, &p.kc_page, &p.kc_head, &p.kc_row);
    void* const vc = c.pool(a[3], type, p, &p.vc_page, &p.vc_head, &p.vc_row);
    int32_t* const table = c.ints(a[4], p.batch, p.table_width);
    int32_t* const cu = c.ints(a[5], p.batch + 1ll);
    int32_t* const lens = c.ints(a[6], p.batch);
    const at::Tensor* const ws = c.tensor(a[7], at::kByte);
    if (ws && !ws->is_contiguous()) c.ok = false;
    void* const o = c.rows(a[8], type, p.tokens, p.heads, &p.o_token, &p.o_head);
    float* lse = nullptr;
    if (a[9] != Py_None) lse = static_cast<float*>(c.dense(a[9], at::kFloat, p.heads, p.tokens));
    if (!c.ok) return none();
    void* const stream = c.stream();
    void* const work = ws->data_ptr();
    const size_t bytes = static_cast<size_t>(ws->numel());
    return launched([&] {
      return entry.paged_fwd(&p, q, kc, vc, table, cu, lens, work, bytes, o, lse, stream);
    });
  });
}

// bind(packed_fwd, paged_plan, paged_store, paged_fwd): the entry points'
// addresses in the loaded libattn.so
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[4] = {};
  for (Py_ssize_t i = 0; i < n && i < 4; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  entry.packed_fwd = reinterpret_cast<decltype(entry.packed_fwd)>(p[0]);
  entry.paged_plan = reinterpret_cast<decltype(entry.paged_plan)>(p[1]);
  entry.paged_store = reinterpret_cast<decltype(entry.paged_store)>(p[2]);
  entry.paged_fwd = reinterpret_cast<decltype(entry.paged_fwd)>(p[3]);
  Py_RETURN_NONE;
}

#define METHOD(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {METHOD(bind),        METHOD(packed_fwd), METHOD(paged_plan),
                         METHOD(paged_store), METHOD(paged_fwd),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  for (int i = 0; i < NAMES; ++i)
    if (!(names[i] = PyUnicode_InternFromString(kNames[i]))) return nullptr;
  PyObject* const m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", CSS_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
