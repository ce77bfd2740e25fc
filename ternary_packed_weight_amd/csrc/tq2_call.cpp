// The binding's short way into libtq2 for the calls of a decode step's
// attention half: a step makes a few of them per layer, each on a kernel of a
// few microseconds, and checking and marshalling ten tensors in Python takes
// longer than that.  Each function checks everything that the binding checks
// (types, layouts, devices) and calls the C ABI.  It returns the call's
// status, or None where the arguments are not the plain case (an output to
// allocate, a wrong type): the binding's own checks then decide.
#include <Python.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tq2.h"

namespace {

decltype(&tq2_qk_norm_rope) f_rope;
decltype(&tq2_kv4_store) f_store;
decltype(&tq2_kv4_load) f_load;
decltype(&tq2_kv4_attn) f_attn;
decltype(&tq2_kv4_attn_workspace_bytes) f_attn_ws;

// The tensors of one call: all on one GPU.
struct Call {
  int device = -1;
  bool ok = true;
  bool none(PyObject* o) const { return o == Py_None; }
  const at::Tensor* any(PyObject* o) {
    if (!THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (device < 0) device = t.get_device();
    return t.get_device() == device ? &t : fail();
  }
  const at::Tensor* whole(PyObject* o, at::ScalarType type, int64_t numel = -1) {
    const at::Tensor* t = any(o);
    if (!t || t->scalar_type() != type || !t->is_contiguous() || (numel >= 0 && t->numel() != numel)) return fail();
    return t;
  }
  // [T, H, D] with contiguous channels
  const at::Tensor* heads(PyObject* o) {
    const at::Tensor* t = any(o);
    if (!t || t->dim() != 3 || (t->stride(2) != 1 && t->size(2) > 1)) return fail();
    return t;
  }
  const at::Tensor* out(PyObject* o, at::ScalarType type, int64_t T, int64_t H, int64_t D) {
    const at::Tensor* t = heads(o);
    if (!t || t->scalar_type() != type || t->size(0) != T || t->size(1) != H || t->size(2) != D || !t->is_contiguous())
      return fail();
    return t;
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
};

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kHalf: return TQ2_F16;
    case at::kBFloat16: return TQ2_BF16;
    case at::kFloat: return TQ2_F32;
    default: return -1;
  }
}
template <class T = void>
T* ptr(const at::Tensor* t) {
  return t && t->numel() ? (T*)t->data_ptr() : nullptr;
}
bool fits(int64_t v) { return v >= 0 && v <= INT32_MAX; }
PyObject* none() { Py_RETURN_NONE; }
// The call's status.  Other threads of the interpreter go on meanwhile: a launch waits where the stream's queue is full.
template <class... P, class... A>
PyObject* status(int32_t (*f)(P...), A... a) {
  int32_t s;
  Py_BEGIN_ALLOW_THREADS
  s = f((P)a...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}
bool whole_number(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return !over;
}
bool number(PyObject* o, double* v) {
  if (!PyFloat_Check(o)) return false;
  *v = PyFloat_AS_DOUBLE(o);
  return true;
}
// A torch stream's handle, or the current device's current stream.
bool stream_of(PyObject* o, tq2_stream_t* s) {
  if (o != Py_None) {
    int64_t v;
    if (!whole_number(o, &v)) return false;
    *s = (tq2_stream_t)v;
    return true;
  }
  *s = (tq2_stream_t)c10::hip::getCurrentHIPStream().stream();
  return true;
}

// cache [pages, Hk, P*(D+8)]
bool cache_shape(const at::Tensor& t, int64_t D, int64_t* P) {
  if (t.dim() != 3 || D < 1 || t.size(2) % (D + 8) || !fits(t.size(1)) || !fits(t.size(2))) return false;
  *P = t.size(2) / (D + 8);
  return true;
}

// q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  double eps;
  tq2_stream_t s;
  if (n != 11 || !number(a[6], &eps)) return none();
  const at::Tensor *q = c.heads(a[0]), *k = c.heads(a[1]);
  if (!c.ok || k->scalar_type() != q->scalar_type() || k->size(0) != q->size(0) || k->size(2) != q->size(2))
    return none();
  const int64_t T = q->size(0), Hq = q->size(1), Hk = k->size(1), D = q->size(2);
  const at::Tensor *pos = c.whole(a[2], at::kInt, T), *inv = c.whole(a[3], at::kFloat);
  const at::Tensor* qw = c.none(a[4]) ? nullptr : c.whole(a[4], at::kFloat, D);
  const at::Tensor* kw = c.none(a[5]) ? nullptr : c.whole(a[5], at::kFloat, D);
  const at::Tensor *qo = c.heads(a[8]), *ko = c.heads(a[9]);
  if (!c.ok || !c.out(a[8], qo->scalar_type(), T, Hq, D) || !c.out(a[9], qo->scalar_type(), T, Hk, D)) return none();
  const int in = dtype_of(*q), out = dtype_of(*qo), il = PyObject_IsTrue(a[7]);
  if (in < 0 || out < 0 || il < 0 || !fits(Hq) || !fits(Hk) || !fits(D) || !fits(2 * inv->numel()) ||
      !stream_of(a[10], &s)) {
    PyErr_Clear();
    return none();
  }
  return status(f_rope, ptr(q), q->stride(0), q->stride(1), Hq, ptr(k), k->stride(0), k->stride(1), Hk, in, T, D,
                ptr<float>(qw), ptr<float>(kw), (float)eps, ptr<int32_t>(pos), ptr<float>(inv), 2 * inv->numel(), il,
                ptr(qo), ptr(ko), out, s);
}

// cache, k, v, slots, stream
PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  tq2_stream_t s;
  if (n != 5) return none();
  const at::Tensor *cache = c.whole(a[0], at::kByte), *k = c.heads(a[1]), *v = c.heads(a[2]);
  if (!c.ok || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type()) return none();
  const int64_t T = k->size(0), Hk = k->size(1), D = k->size(2);
  const at::Tensor* slots = c.whole(a[3], at::kLong, T);
  const int dt = dtype_of(*k);
  int64_t P;
  if (!c.ok || dt < 0 || !cache_shape(*cache, D, &P) || cache->size(1) != Hk || !stream_of(a[4], &s)) return none();
  return status(f_store, ptr<uint8_t>(cache), cache->size(0), P, Hk, D, ptr(k), k->stride(0), k->stride(1), ptr(v),
                v->stride(0), v->stride(1), dt, ptr<int64_t>(slots), T, s);
}

// cache, slots, D, k_out, v_out, stream
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  int64_t D, P;
  tq2_stream_t s;
  if (n != 6 || !whole_number(a[2], &D)) return none();
  const at::Tensor *cache = c.whole(a[0], at::kByte), *slots = c.whole(a[1], at::kLong), *k = c.heads(a[3]);
  if (!c.ok || !cache_shape(*cache, D, &P)) return none();
  const int64_t T = slots->numel(), Hk = cache->size(1);
  const at::Tensor* v = c.out(a[4], k->scalar_type(), T, Hk, D);
  const int dt = dtype_of(*k);
  if (!c.out(a[3], k->scalar_type(), T, Hk, D) || !c.ok || dt < 0 || !stream_of(a[5], &s)) return none();
  return status(f_load, ptr<uint8_t>(cache), cache->size(0), P, Hk, D, ptr<int64_t>(slots), T, ptr(k), ptr(v), dt, s);
}

// q, cache, table, ctx_len, q_start, max_q, scale, window, out, lse, ws, stream
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  int64_t max_q = 0, window, P;
  double scale;
  tq2_stream_t s;
  if (n != 12 || !whole_number(a[7], &window) || !fits(window)) return none();
  const at::Tensor *q = c.heads(a[0]), *cache = c.whole(a[1], at::kByte), *table = c.any(a[2]);
  if (!c.ok) return none();
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
  const int dt = dtype_of(*q);
  if ((dt != TQ2_F16 && dt != TQ2_BF16) || !cache_shape(*cache, D, &P)) return none();
  if (table->dim() != 2 || table->scalar_type() != at::kInt || (table->stride(1) != 1 && table->size(1) > 1)) return none();
  const int64_t B = table->size(0), width = table->size(1), Hk = cache->size(1);
  const at::Tensor* ctx = c.whole(a[3], at::kInt, B);
  const at::Tensor* start = c.none(a[4]) ? nullptr : c.whole(a[4], at::kInt, B + 1);
  const at::Tensor* out = c.out(a[8], q->scalar_type(), T, Hq, D);
  const at::Tensor* lse = c.none(a[9]) ? nullptr : c.whole(a[9], at::kFloat, T * Hq);
  if (!c.ok || B < 1) return none();
  if (c.none(a[5])) {
    if (start || T % B) return none();
    max_q = T / B > 1 ? T / B : 1;
  } else if (!whole_number(a[5], &max_q) || (!start && max_q * B != T)) {
    return none();
  }
  if (c.none(a[6]))
    scale = 1.0 / std::sqrt((double)D);
  else if (!number(a[6], &scale))
    return none();
  if (!fits(max_q) || !fits(B) || !fits(width) || !fits(Hq) || !fits(Hk) || !fits(D) || !fits(P)) return none();
  const size_t need = f_attn_ws(T, Hq, Hk, D, P, width, B, max_q);
  const at::Tensor* ws = nullptr;
  if (need != (size_t)-1 && !c.none(a[10])) {
    ws = c.any(a[10]);
    if (!ws || !ws->is_contiguous()) return none();
  }
  const size_t given = ws ? ws->nbytes() : 0;
  if (need == (size_t)-1 || given < need || !stream_of(a[11], &s)) return none();
  return status(f_attn, ptr(q), q->stride(0), q->stride(1), T, Hq, dt, ptr<uint8_t>(cache), cache->size(0), P, Hk, D,
                ptr<int32_t>(table), table->stride(0), width, ptr<int32_t>(ctx), ptr<int32_t>(start), B, max_q,
                (float)scale, window, ptr(out), ptr<float>(lse), ptr(ws), given, s);
}

// The library's entry points, by address: it is the binding that loads it.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[5];
  if (!PyArg_ParseTuple(args, "KKKKK", &p[0], &p[1], &p[2], &p[3], &p[4])) return nullptr;
  f_rope = (decltype(f_rope))p[0];
  f_store = (decltype(f_store))p[1];
  f_load = (decltype(f_load))p[2];
  f_attn = (decltype(f_attn))p[3];
  f_attn_ws = (decltype(f_attn_ws))p[4];
  Py_RETURN_NONE;
}

// A C++ exception must not cross into the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!f_rope) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return nullptr;
  }
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"qk_norm_rope", (PyCFunction)(void*)guarded<rope>, METH_FASTCALL, nullptr},
    {"kv4_store", (PyCFunction)(void*)guarded<store>, METH_FASTCALL, nullptr},
    {"kv4_load", (PyCFunction)(void*)guarded<load>, METH_FASTCALL, nullptr},
    {"kv4_attn", (PyCFunction)(void*)guarded<attn>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tq2call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tq2call() { return PyModule_Create(&module); }
