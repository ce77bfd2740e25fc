// The binding's short way into libtq2 for the calls around a decode step's
// projections: a step makes a few of them per layer, each on a kernel of a
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
decltype(&tq2_add_rms_norm) f_norm;
decltype(&tq2_add_rms_norm_i8) f_norm_i8;
decltype(&tq2_gemm_gate_up_silu) f_gated;
decltype(&tq2_gemm_i8q_gate_up_silu) f_gated_i8;
decltype(&tq2_gemm_gate_up_silu_workspace_bytes) f_gated_ws, f_gated_i8_ws;
decltype(&tq2_token_logprobs) f_logprobs;
decltype(&tq2_token_logprobs_workspace_bytes) f_logprobs_ws;

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

// Rows [T, D] with contiguous elements.
const at::Tensor* rows(Call& c, PyObject* o) {
  const at::Tensor* t = c.any(o);
  if (!t || t->dim() != 2 || (t->stride(1) != 1 && t->size(1) > 1) || dtype_of(*t) < 0) return c.fail();
  return t;
}
// A tensor that may be left out: null, or whole of this type and size.
const at::Tensor* maybe(Call& c, PyObject* o, at::ScalarType type, int64_t numel) {
  return c.none(o) ? nullptr : c.whole(o, type, numel);
}
// The tensors are the current device's, on whose streams calls run.
bool here(const Call& c) { return c.ok && c.device == c10::hip::current_device(); }

// What both norms take: x, residual, weight, eps, h_out
struct Norm {
  const at::Tensor *x, *r, *w, *h;
  double eps;
  bool from(Call& c, PyObject* const* a) {
    x = rows(c, a[0]);
    if (!c.ok || !number(a[3], &eps)) return false;
    const int64_t T = x->size(0), D = x->size(1);
    r = c.none(a[1]) ? nullptr : rows(c, a[1]);
    w = maybe(c, a[2], at::kFloat, D);
    h = c.none(a[4]) ? nullptr : rows(c, a[4]);
    if (!c.ok || !r != !h || !fits(D)) return false;
    return !r || (r->size(0) == T && r->size(1) == D && h->sizes() == r->sizes() && h->scalar_type() == r->scalar_type() &&
                  (T < 2 || h->stride(0) == r->stride(0)));
  }
  int64_t T() const { return x->size(0); }
  int64_t D() const { return x->size(1); }
};

// x, residual, weight, eps, h_out, out, stream
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  Norm m;
  tq2_stream_t s;
  if (n != 7 || !m.from(c, a)) return none();
  const at::Tensor* out = rows(c, a[5]);
  if (!c.ok || !out->is_contiguous() || out->sizes() != m.x->sizes() || !here(c) || !stream_of(a[6], &s)) return none();
  return status(f_norm, ptr(m.x), m.x->stride(0), dtype_of(*m.x), ptr(m.r), m.r ? m.r->stride(0) : 0,
                m.r ? dtype_of(*m.r) : 0, ptr(m.h), m.T(), m.D(), ptr<float>(m.w), (float)m.eps, ptr(out), dtype_of(*out), s);
}

// x, residual, weight, eps, h_out, s, x_q, x_scales, stream
PyObject* norm_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  Norm m;
  tq2_stream_t st;
  double s = 0;
  if (n != 9 || !m.from(c, a)) return none();
  const at::Tensor *q = c.whole(a[6], at::kChar, m.T() * m.D()), *sc = nullptr;
  if (c.none(a[5]))
    sc = c.whole(a[7], at::kFloat, m.T());
  else if (!number(a[5], &s) || !((float)s > 0) || !c.none(a[7]))
    return none();
  if (!here(c) || q->dim() != 2 || q->sizes() != m.x->sizes() || !stream_of(a[8], &st)) return none();
  return status(f_norm_i8, ptr(m.x), m.x->stride(0), dtype_of(*m.x), ptr(m.r), m.r ? m.r->stride(0) : 0,
                m.r ? dtype_of(*m.r) : 0, ptr(m.h), m.T(), m.D(), ptr<float>(m.w), (float)m.eps, (float)s, ptr<int8_t>(q),
                ptr<float>(sc), st);
}

// codes_g, scales_g, codes_u, scales_u, x, s (None: x is fp16), h, ws, stream
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  tq2_stream_t st;
  double s = 0;
  if (n != 9) return none();
  const at::Tensor* cg = c.whole(a[0], at::kByte);
  if (!c.ok || cg->dim() != 2 || cg->size(1) % 64) return none();
  const int64_t N = cg->size(0), K = cg->size(1) * 4;
  const at::Tensor *sg = c.whole(a[1], at::kHalf, N * (K / 256)), *cu = c.whole(a[2], at::kByte);
  const at::Tensor* su = c.whole(a[3], at::kHalf, N * (K / 256));
  const bool int8 = !c.none(a[5]);
  const at::Tensor *x = c.whole(a[4], int8 ? at::kChar : at::kHalf), *h = rows(c, a[6]), *sc = nullptr;
  if (!c.ok || cu->sizes() != cg->sizes() || x->dim() != 2 || x->size(1) != K) return none();
  const int64_t M = x->size(0);
  if (int8 && THPVariable_Check(a[5]))
    sc = c.whole(a[5], at::kFloat, M);
  else if (int8 && (!number(a[5], &s) || !((float)s > 0)))
    return none();
  if (!here(c) || !h->is_contiguous() || h->size(0) != M || h->size(1) != N) return none();
  const size_t need = (int8 ? f_gated_i8_ws : f_gated_ws)(N, K, M);
  const at::Tensor* ws = nullptr;
  if (!c.none(a[7])) {
    ws = c.any(a[7]);
    if (!ws || !ws->is_contiguous()) return none();
  }
  const size_t given = ws ? ws->nbytes() : 0;
  if (need == (size_t)-1 || given < need || !stream_of(a[8], &st)) return none();
  if (int8)
    return status(f_gated_i8, ptr<uint8_t>(cg), ptr<uint16_t>(sg), ptr<uint8_t>(cu), ptr<uint16_t>(su), N, K,
                  ptr<int8_t>(x), M, (float)s, ptr<float>(sc), ptr(h), dtype_of(*h), ptr(ws), given, st);
  return status(f_gated, ptr<uint8_t>(cg), ptr<uint16_t>(sg), ptr<uint8_t>(cu), ptr<uint16_t>(su), N, K, ptr<uint16_t>(x),
                M, ptr(h), dtype_of(*h), ptr(ws), given, st);
}

// logits, tokens, top, scale, logprobs, entropy, top_tokens, top_logprobs, ws, stream
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  tq2_stream_t st;
  int64_t top;
  double scale;
  if (n != 10 || !whole_number(a[2], &top) || !fits(top) || !number(a[3], &scale)) return none();
  const at::Tensor* x = rows(c, a[0]);
  if (!c.ok) return none();
  const int64_t T = x->size(0), V = x->size(1);
  const at::Tensor *tok = maybe(c, a[1], at::kLong, T), *lp = maybe(c, a[4], at::kFloat, T);
  const at::Tensor *H = maybe(c, a[5], at::kFloat, T), *tt = maybe(c, a[6], at::kLong, T * top);
  const at::Tensor* tl = maybe(c, a[7], at::kFloat, T * top);
  if (!here(c) || !tok != !lp || !tt != !top || !tl != !top) return none();
  if (top && (tt->dim() != 2 || tl->dim() != 2 || tt->size(0) != T || tl->size(0) != T)) return none();
  const size_t need = f_logprobs_ws(T, V, top);
  const at::Tensor* ws = nullptr;
  if (!c.none(a[8])) {
    ws = c.any(a[8]);
    if (!ws || !ws->is_contiguous()) return none();
  }
  const size_t given = ws ? ws->nbytes() : 0;
  if (need == (size_t)-1 || given < need || !here(c) || !stream_of(a[9], &st)) return none();
  return status(f_logprobs, ptr(x), x->stride(0), dtype_of(*x), T, V, (float)scale, ptr<int64_t>(tok), ptr<float>(lp),
                ptr<float>(H), top, ptr<int64_t>(tt), ptr<float>(tl), ptr(ws), given, st);
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
PyObject* bind_step(PyObject*, PyObject* args) {
  unsigned long long p[8];
  if (!PyArg_ParseTuple(args, "KKKKKKKK", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7])) return nullptr;
  f_norm = (decltype(f_norm))p[0];
  f_norm_i8 = (decltype(f_norm_i8))p[1];
  f_gated = (decltype(f_gated))p[2];
  f_gated_i8 = (decltype(f_gated_i8))p[3];
  f_gated_ws = (decltype(f_gated_ws))p[4];
  f_gated_i8_ws = (decltype(f_gated_i8_ws))p[5];
  f_logprobs = (decltype(f_logprobs))p[6];
  f_logprobs_ws = (decltype(f_logprobs_ws))p[7];
  Py_RETURN_NONE;
}

// A C++ exception must not cross into the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!f_rope || !f_norm) {
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
    {"bind_step", bind_step, METH_VARARGS, nullptr},
    {"qk_norm_rope", (PyCFunction)(void*)guarded<rope>, METH_FASTCALL, nullptr},
    {"kv4_store", (PyCFunction)(void*)guarded<store>, METH_FASTCALL, nullptr},
    {"kv4_load", (PyCFunction)(void*)guarded<load>, METH_FASTCALL, nullptr},
    {"kv4_attn", (PyCFunction)(void*)guarded<attn>, METH_FASTCALL, nullptr},
    {"add_rms_norm", (PyCFunction)(void*)guarded<norm>, METH_FASTCALL, nullptr},
    {"add_rms_norm_i8", (PyCFunction)(void*)guarded<norm_i8>, METH_FASTCALL, nullptr},
    {"gate_up_silu", (PyCFunction)(void*)guarded<gated>, METH_FASTCALL, nullptr},
    {"token_logprobs", (PyCFunction)(void*)guarded<logprobs>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tq2call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tq2call() { return PyModule_Create(&module); }
