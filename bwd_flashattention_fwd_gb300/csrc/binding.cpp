// The Python binding's calls around attention (gbattn.py): tensors checked and
// taken apart in C++.  A serving loop makes these calls every few microseconds,
// and in Python checking and converting ten tensors costs more than the kernels
// take.  Each function takes what its wrapper takes, in order, and a stream's
// handle (None: the current stream), and calls the C ABI; it returns the status,
// or -1 where a tensor is not what the call takes: the wrapper then goes through
// its own checks, which name what is wrong.  The C ABI's functions come as
// addresses (init), so one module serves both builds of the library.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/gbattn.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Entry {
  const char* name;
  void* at;
};
Entry entries[] = {{"attn_qk_norm_rope", nullptr}, {"attn_qk_norm_rope_bwd", nullptr}, {"attn_paged_write", nullptr},
                   {"attn_paged_read", nullptr},   {"attn_fwd_paged", nullptr},        {"attn_draft_verify", nullptr}};

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// One call's tensors: every test that fails leaves `ok` false.
struct Call {
  int dev = -1;
  bool ok = true;

  void first(const Tensor* t, int dims) {  // the tensor that the others go by
    ok = t && t->is_cuda() && t->dim() == dims && t->get_device() == c10::cuda::current_device();
    if (ok) dev = t->get_device();
  }
  bool like(const Tensor* t, ScalarType type, at::IntArrayRef shape) {  // type, device and shape
    ok = ok && t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->sizes() == shape;
    return ok;
  }
  void* dense(const Tensor* t, ScalarType type, at::IntArrayRef shape) {
    return like(t, type, shape) && (ok = t->is_contiguous()) ? t->data_ptr() : nullptr;
  }
  void* dense(PyObject* o, ScalarType type, at::IntArrayRef shape) { return ok ? dense(tensor(o), type, shape) : nullptr; }
  void* maybe(PyObject* o, ScalarType type, at::IntArrayRef shape) { return o == Py_None ? nullptr : dense(o, type, shape); }
  void* rows(PyObject* o, ScalarType type, at::IntArrayRef shape, int64_t* strides) {  // [B, H, L, D], D contiguous
    const Tensor* t = ok ? tensor(o) : nullptr;
    if (!like(t, type, shape) || !(ok = t->stride(3) == 1)) return nullptr;
    for (int i = 0; i < 3; ++i) strides[i] = t->stride(i);
    return t->data_ptr();
  }
  cudaStream_t stream(PyObject* o) {
    if (!ok) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    void* h = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) PyErr_Clear(), ok = false;
    return static_cast<cudaStream_t>(h);
  }
  double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return x;
  }
};

bool half(ScalarType t) { return t == ScalarType::BFloat16 || t == ScalarType::Half; }
attn_dtype_t code(ScalarType t) { return t == ScalarType::BFloat16 ? ATTN_DTYPE_BF16 : ATTN_DTYPE_FP16; }

template <class F, class... A>
PyObject* launch(int entry, cudaStream_t stream, F, A... args) {
  attn_status_t s;
  Py_BEGIN_ALLOW_THREADS
  s = reinterpret_cast<F>(entries[entry].at)(args..., stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

#define GBATTN_CALL(name, n_args)                                                          \
  PyObject* name##_checked(PyObject* const* a);                                            \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {                            \
    try {                                                                                  \
      PyObject* r = n == n_args ? name##_checked(a) : nullptr;                             \
      return r ? r : PyLong_FromLong(-1);                                                  \
    } catch (...) { /* (a tensor without storage, say) */                                  \
      return PyLong_FromLong(-1);                                                          \
    }                                                                                      \
  }                                                                                        \
  PyObject* name##_checked(PyObject* const* a)

// q, k, q_out, k_out, pos, freq, q_weight, k_weight, axis, eps, interleaved, stream
GBATTN_CALL(qk_norm_rope, 12) {
  const Tensor *q = tensor(a[0]), *k = tensor(a[1]), *pos = tensor(a[4]), *freq = tensor(a[5]);
  Call c;
  c.first(q, 4);
  if (!c.ok || !half(q->scalar_type()) || !k || k->dim() != 4 || !pos || !freq || freq->dim() != 1) return nullptr;
  const ScalarType t = q->scalar_type();
  const int64_t B = q->size(0), Hq = q->size(1), L = q->size(2), D = q->size(3), Hkv = k->size(1), half_rot = freq->size(0);
  const int64_t axes = pos->dim() == 3 ? pos->size(0) : 1;
  int64_t qs[3], ks[3];
  const void* qp = c.rows(a[0], t, {B, Hq, L, D}, qs);
  const void* kp = c.rows(a[1], t, {B, Hkv, L, D}, ks);
  void* qo = c.dense(a[2], t, {B, Hq, L, D});
  void* ko = c.dense(a[3], t, {B, Hkv, L, D});
  const void* pp = pos->dim() == 3 ? c.dense(pos, ScalarType::Int, {axes, B, L}) : c.dense(pos, ScalarType::Int, {B, L});
  const void* fp = c.dense(freq, ScalarType::Float, {half_rot});
  const void* qw = c.maybe(a[6], t, {D});
  const void* kw = c.maybe(a[7], t, {D});
  const void* ax = c.maybe(a[8], ScalarType::Byte, {half_rot});
  const float eps = static_cast<float>(c.number(a[9]));
  const int inter = PyObject_IsTrue(a[10]);
  const cudaStream_t stream = c.stream(a[11]);
  if (!c.ok || inter < 0) return PyErr_Clear(), nullptr;
  return launch(0, stream, &attn_qk_norm_rope, qp, kp, qw, kw, static_cast<const int32_t*>(pp), static_cast<const float*>(fp),
                static_cast<const uint8_t*>(ax), qo, ko, static_cast<const int64_t*>(qs), static_cast<const int64_t*>(ks), static_cast<int>(B),
                static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(L), static_cast<int>(D), static_cast<int>(2 * half_rot),
                static_cast<int>(axes), eps, inter, code(t));
}

// q, k, dq_out, dk_out, pos, freq, dq, dk, q_weight, k_weight, dq_weight, dk_weight, workspace, axis, eps, interleaved, stream
GBATTN_CALL(qk_norm_rope_bwd, 17) {
  const Tensor *q = tensor(a[0]), *k = tensor(a[1]), *pos = tensor(a[4]), *freq = tensor(a[5]), *ws = tensor(a[12]);
  Call c;
  c.first(q, 4);
  if (!c.ok || !half(q->scalar_type()) || !k || k->dim() != 4 || !pos || !freq || freq->dim() != 1 || !ws) return nullptr;
  const ScalarType t = q->scalar_type();
  const int64_t B = q->size(0), Hq = q->size(1), L = q->size(2), D = q->size(3), Hkv = k->size(1), half_rot = freq->size(0);
  const int64_t axes = pos->dim() == 3 ? pos->size(0) : 1;
  int64_t qs[3], ks[3], dqs[3], dks[3];
  const void* qp = c.rows(a[0], t, {B, Hq, L, D}, qs);
  const void* kp = c.rows(a[1], t, {B, Hkv, L, D}, ks);
  const void* gq = c.dense(a[2], t, {B, Hq, L, D});
  const void* gk = c.dense(a[3], t, {B, Hkv, L, D});
  const void* pp = pos->dim() == 3 ? c.dense(pos, ScalarType::Int, {axes, B, L}) : c.dense(pos, ScalarType::Int, {B, L});
  const void* fp = c.dense(freq, ScalarType::Float, {half_rot});
  void* dq = c.rows(a[6], t, {B, Hq, L, D}, dqs);
  void* dk = c.rows(a[7], t, {B, Hkv, L, D}, dks);
  const void* qw = c.maybe(a[8], t, {D});
  const void* kw = c.maybe(a[9], t, {D});
  void* dqw = c.maybe(a[10], ScalarType::Float, {D});
  void* dkw = c.maybe(a[11], ScalarType::Float, {D});
  void* wp = c.dense(ws, ScalarType::Byte, ws->sizes());
  const void* ax = c.maybe(a[13], ScalarType::Byte, {half_rot});
  const float eps = static_cast<float>(c.number(a[14]));
  const int inter = PyObject_IsTrue(a[15]);
  const cudaStream_t stream = c.stream(a[16]);
  if (!c.ok || inter < 0) return PyErr_Clear(), nullptr;
  return launch(1, stream, &attn_qk_norm_rope_bwd, qp, kp, qw, kw, static_cast<const int32_t*>(pp), static_cast<const float*>(fp),
                static_cast<const uint8_t*>(ax), gq, gk, dq, dk, static_cast<float*>(dqw), static_cast<float*>(dkw), wp,
                static_cast<size_t>(ws->numel()), static_cast<const int64_t*>(qs), static_cast<const int64_t*>(ks),
                static_cast<const int64_t*>(dqs), static_cast<const int64_t*>(dks), static_cast<int>(B), static_cast<int>(Hq),
                static_cast<int>(Hkv), static_cast<int>(L), static_cast<int>(D), static_cast<int>(2 * half_rot), static_cast<int>(axes), eps,
                inter, code(t));
}

// A paged cache's tensors: pages, exponents (both or neither), table.
struct Pool {
  void *k, *v, *ke, *ve;
  const int32_t* table;
  int64_t n, Hkv, page, D, B, per_seq;

  bool take(Call& c, ScalarType t, PyObject* k_pages, PyObject* v_pages, PyObject* tab, PyObject* k_exp, PyObject* v_exp) {
    const Tensor *kt = tensor(k_pages), *tt = tensor(tab);
    if (!kt || kt->dim() != 4 || !tt || tt->dim() != 2 || (k_exp == Py_None) != (v_exp == Py_None)) return c.ok = false;
    n = kt->size(0), Hkv = kt->size(1), page = kt->size(2), D = kt->size(3), B = tt->size(0), per_seq = tt->size(1);
    const ScalarType held = k_exp == Py_None ? t : ScalarType::Float8_e4m3fn;
    k = c.dense(kt, held, {n, Hkv, page, D});
    v = c.dense(v_pages, held, {n, Hkv, page, D});
    ke = c.maybe(k_exp, ScalarType::Char, {n, Hkv, page});
    ve = c.maybe(v_exp, ScalarType::Char, {n, Hkv, page});
    table = static_cast<const int32_t*>(c.dense(tt, ScalarType::Int, {B, per_seq}));
    return c.ok;
  }
};

// k_new, v_new, k_pages, v_pages, table, cache_len, cache_len_out, new_len, k_exp, v_exp, stream
GBATTN_CALL(paged_write, 11) {
  const Tensor* kn = tensor(a[0]);
  Call c;
  c.first(kn, 4);
  if (!c.ok || !half(kn->scalar_type())) return nullptr;
  const ScalarType t = kn->scalar_type();
  Pool p;
  if (!p.take(c, t, a[2], a[3], a[4], a[8], a[9])) return nullptr;
  const int64_t T = kn->size(2);
  const void* kp = c.dense(kn, t, {p.B, p.Hkv, T, p.D});
  const void* vp = c.dense(a[1], t, {p.B, p.Hkv, T, p.D});
  const void* len = c.dense(a[5], ScalarType::Int, {p.B});
  void* out = c.dense(a[6], ScalarType::Int, {p.B});
  const void* fresh = c.maybe(a[7], ScalarType::Int, {p.B});
  const cudaStream_t stream = c.stream(a[10]);
  if (!c.ok) return nullptr;
  return launch(2, stream, &attn_paged_write, kp, vp, p.k, p.v, static_cast<int8_t*>(p.ke), static_cast<int8_t*>(p.ve), p.table,
                static_cast<const int32_t*>(len), static_cast<const int32_t*>(fresh), static_cast<int32_t*>(out), static_cast<int>(p.B),
                static_cast<int>(p.Hkv), static_cast<int>(T), static_cast<int>(p.n), static_cast<int>(p.page), static_cast<int>(p.per_seq),
                static_cast<int>(p.D), code(t));
}

// k_pages, v_pages, table, cache_len, k, v, k_exp, v_exp, stream
GBATTN_CALL(paged_read, 9) {
  const Tensor* k = tensor(a[4]);
  Call c;
  c.first(k, 4);
  if (!c.ok || !half(k->scalar_type())) return nullptr;
  const ScalarType t = k->scalar_type();
  Pool p;
  if (!p.take(c, t, a[0], a[1], a[2], a[6], a[7])) return nullptr;
  const int64_t Lk = k->size(2);
  const void* len = c.dense(a[3], ScalarType::Int, {p.B});
  const Tensor* v = tensor(a[5]);
  if (!c.like(k, t, {p.B, p.Hkv, Lk, p.D}) || !c.like(v, t, k->sizes())) return nullptr;
  int64_t pitch = 0;  // contiguous, or the first Lk rows of a [B, Hkv, pitch, D] buffer (as kv_row_pitch in gbattn.py)
  if (!k->is_contiguous() || !v->is_contiguous()) {
    const auto st = k->strides();
    if (st[3] != 1 || st[2] != p.D || st[1] % p.D != 0 || st[1] < Lk * p.D || st[0] != p.Hkv * st[1] || v->strides() != st) return nullptr;
    pitch = st[1] / p.D;
  }
  void *ko = k->data_ptr(), *vo = v->data_ptr();
  const cudaStream_t stream = c.stream(a[8]);
  if (!c.ok) return nullptr;
  return launch(3, stream, &attn_paged_read, static_cast<const void*>(p.k), static_cast<const void*>(p.v), static_cast<const int8_t*>(p.ke),
                static_cast<const int8_t*>(p.ve), p.table, static_cast<const int32_t*>(len), ko, vo, pitch, static_cast<int>(p.B),
                static_cast<int>(p.Hkv), static_cast<int>(Lk), static_cast<int>(p.n), static_cast<int>(p.page), static_cast<int>(p.per_seq),
                static_cast<int>(p.D), code(t));
}

// q, k_pages, v_pages, table, cache_len, o, lse, workspace, scale, k_exp, v_exp, stream
GBATTN_CALL(fwd_paged, 12) {
  const Tensor *q = tensor(a[0]), *ws = tensor(a[7]);
  Call c;
  c.first(q, 4);
  if (!c.ok || !half(q->scalar_type()) || !ws) return nullptr;
  const ScalarType t = q->scalar_type();
  Pool p;
  if (!p.take(c, t, a[1], a[2], a[3], a[9], a[10])) return nullptr;
  const int64_t Hq = q->size(1), T = q->size(2);
  const void* qp = c.dense(q, t, {p.B, Hq, T, p.D});
  const void* len = c.dense(a[4], ScalarType::Int, {p.B});
  void* o = c.dense(a[5], t, {p.B, Hq, T, p.D});
  void* lse = c.dense(a[6], ScalarType::Float, {p.B, Hq, T});
  void* wp = c.dense(ws, ScalarType::Byte, ws->sizes());
  const float scale = static_cast<float>(c.number(a[8]));
  const cudaStream_t stream = c.stream(a[11]);
  if (!c.ok) return nullptr;
  return launch(4, stream, &attn_fwd_paged, qp, static_cast<const void*>(p.k), static_cast<const void*>(p.v), static_cast<const int8_t*>(p.ke),
                static_cast<const int8_t*>(p.ve), p.table, static_cast<const int32_t*>(len), o, static_cast<float*>(lse), wp,
                static_cast<size_t>(ws->numel()), static_cast<int>(p.B), static_cast<int>(Hq), static_cast<int>(p.Hkv), static_cast<int>(T),
                static_cast<int>(p.n), static_cast<int>(p.page), static_cast<int>(p.per_seq), static_cast<int>(p.D), scale, code(t));
}

// target, draft, tokens, u, r, accept_len, token, draft_len, stream
GBATTN_CALL(draft_verify, 9) {
  const Tensor* target = tensor(a[0]);
  Call c;
  c.first(target, 3);
  if (!c.ok) return nullptr;
  const int64_t B = target->size(0), T = target->size(1) - 1, V = target->size(2);
  const void* tp = c.dense(target, ScalarType::Float, {B, T + 1, V});
  const void* dp = c.maybe(a[1], ScalarType::Float, {B, T, V});
  const void* tok = c.dense(a[2], ScalarType::Int, {B, T});
  const void* u = c.dense(a[3], ScalarType::Float, {B, T});
  const void* r = c.dense(a[4], ScalarType::Float, {B});
  void* acc = c.dense(a[5], ScalarType::Int, {B});
  void* out = c.dense(a[6], ScalarType::Int, {B});
  const void* len = c.maybe(a[7], ScalarType::Int, {B});
  const cudaStream_t stream = c.stream(a[8]);
  if (!c.ok) return nullptr;
  return launch(5, stream, &attn_draft_verify, static_cast<const float*>(tp), static_cast<const float*>(dp), static_cast<const int32_t*>(tok),
                static_cast<const float*>(u), static_cast<const float*>(r), static_cast<const int32_t*>(len), static_cast<int32_t*>(acc),
                static_cast<int32_t*>(out), static_cast<int>(B), static_cast<int>(T), static_cast<int>(V));
}

// init({name: address of the C ABI's function})
PyObject* init(PyObject*, PyObject* addresses) {
  for (Entry& e : entries) {
    PyObject* x = PyDict_Check(addresses) ? PyDict_GetItemString(addresses, e.name) : nullptr;
    void* at = x ? PyLong_AsVoidPtr(x) : nullptr;
    if (!at) {
      if (!PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "no address of %s", e.name);
      return nullptr;
    }
    e.at = at;
  }
  Py_RETURN_NONE;
}

#define GBATTN_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"init", init, METH_O, nullptr},   GBATTN_METHOD(qk_norm_rope), GBATTN_METHOD(qk_norm_rope_bwd),
                         GBATTN_METHOD(paged_write),        GBATTN_METHOD(paged_read),   GBATTN_METHOD(fwd_paged),
                         GBATTN_METHOD(draft_verify),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (what the wrapper compares with the Python and torch that it runs under)
extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", GBATTN_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
