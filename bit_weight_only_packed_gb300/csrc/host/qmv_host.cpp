// qmv_host.cpp -- the usual form of the verification-step and decode-step calls, marshalled in C++.
//
// These kernels take a few microseconds, so a decode loop that is not captured in a
// graph is bound by the host's steps between two calls.  Each function here takes
// the arguments of a call as its Python wrapper (qmv.py) got them.  In the usual case
// (contiguous tensors of the expected types and shapes on the current CUDA device,
// fresh outputs, the current stream) it allocates the outputs, calls the C ABI and
// returns them; it returns None for anything else, and the wrapper then checks the
// call in full, raises what is to be raised, or runs it.  A failing status is
// returned as a number.
//
// Only torch's own handles are used: a tensor's type, sizes, address and device, a
// fresh tensor, the current stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qmv.h"

namespace {

decltype(&qmv_w4_gemv) f_w4;
decltype(&qmv_block_norm) f_norm;
decltype(&qmv_softmax) f_softmax;
decltype(&qmv_verify_draft) f_verify;
decltype(&qmv_qk_norm_rope) f_rope;
decltype(&qmv_route) f_route;
decltype(&qmv_w4_experts) f_experts;
decltype(&qmv_w4_experts_workspace_bytes) f_experts_ws;
decltype(&qmv_w4_experts_form) f_experts_form;
decltype(&qmv_w4_experts_form_bytes) f_experts_form_ws;
decltype(&qmv_sample) f_sample;

// init(function addresses): the library is loaded by the binding
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long f[11];
  if (!PyArg_ParseTuple(args, "KKKKKKKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8], &f[9], &f[10]))
    return nullptr;
  f_w4 = reinterpret_cast<decltype(f_w4)>(f[0]);
  f_norm = reinterpret_cast<decltype(f_norm)>(f[1]);
  f_softmax = reinterpret_cast<decltype(f_softmax)>(f[2]);
  f_verify = reinterpret_cast<decltype(f_verify)>(f[3]);
  f_rope = reinterpret_cast<decltype(f_rope)>(f[4]);
  f_route = reinterpret_cast<decltype(f_route)>(f[5]);
  f_experts = reinterpret_cast<decltype(f_experts)>(f[6]);
  f_experts_ws = reinterpret_cast<decltype(f_experts_ws)>(f[7]);
  f_experts_form = reinterpret_cast<decltype(f_experts_form)>(f[8]);
  f_experts_form_ws = reinterpret_cast<decltype(f_experts_form_ws)>(f[9]);
  f_sample = reinterpret_cast<decltype(f_sample)>(f[10]);
  Py_RETURN_NONE;
}

constexpr int64_t MOST = INT32_MAX;

int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return QMV_F32;
    case at::kHalf: return QMV_F16;
    case at::kBFloat16: return QMV_BF16;
    default: return -1;
  }
}

// A contiguous CUDA tensor on device `dev` (any where it is -1, which it then sets).
const at::Tensor* tensor(PyObject* o, int& dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || !t.is_contiguous() || t.layout() != at::kStrided) return nullptr;
  const int at = t.get_device();
  if (dev >= 0 && at != dev) return nullptr;
  dev = at;
  return &t;
}

// The same of one type and shape; `o` may be None where `none` says so (out = null).
bool of(PyObject* o, int& dev, at::ScalarType type, at::IntArrayRef shape, bool none, void** out) {
  *out = nullptr;
  if (none && o == Py_None) return true;
  const at::Tensor* t = tensor(o, dev);
  if (!t || t->scalar_type() != type || t->sizes() != shape) return false;
  *out = t->data_ptr();
  return true;
}

bool stream_of(int dev, void** stream) {
  if (c10::cuda::current_device() != dev) return false;
  *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  return true;
}

at::Tensor fresh(const at::Tensor& like, at::ScalarType type, at::IntArrayRef shape) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

constexpr at::ScalarType TYPES[] = {at::kFloat, at::kHalf, at::kBFloat16};

PyObject* leave() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject* one(int rc, at::Tensor&& a) { return rc == QMV_OK ? THPVariable_Wrap(std::move(a)) : PyLong_FromLong(rc); }

PyObject* two(int rc, at::Tensor&& a, at::Tensor&& b) {
  if (rc != QMV_OK) return PyLong_FromLong(rc);
  PyObject *r = PyTuple_New(2), *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
  if (!r || !x || !y) {
    Py_XDECREF(r);
    Py_XDECREF(x);
    Py_XDECREF(y);
    return nullptr;
  }
  PyTuple_SET_ITEM(r, 0, x);
  PyTuple_SET_ITEM(r, 1, y);
  return r;
}

// w4_gemv(pack handle, device, N, K, x, y_dtype)
PyObject* w4_gemv(PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return leave();
  const auto* p = static_cast<const qmv_w4pack*>(PyLong_AsVoidPtr(a[0]));
  int dev = static_cast<int>(PyLong_AsLong(a[1]));
  const int64_t N = PyLong_AsLongLong(a[2]), K = PyLong_AsLongLong(a[3]);
  const long yd = PyLong_AsLong(a[5]);
  if (PyErr_Occurred() || !p || dev < 0 || yd < QMV_F32 || yd > QMV_BF16) return leave();
  const at::Tensor* x = tensor(a[4], dev);
  void* st;
  if (!x || x->dim() != 2 || x->size(1) != K || x->size(0) < 1 || x->size(0) > 4096) return leave();
  const int xd = type_of(*x), M = static_cast<int>(x->size(0));
  if ((xd != QMV_F16 && xd != QMV_BF16) || !stream_of(dev, &st)) return leave();
  at::Tensor y = fresh(*x, TYPES[yd], {M, N});
  return one(f_w4(p, M, x->data_ptr(), static_cast<int>(K), xd, y.data_ptr(), static_cast<int>(N),
                  static_cast<int>(yd), st),
             std::move(y));
}

// block_norm(y, residual, gamma_pre, gamma_post, gate, residual_scale, branch_scale, gamma_offset, eps)
PyObject* block_norm(PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return leave();
  float f[4];
  for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(PyFloat_AsDouble(a[5 + i]));
  if (PyErr_Occurred()) return leave();
  int dev = -1, ldg = 0;
  const at::Tensor *r = tensor(a[1], dev), *y = tensor(a[0], dev);
  if (!r || !y || r->dim() != 2 || y->sizes() != r->sizes()) return leave();
  const int td = type_of(*r), yd = type_of(*y);
  const int64_t M = r->size(0), D = r->size(1);
  if ((td != QMV_F16 && td != QMV_BF16) || yd < 0 || M < 1 || D < 1 || M > MOST || D > MOST) return leave();
  const at::ScalarType type = r->scalar_type();
  void *gpre, *gpost, *gate, *st;
  if (!of(a[2], dev, type, {D}, false, &gpre) || !of(a[3], dev, type, {D}, true, &gpost)) return leave();
  if (!of(a[4], dev, type, {D}, true, &gate)) {
    if (!of(a[4], dev, type, {M, D}, false, &gate)) return leave();
    ldg = static_cast<int>(D);
  }
  if (!stream_of(dev, &st)) return leave();
  at::Tensor h = fresh(*r, type, {M, D}), o = fresh(*r, type, {M, D});
  const int ld = static_cast<int>(D);
  const int rc = f_norm(static_cast<int>(M), ld, y->data_ptr(), ld, yd, r->data_ptr(), ld, gpost, gate, ldg, f[0], f[1],
                        gpre, f[2], f[3], h.data_ptr(), ld, o.data_ptr(), ld, td, st);
  return two(rc, std::move(h), std::move(o));
}

// softmax(logits, temperature)
PyObject* softmax(PyObject* const* a, Py_ssize_t n) {
  if (n != 2) return leave();
  int dev = -1;
  const at::Tensor* x = tensor(a[0], dev);
  if (!x || x->dim() != 2) return leave();
  const int xd = type_of(*x);
  const int64_t rows = x->size(0), V = x->size(1);
  if (xd < 0 || rows < 1 || V < 1 || rows > MOST || V > MOST) return leave();
  void *t = nullptr, *st;
  float t0 = 1.0f;
  if (THPVariable_Check(a[1])) {
    if (!of(a[1], dev, at::kFloat, {rows}, false, &t)) return leave();
  } else {
    t0 = static_cast<float>(PyFloat_AsDouble(a[1]));
    if (PyErr_Occurred()) return leave();
  }
  if (!stream_of(dev, &st)) return leave();
  at::Tensor o = fresh(*x, at::kFloat, {rows, V});
  const int ld = static_cast<int>(V);
  return one(f_softmax(static_cast<int>(rows), ld, x->data_ptr(), ld, xd, static_cast<const float*>(t), t0,
                       static_cast<float*>(o.data_ptr()), ld, st),
             std::move(o));
}

// verify_draft(target, draft_probs, draft, u_accept, u_sample, n_draft)
PyObject* verify_draft(PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return leave();
  int dev = -1;
  const at::Tensor* p = tensor(a[0], dev);
  if (!p || p->dim() != 3 || p->scalar_type() != at::kFloat) return leave();
  const int64_t B = p->size(0), S = p->size(1) - 1, V = p->size(2);
  if (B < 1 || S < 1 || V < 1 || B > MOST || S > MOST || V > MOST) return leave();
  void *q, *d, *ua, *us, *nd, *st;
  if (!of(a[1], dev, at::kFloat, {B, S, V}, true, &q) || !of(a[2], dev, at::kInt, {B, S}, false, &d) ||
      !of(a[3], dev, at::kFloat, {B, S}, false, &ua) || !of(a[4], dev, at::kFloat, {B}, false, &us) ||
      !of(a[5], dev, at::kInt, {B}, true, &nd) || !stream_of(dev, &st))
    return leave();
  at::Tensor t = fresh(*p, at::kInt, {B, S + 1}), c = fresh(*p, at::kInt, {B});
  const int rc = f_verify(static_cast<int>(B), static_cast<int>(S), static_cast<int>(V),
                          static_cast<const float*>(p->data_ptr()), static_cast<const float*>(q),
                          static_cast<const int*>(d), static_cast<const int*>(nd), static_cast<const float*>(ua),
                          static_cast<const float*>(us), static_cast<int*>(t.data_ptr()),
                          static_cast<int*>(c.data_ptr()), st);
  return two(rc, std::move(t), std::move(c));
}

// A number argument as int (within its range) or float; `ok` is left as it is or cleared.
int whole(PyObject* o, bool& ok) {
  const long v = PyLong_AsLong(o);
  ok = ok && v >= INT32_MIN && v <= INT32_MAX;
  return static_cast<int>(v);
}
float real(PyObject* o) { return static_cast<float>(PyFloat_AsDouble(o)); }

// qk_norm_rope(qkv, n_q, n_k, D, turns, rot, layout, amplitude, positions, gamma_q, gamma_k, gamma_offset, eps, y_dtype)
PyObject* qk_norm_rope(PyObject* const* a, Py_ssize_t n) {
  if (n != 14) return leave();
  bool ok = true;
  const int nq = whole(a[1], ok), nk = whole(a[2], ok), D = whole(a[3], ok), rot = whole(a[5], ok), layout = whole(a[6], ok);
  const float amp = real(a[7]), goff = real(a[11]), eps = real(a[12]);
  int yd = a[13] == Py_None ? -1 : whole(a[13], ok);
  if (PyErr_Occurred() || !ok || nq < 1 || nk < 1 || D < 1 || nq > 4096 || nk > 4096 || D > 1024 || rot < 0 || rot > D) return leave();
  int dev = -1;
  const at::Tensor* x = tensor(a[0], dev);
  if (!x || x->dim() != 2) return leave();
  const int xd = type_of(*x);
  const int64_t M = x->size(0), C = x->size(1), wq = (int64_t)nq * D, wk = (int64_t)nk * D;
  if (xd < 0 || M < 1 || M > MOST || C > MOST || C < wq + wk) return leave();
  if (yd == -1) {
    yd = xd;
    for (int i = 9; i < 11 && yd == QMV_F32; ++i)
      if (THPVariable_Check(a[i])) yd = type_of(THPVariable_Unpack(a[i]));
    if (yd == QMV_F32) yd = QMV_F16;
  }
  if (yd != QMV_F16 && yd != QMV_BF16) return leave();
  void *pos, *turns, *gq, *gk, *st;
  if (!of(a[8], dev, at::kInt, {M}, rot == 0, &pos) || !of(a[4], dev, at::kLong, {rot / 2}, rot == 0, &turns) ||
      (pos != nullptr) != (rot != 0) || (turns != nullptr) != (rot != 0) || !of(a[9], dev, TYPES[yd], {D}, true, &gq) ||
      !of(a[10], dev, TYPES[yd], {D}, true, &gk) || !stream_of(dev, &st))
    return leave();
  at::Tensor q = fresh(*x, TYPES[yd], {M, nq, D}), k = fresh(*x, TYPES[yd], {M, nk, D});
  const int rc = f_rope(static_cast<int>(M), nq, nk, D, x->data_ptr(), static_cast<int>(C), xd, static_cast<const int*>(pos),
                        static_cast<const int64_t*>(turns), rot, layout, amp, gq, gk, goff, eps, q.data_ptr(),
                        static_cast<int>(wq), k.data_ptr(), static_cast<int>(wk), yd, st);
  return two(rc, std::move(q), std::move(k));
}

// route(logits, T, score, bias, groups, group_k, group_top, renormalise, scale)
PyObject* route(PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return leave();
  bool ok = true;
  const int T = whole(a[1], ok), score = whole(a[2], ok), groups = whole(a[4], ok), gk = whole(a[5], ok), gt = whole(a[6], ok);
  const int renorm = PyObject_IsTrue(a[7]);
  const float scale = real(a[8]);
  if (PyErr_Occurred() || !ok || T < 1 || renorm < 0) return leave();
  int dev = -1;
  const at::Tensor* x = tensor(a[0], dev);
  if (!x || x->dim() != 2) return leave();
  const int xd = type_of(*x);
  const int64_t M = x->size(0), E = x->size(1);
  void *bias, *st;
  if (xd < 0 || M < 1 || M > MOST || E < 1 || E > 1024 || T > E || !of(a[3], dev, at::kFloat, {E}, true, &bias) ||
      !stream_of(dev, &st))
    return leave();
  at::Tensor ids = fresh(*x, at::kInt, {M, T}), w = fresh(*x, at::kFloat, {M, T});
  const int rc = f_route(static_cast<int>(M), static_cast<int>(E), T, x->data_ptr(), static_cast<int>(E), xd, score,
                         static_cast<const float*>(bias), groups, gk, gt, renorm, scale, static_cast<int*>(ids.data_ptr()),
                         static_cast<float*>(w.data_ptr()), st);
  return two(rc, std::move(ids), std::move(w));
}

// w4_experts(pack handle, device, K, rows_per_expert, ids, x, weights, act, y_dtype, workspace)
PyObject* w4_experts(PyObject* const* a, Py_ssize_t n) {
  if (n != 10) return leave();
  bool ok = true;
  const auto* p = static_cast<const qmv_w4pack*>(PyLong_AsVoidPtr(a[0]));
  int dev = whole(a[1], ok);
  const int K = whole(a[2], ok), R = whole(a[3], ok), act = whole(a[7], ok), yd = whole(a[8], ok);
  if (PyErr_Occurred() || !ok || !p || dev < 0 || R < 1 || yd < QMV_F32 || yd > QMV_BF16) return leave();
  const at::Tensor *ids = tensor(a[4], dev), *x = tensor(a[5], dev);
  if (!ids || !x || ids->dim() != 2 || ids->scalar_type() != at::kInt) return leave();
  const int64_t M = ids->size(0), T = ids->size(1), width = act == QMV_ACT_NONE ? K : 2 * (int64_t)K;
  const bool per_pair = x->dim() == 3;
  if (M < 1 || T < 1 || M > 4096 || T > 64 || width > MOST ||
      (per_pair ? x->sizes() != at::IntArrayRef({M, T, width}) : x->sizes() != at::IntArrayRef({M, width})))
    return leave();
  const int xd = type_of(*x);
  void *w, *st, *ws = nullptr;
  if ((xd != QMV_F16 && xd != QMV_BF16) || !of(a[6], dev, at::kFloat, {M, T}, true, &w) || !stream_of(dev, &st)) return leave();
  size_t have;
  at::Tensor made;
  const bool own = a[9] == Py_None;        // scratch for this call's form alone
  if (!own) {
    const at::Tensor* given = tensor(a[9], dev);
    if (!given) return leave();
    have = given->nbytes();
    ws = given->data_ptr();
    if (have < f_experts_ws(p, R, static_cast<int>(M), static_cast<int>(T))) return leave();
  } else if ((have = f_experts_form_ws(p, R, static_cast<int>(M), static_cast<int>(T), w != nullptr, x->data_ptr(),
                                       static_cast<int>(width), per_pair, xd, act))) {
    made = fresh(*x, at::kByte, {static_cast<int64_t>(have)});
    ws = made.data_ptr();
  }
  at::Tensor y = w ? fresh(*x, TYPES[yd], {M, R}) : fresh(*x, TYPES[yd], {M, T, R});
  return one((own ? f_experts_form : f_experts)(p, R, static_cast<int>(M), static_cast<int>(T),
                                                static_cast<const int*>(ids->data_ptr()), static_cast<const float*>(w),
                                                x->data_ptr(), static_cast<int>(width), per_pair, xd, act, y.data_ptr(), R, yd,
                                                ws, have, st),
             std::move(y));
}

// sample(logits, u, temperature, top_k, top_p, min_p)
PyObject* sample(PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return leave();
  int dev = -1;
  const at::Tensor* x = tensor(a[0], dev);
  if (!x || x->dim() != 2) return leave();
  const int xd = type_of(*x);
  const int64_t rows = x->size(0), V = x->size(1);
  void *u, *at[4] = {}, *st;
  if (xd < 0 || rows < 1 || V < 1 || rows > MOST || V > MOST || !of(a[1], dev, at::kFloat, {rows}, false, &u)) return leave();
  float num[4] = {};
  int k = 0;
  bool ok = true;
  for (int i = 0; i < 4; ++i) {
    if (THPVariable_Check(a[2 + i])) {
      if (!of(a[2 + i], dev, i == 1 ? at::kInt : at::kFloat, {rows}, false, &at[i])) return leave();
    } else if (i == 1) {
      k = whole(a[3], ok);
    } else {
      num[i] = real(a[2 + i]);
    }
  }
  if (PyErr_Occurred() || !ok || !stream_of(dev, &st)) return leave();
  at::Tensor t = fresh(*x, at::kInt, {rows});
  return one(f_sample(static_cast<int>(rows), static_cast<int>(V), x->data_ptr(), static_cast<int>(V), xd,
                      static_cast<const float*>(at[0]), num[0], static_cast<const int*>(at[1]), k,
                      static_cast<const float*>(at[2]), num[2], static_cast<const float*>(at[3]), num[3],
                      static_cast<const float*>(u), static_cast<int*>(t.data_ptr()), st),
             std::move(t));
}

// No C++ exception (out of memory, say) leaves a function: the wrapper meets it again.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (...) {
    return leave();
  }
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr}, method<w4_gemv>("w4_gemv"),   method<block_norm>("block_norm"),
    method<softmax>("softmax"),            method<verify_draft>("verify_draft"),
    method<qk_norm_rope>("qk_norm_rope"), method<route>("route"), method<w4_experts>("w4_experts"), method<sample>("sample"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "qmv_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qmv_host(void) { return PyModule_Create(&module); }
