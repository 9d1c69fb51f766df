/*
 * qmv_host.c -- the usual form of the verification-step calls, marshalled in C.
 *
 * These kernels take a few microseconds, so a decode loop that is not captured
 * in a graph is bound by the host's steps between two calls.  Each function
 * here takes the tensors of a call as its Python wrapper (qmv.py) got them.  When
 * they are the usual case (contiguous tensors of the expected types and shapes
 * on the current CUDA device, fresh outputs, the current stream) it allocates the
 * outputs, calls the C ABI and returns them; it returns None for anything else,
 * and the wrapper then checks the call in full, raises what is to be raised, or
 * runs it.  A failing status is returned as a number.  Host times on a GB300's
 * CPU, call after call: qmv_block_norm 12.2 us by the wrapper alone.
 *
 * Plain CPython C API: tensors are read through their public attributes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "qmv.h"

typedef int (*w4_fn)(const qmv_w4pack *, int, const void *, int, int, void *, int, int, void *);
typedef int (*norm_fn)(int, int, const void *, int, int, const void *, int, const void *, const void *, int, float,
                       float, const void *, float, float, void *, int, void *, int, int, void *);
typedef int (*softmax_fn)(int, int, const void *, int, int, const float *, float, float *, int, void *);
typedef int (*verify_fn)(int, int, int, const float *, const float *, const int *, const int *, const float *,
                         const float *, int *, int *, void *);

static w4_fn f_w4;
static norm_fn f_norm;
static softmax_fn f_softmax;
static verify_fn f_verify;

static PyObject *tensor_type, *empty_fn, *device_fn, *stream_fn; /* torch.Tensor, torch.empty, current device, raw stream */
static PyObject *dt[4];                                          /* float32, float16, bfloat16, int32 */
static PyObject *s_dtype, *s_shape, *s_device, *s_contig, *s_ptr, *s_dev, *kw_empty;
enum { I32 = 3 };

/* init(torch.Tensor, torch.empty, device fn, stream fn, (dtypes), (function addresses)) */
static PyObject *init(PyObject *self, PyObject *args) {
    PyObject *dts, *fns;
    if (!PyArg_ParseTuple(args, "OOOOO!O!", &tensor_type, &empty_fn, &device_fn, &stream_fn, &PyTuple_Type, &dts,
                          &PyTuple_Type, &fns))
        return NULL;
    if (PyTuple_GET_SIZE(dts) != 4 || PyTuple_GET_SIZE(fns) != 4) {
        PyErr_SetString(PyExc_ValueError, "four dtypes and four functions");
        return NULL;
    }
    void *f[4];
    for (int i = 0; i < 4; ++i) {
        dt[i] = PyTuple_GET_ITEM(dts, i);
        Py_INCREF(dt[i]);
        f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(fns, i));
        if (!f[i]) return NULL;
    }
    f_w4 = (w4_fn)f[0];
    f_norm = (norm_fn)f[1];
    f_softmax = (softmax_fn)f[2];
    f_verify = (verify_fn)f[3];
    Py_INCREF(tensor_type);
    Py_INCREF(empty_fn);
    Py_INCREF(device_fn);
    Py_INCREF(stream_fn);
    Py_RETURN_NONE;
}

/* A contiguous tensor on device `dev` (any CUDA device where *dev < 0, which then
 * becomes its index): its type's number, its shape and its address. */
typedef struct {
    int type, nd;
    int64_t n[3];
    char *ptr;
} view;

static PyObject *call0(PyObject *t, PyObject *name) {
    PyObject *a[1] = {t};
    return PyObject_VectorcallMethod(name, a, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}

static long long call_int(PyObject *t, PyObject *name) {
    PyObject *r = call0(t, name);
    if (!r) return -1;
    const long long v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return v;
}

static int look(PyObject *t, view *v, int *dev) {
    if (!PyObject_TypeCheck(t, (PyTypeObject *)tensor_type)) return 0;
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return 0;
    for (v->type = 0; v->type < 4 && dt[v->type] != d; ++v->type) {}
    Py_DECREF(d);
    if (v->type == 4) return 0;
    PyObject *s = PyObject_GetAttr(t, s_shape);
    if (!s) return 0;
    v->nd = PyTuple_Check(s) ? (int)PyTuple_GET_SIZE(s) : 4;
    if (v->nd > 3) {
        Py_DECREF(s);
        return 0;
    }
    for (int i = 0; i < v->nd; ++i) v->n[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
    Py_DECREF(s);
    PyObject *c = call0(t, s_contig);
    Py_XDECREF(c);
    if (c != Py_True) return 0;
    const long long at = call_int(t, s_dev);
    if (at < 0 || (*dev >= 0 && at != *dev)) return 0;
    *dev = (int)at;
    c = call0(t, s_ptr);
    if (!c) return 0;
    v->ptr = (char *)PyLong_AsVoidPtr(c);
    Py_DECREF(c);
    return !PyErr_Occurred();
}

static int is(const view *v, int type, int nd, int64_t a, int64_t b, int64_t c) {
    return v->type == type && v->nd == nd && (nd < 1 || v->n[0] == a) && (nd < 2 || v->n[1] == b) &&
           (nd < 3 || v->n[2] == c);
}

/* Whether `dev` is the current device, and its current stream. */
static int stream_of(int dev, void **stream) {
    PyObject *r = PyObject_CallNoArgs(device_fn);
    if (!r) return 0;
    const long cur = PyLong_AsLong(r);
    Py_DECREF(r);
    if (cur != dev) return 0;
    PyObject *i = PyLong_FromLong(dev);
    if (!i) return 0;
    r = PyObject_CallOneArg(stream_fn, i);
    Py_DECREF(i);
    if (!r) return 0;
    *stream = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

static PyObject *fresh(PyObject *like, int type, int64_t rows, int64_t cols, char **ptr) {
    PyObject *shape = cols < 0 ? Py_BuildValue("(L)", (long long)rows) : Py_BuildValue("(LL)", (long long)rows, (long long)cols);
    PyObject *device = PyObject_GetAttr(like, s_device), *t = NULL;
    if (shape && device) {
        PyObject *a[3] = {shape, dt[type], device};
        t = PyObject_Vectorcall(empty_fn, a, 1, kw_empty);
    }
    Py_XDECREF(shape);
    Py_XDECREF(device);
    if (t) {
        PyObject *p = call0(t, s_ptr);
        if (!p) {
            Py_DECREF(t);
            return NULL;
        }
        *ptr = (char *)PyLong_AsVoidPtr(p);
        Py_DECREF(p);
    }
    return t;
}

/* Not the usual case, or an error on the way: the wrapper sees to it. */
static PyObject *leave(void) {
    PyErr_Clear();
    Py_RETURN_NONE;
}

static PyObject *result(int rc, PyObject *a, PyObject *b) {
    if (rc != QMV_OK) {
        Py_DECREF(a);
        Py_XDECREF(b);
        return PyLong_FromLong(rc);
    }
    if (!b) return a;
    PyObject *r = PyTuple_New(2);
    if (!r) {
        Py_DECREF(a);
        Py_DECREF(b);
        return NULL;
    }
    PyTuple_SET_ITEM(r, 0, a);
    PyTuple_SET_ITEM(r, 1, b);
    return r;
}

/* w4_gemv(pack handle, device, N, K, x, y_dtype) */
static PyObject *w4_gemv(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view x;
    void *st;
    char *yp;
    if (n != 6) return leave();
    int dev = (int)PyLong_AsLong(a[1]);
    const int64_t N = PyLong_AsLongLong(a[2]), K = PyLong_AsLongLong(a[3]);
    const long yd = PyLong_AsLong(a[5]);
    if (PyErr_Occurred() || dev < 0 || yd < QMV_F32 || yd > QMV_BF16) return leave();
    if (!look(a[4], &x, &dev) || (x.type != QMV_F16 && x.type != QMV_BF16) || x.nd != 2 || x.n[1] != K || x.n[0] < 1 ||
        x.n[0] > 4096 || !stream_of(dev, &st))
        return leave();
    const qmv_w4pack *p = (const qmv_w4pack *)PyLong_AsVoidPtr(a[0]);
    PyObject *y = fresh(a[4], (int)yd, x.n[0], N, &yp);
    if (!p || !y) {
        Py_XDECREF(y);
        return leave();
    }
    return result(f_w4(p, (int)x.n[0], x.ptr, (int)K, x.type, yp, (int)N, (int)yd, st), y, NULL);
}

/* block_norm(y, residual, gamma_pre, gamma_post, gate, residual_scale, branch_scale, gamma_offset, eps) */
static PyObject *block_norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view y, r, gp, gq = {0}, gt = {0};
    void *st;
    char *hp, *op;
    int dev = -1, ldg = 0;
    if (n != 9) return leave();
    float f[4];
    for (int i = 0; i < 4; ++i) f[i] = (float)PyFloat_AsDouble(a[5 + i]);
    if (PyErr_Occurred()) return leave();
    if (!look(a[1], &r, &dev) || (r.type != QMV_F16 && r.type != QMV_BF16) || r.nd != 2) return leave();
    const int64_t M = r.n[0], D = r.n[1];
    if (M < 1 || D < 1 || M > INT32_MAX || D > INT32_MAX) return leave();
    if (!look(a[0], &y, &dev) || y.type > QMV_BF16 || !is(&y, y.type, 2, M, D, 0)) return leave();
    if (!look(a[2], &gp, &dev) || !is(&gp, r.type, 1, D, 0, 0)) return leave();
    if (a[3] != Py_None && (!look(a[3], &gq, &dev) || !is(&gq, r.type, 1, D, 0, 0))) return leave();
    if (a[4] != Py_None) {
        if (!look(a[4], &gt, &dev)) return leave();
        if (is(&gt, r.type, 2, M, D, 0)) ldg = (int)D;
        else if (!is(&gt, r.type, 1, D, 0, 0)) return leave();
    }
    if (!stream_of(dev, &st)) return leave();
    PyObject *h = fresh(a[1], r.type, M, D, &hp), *o = h ? fresh(a[1], r.type, M, D, &op) : NULL;
    if (!o) {
        Py_XDECREF(h);
        return leave();
    }
    return result(f_norm((int)M, (int)D, y.ptr, (int)D, y.type, r.ptr, (int)D, gq.ptr, gt.ptr, ldg, f[0], f[1], gp.ptr,
                         f[2], f[3], hp, (int)D, op, (int)D, r.type, st),
                  h, o);
}

/* softmax(logits, temperature) */
static PyObject *softmax(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view x, t = {0};
    void *st;
    char *op;
    int dev = -1;
    float t0 = 1.0f;
    if (n != 2 || !look(a[0], &x, &dev) || x.type > QMV_BF16 || x.nd != 2) return leave();
    if (PyObject_TypeCheck(a[1], (PyTypeObject *)tensor_type)) {
        if (!look(a[1], &t, &dev) || !is(&t, QMV_F32, 1, x.n[0], 0, 0)) return leave();
    } else {
        t0 = (float)PyFloat_AsDouble(a[1]);
        if (PyErr_Occurred()) return leave();
    }
    if (x.n[0] < 1 || x.n[1] < 1 || x.n[0] > INT32_MAX || x.n[1] > INT32_MAX || !stream_of(dev, &st)) return leave();
    PyObject *o = fresh(a[0], QMV_F32, x.n[0], x.n[1], &op);
    if (!o) return leave();
    return result(f_softmax((int)x.n[0], (int)x.n[1], x.ptr, (int)x.n[1], x.type, (float *)t.ptr, t0, (float *)op,
                            (int)x.n[1], st),
                  o, NULL);
}

/* verify_draft(target, draft_probs, draft, u_accept, u_sample, n_draft) */
static PyObject *verify_draft(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view p, q = {0}, d, ua, us, nd = {0};
    void *st;
    char *tp, *np;
    int dev = -1;
    if (n != 6 || !look(a[0], &p, &dev) || p.type != QMV_F32 || p.nd != 3) return leave();
    const int64_t B = p.n[0], S = p.n[1] - 1, V = p.n[2];
    if (B < 1 || S < 1 || V < 1 || B > INT32_MAX || S > INT32_MAX || V > INT32_MAX) return leave();
    if (a[1] != Py_None && (!look(a[1], &q, &dev) || !is(&q, QMV_F32, 3, B, S, V))) return leave();
    if (!look(a[2], &d, &dev) || !is(&d, I32, 2, B, S, 0)) return leave();
    if (!look(a[3], &ua, &dev) || !is(&ua, QMV_F32, 2, B, S, 0)) return leave();
    if (!look(a[4], &us, &dev) || !is(&us, QMV_F32, 1, B, 0, 0)) return leave();
    if (a[5] != Py_None && (!look(a[5], &nd, &dev) || !is(&nd, I32, 1, B, 0, 0))) return leave();
    if (!stream_of(dev, &st)) return leave();
    PyObject *t = fresh(a[0], I32, B, S + 1, &tp), *c = t ? fresh(a[0], I32, B, -1, &np) : NULL;
    if (!c) {
        Py_XDECREF(t);
        return leave();
    }
    return result(f_verify((int)B, (int)S, (int)V, (float *)p.ptr, (float *)q.ptr, (int *)d.ptr, (int *)nd.ptr,
                           (float *)ua.ptr, (float *)us.ptr, (int *)tp, (int *)np, st),
                  t, c);
}

static PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, NULL},
    {"w4_gemv", (PyCFunction)(void (*)(void))w4_gemv, METH_FASTCALL, NULL},
    {"block_norm", (PyCFunction)(void (*)(void))block_norm, METH_FASTCALL, NULL},
    {"softmax", (PyCFunction)(void (*)(void))softmax, METH_FASTCALL, NULL},
    {"verify_draft", (PyCFunction)(void (*)(void))verify_draft, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "qmv_host", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_qmv_host(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_device = PyUnicode_InternFromString("device");
    s_contig = PyUnicode_InternFromString("is_contiguous");
    s_ptr = PyUnicode_InternFromString("data_ptr");
    s_dev = PyUnicode_InternFromString("get_device");
    kw_empty = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_dtype || !s_shape || !s_device || !s_contig || !s_ptr || !s_dev || !kw_empty) return NULL;
    return PyModule_Create(&module);
}
