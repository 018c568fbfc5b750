/*
 * The calling side of the per-head-decay delta rule, the q/k norm and what stands around
 * them in a block for Python (module _kda_py): turns tensors into kda_tensor_t descriptors and calls the C entry
 * point, so that a one-token call's host share is a few microseconds.  Tensors are
 * read through their own methods (get_device, data_ptr, dim, shape, stride, dtype);
 * nothing of torch's headers or of the library is linked: bind() hands over the entry
 * points' addresses and the dtypes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/kda.h"

enum {
    GDR_FWD, GDR_BWD, GDR_DECODE, QK_NORM, QK_NORM_BWD, CONV, CONV_BWD, CONV_DECODE, GATED_NORM, GATED_NORM_BWD,
    ADD_NORM, ADD_NORM_BWD, SSM_FWD, SSM_BWD, SSM_DECODE, ENTRIES
};
#define MOST_TENSORS 20

typedef const kda_tensor_t* T;
static void* entry_point[ENTRIES];
static const char* const entry_name[ENTRIES] = {"kda_gdr_fwd", "kda_gdr_bwd", "kda_gdr_decode", "kda_qk_norm",
                                                "kda_qk_norm_bwd", "kda_conv", "kda_conv_bwd", "kda_conv_decode",
                                                "kda_gated_norm", "kda_gated_norm_bwd", "kda_add_norm", "kda_add_norm_bwd",
                                                "kda_ssm_fwd", "kda_ssm_bwd", "kda_ssm_decode"};
static const int entry_tensors[ENTRIES] = {9, 15, 9, 9, 13, 7, 11, 7, 4, 7, 5, 7, 11, 19, 11};
static const int entry_scalars[ENTRIES] = {1, 1, 1, 3, 3, 1, 1, 1, 3, 3, 2, 2, 1, 1, 1};
static PyObject* dtypes[4];   /* by kda_dtype_t */
static PyObject *s_get_device, *s_data_ptr, *s_dim, *s_shape, *s_stride, *s_dtype, *s_nbytes;

/* The integer that t.name() returns; -1 with an error set if it does not. */
static int method_int(PyObject* t, PyObject* name, long long* v) {
    PyObject* r = PyObject_CallMethodNoArgs(t, name);
    if (!r) return -1;
    *v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

static int copy_sizes(PyObject* seq, int64_t* to, int n) {
    if (!seq) return -1;
    int bad = !PyTuple_Check(seq) || PyTuple_GET_SIZE(seq) != n;
    if (bad) PyErr_SetString(PyExc_TypeError, "a tensor's shape and strides must be tuples of its rank");
    for (int i = 0; !bad && i < n; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
        bad = to[i] == -1 && PyErr_Occurred();
    }
    Py_DECREF(seq);
    return bad ? -1 : 0;
}

/* t's descriptor.  Every tensor has to lie on the GPU `dev`. */
static int describe(PyObject* t, long long dev, const char* entry, kda_tensor_t* d) {
    long long on, n, ptr;
    if (method_int(t, s_get_device, &on)) return -1;
    if (on != dev) {
        if (on < 0) PyErr_Format(PyExc_ValueError, "%s needs every tensor on the GPU", entry);
        else PyErr_Format(PyExc_ValueError, "%s needs every tensor on one GPU (got %lld and %lld)", entry, dev, on);
        return -1;
    }
    if (method_int(t, s_dim, &n) || method_int(t, s_data_ptr, &ptr)) return -1;
    if (n > 4) {
        PyErr_SetString(PyExc_ValueError, "kda tensors have at most 4 dimensions");
        return -1;
    }
    d->data = (void*)(intptr_t)ptr;
    d->ndim = (int32_t)n;
    if (copy_sizes(PyObject_GetAttr(t, s_shape), d->shape, (int)n)) return -1;
    if (copy_sizes(PyObject_CallMethodNoArgs(t, s_stride), d->stride, (int)n)) return -1;
    PyObject* dt = PyObject_GetAttr(t, s_dtype);
    if (!dt) return -1;
    int code = 99;   /* a dtype the library has no name for: it refuses it */
    for (int i = 0; i < 4; ++i)
        if (dt == dtypes[i]) code = i;
    d->dtype = (kda_dtype_t)code;
    Py_DECREF(dt);
    return 0;
}

/* call(entry, device, stream, workspace, scalars, tensors) -> status */
static PyObject* call(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    if (na != 6 || !PyTuple_Check(a[4]) || !PyTuple_Check(a[5])) {
        PyErr_SetString(PyExc_TypeError, "call(entry, device, stream, workspace, scalars, tensors)");
        return NULL;
    }
    const long e = PyLong_AsLong(a[0]);
    const long long dev = PyLong_AsLongLong(a[1]);
    void* stream = PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) return NULL;
    if (e < 0 || e >= ENTRIES || !entry_point[e]) {
        PyErr_SetString(PyExc_RuntimeError, "no such entry point");
        return NULL;
    }
    const Py_ssize_t nt = PyTuple_GET_SIZE(a[5]), ns = PyTuple_GET_SIZE(a[4]);
    if (nt != entry_tensors[e] || ns != entry_scalars[e]) {
        PyErr_Format(PyExc_TypeError, "%s takes %d tensors and %d scalars", entry_name[e], entry_tensors[e],
                     entry_scalars[e]);
        return NULL;
    }
    if (dev < 0) {
        PyErr_Format(PyExc_ValueError, "%s needs every tensor on the GPU", entry_name[e]);
        return NULL;
    }
    kda_tensor_t d[MOST_TENSORS];
    T t[MOST_TENSORS];
    for (Py_ssize_t i = 0; i < nt; ++i) {
        PyObject* o = PyTuple_GET_ITEM(a[5], i);
        t[i] = o == Py_None ? NULL : &d[i];
        if (o != Py_None && describe(o, dev, entry_name[e], &d[i])) return NULL;
    }
    double s[3];
    for (Py_ssize_t i = 0; i < ns; ++i) {
        s[i] = PyFloat_AsDouble(PyTuple_GET_ITEM(a[4], i));
        if (s[i] == -1.0 && PyErr_Occurred()) return NULL;
    }
    void* ws = NULL;
    long long ws_bytes = 0;
    if (a[3] != Py_None) {
        long long p, on;
        if (method_int(a[3], s_get_device, &on) || method_int(a[3], s_data_ptr, &p)) return NULL;
        if (on != dev) {
            PyErr_Format(PyExc_ValueError, "%s needs its workspace on the tensors' GPU", entry_name[e]);
            return NULL;
        }
        PyObject* b = PyObject_GetAttr(a[3], s_nbytes);
        if (!b) return NULL;
        ws_bytes = PyLong_AsLongLong(b);
        Py_DECREF(b);
        if (PyErr_Occurred()) return NULL;
        ws = (void*)(intptr_t)p;
    }
    kda_status_t st = KDA_OK;
    Py_BEGIN_ALLOW_THREADS
    switch (e) {
        case GDR_FWD:
            st = ((kda_status_t(*)(T, T, T, T, T, float, T, T, T, T, void*, int64_t, void*))entry_point[e])(
                t[0], t[1], t[2], t[3], t[4], (float)s[0], t[5], t[6], t[7], t[8], ws, ws_bytes, stream);
            break;
        case GDR_BWD:
            st = ((kda_status_t(*)(T, T, T, T, T, float, T, T, T, T, T, T, T, T, T, T, void*, int64_t,
                                   void*))entry_point[e])(t[0], t[1], t[2], t[3], t[4], (float)s[0], t[5], t[6], t[7],
                                                          t[8], t[9], t[10], t[11], t[12], t[13], t[14], ws, ws_bytes,
                                                          stream);
            break;
        case GDR_DECODE:
            st = ((kda_status_t(*)(T, T, T, T, T, float, T, T, T, T, void*))entry_point[e])(
                t[0], t[1], t[2], t[3], t[4], (float)s[0], t[5], t[6], t[7], t[8], stream);
            break;
        case QK_NORM:
            st = ((kda_status_t(*)(T, T, T, T, int32_t, float, T, T, T, int32_t, T, T, void*))entry_point[e])(
                t[0], t[1], t[2], t[3], (int32_t)s[0], (float)s[1], t[4], t[5], t[6], (int32_t)s[2], t[7], t[8],
                stream);
            break;
        case QK_NORM_BWD:
            st = ((kda_status_t(*)(T, T, T, T, T, T, int32_t, float, T, T, T, int32_t, T, T, T, T, void*, int64_t,
                                   void*))entry_point[e])(t[0], t[1], t[2], t[3], t[4], t[5], (int32_t)s[0],
                                                          (float)s[1], t[6], t[7], t[8], (int32_t)s[2], t[9], t[10],
                                                          t[11], t[12], ws, ws_bytes, stream);
            break;
        case CONV:
            st = ((kda_status_t(*)(T, T, T, int32_t, T, T, T, T, void*))entry_point[e])(
                t[0], t[1], t[2], (int32_t)s[0], t[3], t[4], t[5], t[6], stream);
            break;
        case CONV_BWD:
            st = ((kda_status_t(*)(T, T, T, int32_t, T, T, T, T, T, T, T, T, void*, int64_t, void*))entry_point[e])(
                t[0], t[1], t[2], (int32_t)s[0], t[3], t[4], t[5], t[6], t[7], t[8], t[9], t[10], ws, ws_bytes, stream);
            break;
        case CONV_DECODE:
            st = ((kda_status_t(*)(T, T, T, int32_t, T, T, T, T, void*))entry_point[e])(
                t[0], t[1], t[2], (int32_t)s[0], t[3], t[4], t[5], t[6], stream);
            break;
        case GATED_NORM:
            st = ((kda_status_t(*)(T, T, T, int32_t, int32_t, float, T, void*))entry_point[e])(
                t[0], t[1], t[2], (int32_t)s[0], (int32_t)s[1], (float)s[2], t[3], stream);
            break;
        case GATED_NORM_BWD:
            st = ((kda_status_t(*)(T, T, T, int32_t, int32_t, float, T, T, T, T, void*, int64_t, void*))entry_point[e])(
                t[0], t[1], t[2], (int32_t)s[0], (int32_t)s[1], (float)s[2], t[3], t[4], t[5], t[6], ws, ws_bytes, stream);
            break;
        case ADD_NORM:
            st = ((kda_status_t(*)(T, T, T, float, float, T, T, void*))entry_point[e])(t[0], t[1], t[2], (float)s[0],
                                                                                       (float)s[1], t[3], t[4], stream);
            break;
        case ADD_NORM_BWD:
            st = ((kda_status_t(*)(T, T, float, float, T, T, T, T, T, void*, int64_t, void*))entry_point[e])(
                t[0], t[1], (float)s[0], (float)s[1], t[2], t[3], t[4], t[5], t[6], ws, ws_bytes, stream);
            break;
        case SSM_FWD:
            st = ((kda_status_t(*)(T, T, T, T, T, T, T, int32_t, T, T, T, T, void*, int64_t, void*))entry_point[e])(
                t[0], t[1], t[2], t[3], t[4], t[5], t[6], (int32_t)s[0], t[7], t[8], t[9], t[10], ws, ws_bytes, stream);
            break;
        case SSM_BWD:
            st = ((kda_status_t(*)(T, T, T, T, T, T, T, int32_t, T, T, T, T, T, T, T, T, T, T, T, T, void*, int64_t,
                                   void*))entry_point[e])(t[0], t[1], t[2], t[3], t[4], t[5], t[6], (int32_t)s[0], t[7],
                                                          t[8], t[9], t[10], t[11], t[12], t[13], t[14], t[15], t[16],
                                                          t[17], t[18], ws, ws_bytes, stream);
            break;
        case SSM_DECODE:
            st = ((kda_status_t(*)(T, T, T, T, T, T, T, int32_t, T, T, T, T, void*))entry_point[e])(
                t[0], t[1], t[2], t[3], t[4], t[5], t[6], (int32_t)s[0], t[7], t[8], t[9], t[10], stream);
            break;
    }
    Py_END_ALLOW_THREADS
    return PyLong_FromLong((long)st);
}

/* bind(addresses, dtypes): the entry points in the order above, the dtypes by code. */
static PyObject* bind(PyObject* self, PyObject* args) {
    (void)self;
    PyObject *fns, *dts;
    if (!PyArg_ParseTuple(args, "O!O!", &PyTuple_Type, &fns, &PyTuple_Type, &dts)) return NULL;
    if (PyTuple_GET_SIZE(fns) != ENTRIES || PyTuple_GET_SIZE(dts) != 4) {
        PyErr_SetString(PyExc_TypeError, "bind() takes one address for each entry point and four dtypes");
        return NULL;
    }
    void* p[ENTRIES];
    for (int i = 0; i < ENTRIES; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(fns, i));
        if (PyErr_Occurred()) return NULL;
    }
    for (int i = 0; i < ENTRIES; ++i) entry_point[i] = p[i];
    for (int i = 0; i < 4; ++i) {
        Py_INCREF(PyTuple_GET_ITEM(dts, i));
        Py_XSETREF(dtypes[i], PyTuple_GET_ITEM(dts, i));
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "Calls an entry point."},
                                {"bind", bind, METH_VARARGS, "Sets the entry points and the dtypes."},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_py", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__kda_py(void) {
    s_get_device = PyUnicode_InternFromString("get_device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_dim = PyUnicode_InternFromString("dim");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    if (!s_get_device || !s_data_ptr || !s_dim || !s_shape || !s_stride || !s_dtype || !s_nbytes) return NULL;
    return PyModule_Create(&module);
}
