/* kd_py.c -- argument marshalling of the op-level calls that a decode loop makes per
 * token and layer, as a CPython module.  No arithmetic: each function converts its
 * arguments and calls the C entry point of the same name, and returns its status.
 * Calls in a row, one row's windowed attention (kernel 4.1 us): 4.2 us a call, 7.6
 * through ctypes; the smallest reorder (kernel 3.6 us): 3.8, 8.6 through ctypes.
 *
 * The Python helpers of the package (handed over by setup) convert what is not the
 * usual case: pointers of numpy arrays, lists of slots, streams. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "kd.h"

static PyObject *s_is_contiguous, *s_data_ptr, *s_nbytes;
static PyObject *h_ptr, *h_i32, *h_stream; /* _ptr, _i32, _stream */

/* Address of a contiguous tensor, an int, or None (0); anything else through _ptr. */
static int get_ptr(PyObject* o, void** out) {
    PyObject* v = NULL;
    *out = NULL;
    if (o == Py_None) return 0;
    if (PyLong_CheckExact(o)) {
        *out = PyLong_AsVoidPtr(o);
        return *out == NULL && PyErr_Occurred() ? -1 : 0;
    }
    v = PyObject_CallMethodNoArgs(o, s_is_contiguous);
    if (v) {
        const int yes = PyObject_IsTrue(v);
        Py_DECREF(v);
        if (yes < 0) return -1;
        if (!yes) {
            PyErr_SetString(PyExc_ValueError, "tensors passed to libkd must be contiguous");
            return -1;
        }
        v = PyObject_CallMethodNoArgs(o, s_data_ptr);
    } else if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
        PyErr_Clear();
        v = PyObject_CallOneArg(h_ptr, o);
    }
    if (!v) return -1;
    if (v != Py_None) *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

static int get_i32(PyObject* o, int32_t* out) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v != (int32_t)v) {
        PyErr_Format(PyExc_OverflowError, "%ld does not fit 32 bits", v);
        return -1;
    }
    *out = (int32_t)v;
    return 0;
}

static int get_nbytes(PyObject* o, size_t* out) {
    PyObject* v = PyObject_GetAttr(o, s_nbytes);
    if (!v) return -1;
    *out = PyLong_AsSize_t(v);
    Py_DECREF(v);
    return *out == (size_t)-1 && PyErr_Occurred() ? -1 : 0;
}

static int get_stream(PyObject* o, void** out) {
    PyObject* v;
    if (PyLong_CheckExact(o)) return get_ptr(o, out);
    v = PyObject_CallOneArg(h_stream, o);
    if (!v) return -1;
    *out = NULL;
    if (v != Py_None) *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* A host array of int32: a contiguous int32 buffer as it lies, anything else through _i32. */
typedef struct {
    Py_buffer b;
    int held;
} Ints;
static int view_i32(PyObject* o, Ints* a) {
    if (PyObject_GetBuffer(o, &a->b, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) < 0) return -1;
    if (a->b.itemsize == 4 && a->b.format && a->b.format[0] == 'i' && !a->b.format[1]) {
        a->held = 1;
        return 0;
    }
    PyBuffer_Release(&a->b);
    return -1;
}
static int get_ints(PyObject* o, Ints* a, Py_ssize_t want, int32_t* n) {
    a->held = 0;
    if (view_i32(o, a) < 0) {
        PyObject* v;
        PyErr_Clear();
        v = PyObject_CallOneArg(h_i32, o);
        if (!v) return -1;
        if (view_i32(v, a) < 0) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "expected an array of int32");
            Py_DECREF(v);
            return -1;
        }
        Py_DECREF(v); /* the view holds it */
    }
    if (want >= 0 && a->b.len / 4 != want) {
        PyErr_Format(PyExc_ValueError, "expected %zd entries, got %zd", want, a->b.len / 4);
        return -1;
    }
    if (n) {
        if (a->b.len / 4 > INT32_MAX) {
            PyErr_SetString(PyExc_OverflowError, "too many entries");
            return -1;
        }
        *n = (int32_t)(a->b.len / 4);
    }
    return 0;
}
static void drop(Ints* a) {
    if (a->held) PyBuffer_Release(&a->b);
    a->held = 0;
}

static int arity(const char* fn, Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", fn, want, n);
    return -1;
}

/* q, k_new, v_new, <planes>, slots, positions, n_heads, n_kv_heads, [head_dim,] n_slots, cap, window, sinks,
 * out, workspace, stream */
static PyObject* window_call(PyObject* const* a, Py_ssize_t n, int q8) {
    const int planes = q8 ? 4 : 2, n_int = q8 ? 6 : 7;
    void *p[7], *out, *ws, *st;
    int32_t v[7], B = 0;
    size_t bytes;
    Ints slots = {.held = 0}, pos = {.held = 0};
    PyObject* r = NULL;
    int i;
    kd_status s;
    if (arity("the windowed attention", n, 3 + planes + 2 + n_int + 3) < 0) return NULL;
    for (i = 0; i < 3 + planes; ++i)
        if (get_ptr(*a++, &p[i]) < 0) return NULL;
    if (get_ints(*a++, &slots, -1, &B) < 0 || get_ints(*a++, &pos, B, NULL) < 0) goto done;
    for (i = 0; i < n_int; ++i)
        if (get_i32(*a++, &v[i]) < 0) goto done;
    if (get_ptr(a[0], &out) < 0 || get_ptr(a[1], &ws) < 0 || get_nbytes(a[1], &bytes) < 0 || get_stream(a[2], &st) < 0)
        goto done;
    Py_BEGIN_ALLOW_THREADS
    if (q8)
        s = kd_attn_window_append_decode_q8(p[0], p[1], p[2], p[3], p[4], p[5], p[6], slots.b.buf, pos.b.buf, B, v[0], v[1],
                                            v[2], v[3], v[4], v[5], out, ws, bytes, st);
    else
        s = kd_attn_window_append_decode(p[0], p[1], p[2], p[3], p[4], slots.b.buf, pos.b.buf, B, v[0], v[1], v[2], v[3],
                                         v[4], v[5], v[6], out, ws, bytes, st);
    Py_END_ALLOW_THREADS
    r = PyLong_FromLong(s);
done:
    drop(&slots);
    drop(&pos);
    return r;
}
static PyObject* py_window(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return window_call(a, n, 0);
}
static PyObject* py_window_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return window_call(a, n, 1);
}

/* logits, ld, n_groups, n_beams, V, scores, done, eos, n_out, parents, tokens, scores_out, done_out, workspace, stream */
static PyObject* py_beam(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *x, *scores, *fin, *o[4], *ws, *st;
    int32_t G, W, V, eos, n_out;
    long long ld;
    size_t bytes;
    int i;
    kd_status s;
    (void)self;
    if (arity("kd_beam_select", n, 15) < 0 || get_ptr(a[0], &x) < 0) return NULL;
    ld = PyLong_AsLongLong(a[1]);
    if (ld == -1 && PyErr_Occurred()) return NULL;
    if (get_i32(a[2], &G) < 0 || get_i32(a[3], &W) < 0 || get_i32(a[4], &V) < 0 || get_ptr(a[5], &scores) < 0 ||
        get_ptr(a[6], &fin) < 0 || get_i32(a[7], &eos) < 0 || get_i32(a[8], &n_out) < 0)
        return NULL;
    for (i = 0; i < 4; ++i)
        if (get_ptr(a[9 + i], &o[i]) < 0) return NULL;
    if (get_ptr(a[13], &ws) < 0 || get_nbytes(a[13], &bytes) < 0 || get_stream(a[14], &st) < 0) return NULL;
    Py_BEGIN_ALLOW_THREADS
    s = kd_beam_select(x, ld, G, W, V, scores, fin, eos, n_out, o[0], o[1], o[2], o[3], ws, bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

/* planes (a sequence), dst, src, lens, n_layers, n_slots, n_kv_heads, cap, window, sinks, stream */
static PyObject* py_reorder(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *p[8], *st;
    int32_t width[8], v[6], m = 0;
    size_t bytes, rows;
    Ints dst = {.held = 0}, src = {.held = 0}, lens = {.held = 0};
    PyObject *seq, *r = NULL;
    Py_ssize_t i, k;
    kd_status s;
    (void)self;
    if (arity("kd_kv_reorder", n, 11) < 0) return NULL;
    seq = PySequence_Fast(a[0], "planes must be a sequence");
    if (!seq) return NULL;
    k = PySequence_Fast_GET_SIZE(seq);
    if (k > 8) k = 8; /* more than the call takes: refused by its count */
    for (i = 0; i < 6; ++i)
        if (get_i32(a[4 + i], &v[i]) < 0) goto done;
    if (v[0] < 1 || v[1] < 1 || v[2] < 1 || v[3] < 1) {
        PyErr_SetString(PyExc_ValueError, "n_layers, n_slots, n_kv_heads and cap must be positive");
        goto done;
    }
    if (__builtin_mul_overflow((size_t)v[0] * (size_t)v[1], (size_t)v[2], &rows) ||
        __builtin_mul_overflow(rows, (size_t)v[3], &rows)) {
        PyErr_SetString(PyExc_ValueError, "a plane's size must be a whole number of bytes per row");
        goto done;
    }
    for (i = 0; i < k; ++i) {
        PyObject* plane = PySequence_Fast_GET_ITEM(seq, i);
        if (get_ptr(plane, &p[i]) < 0 || get_nbytes(plane, &bytes) < 0) goto done;
        if (bytes % rows || bytes / rows > INT32_MAX) {
            PyErr_SetString(PyExc_ValueError, "a plane's size must be a whole number of bytes per row");
            goto done;
        }
        width[i] = (int32_t)(bytes / rows);
    }
    if (get_ints(a[1], &dst, -1, &m) < 0 || get_ints(a[2], &src, m, NULL) < 0 || get_ints(a[3], &lens, m, NULL) < 0 ||
        get_stream(a[10], &st) < 0)
        goto done;
    Py_BEGIN_ALLOW_THREADS
    s = kd_kv_reorder(p, width, (int32_t)k, v[0], v[1], v[2], v[3], dst.b.buf, src.b.buf, lens.b.buf, m, v[4], v[5], st);
    Py_END_ALLOW_THREADS
    r = PyLong_FromLong(s);
done:
    drop(&dst);
    drop(&src);
    drop(&lens);
    Py_DECREF(seq);
    return r;
}

/* setup(_ptr, _i32, _stream) */
static PyObject* py_setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (arity("setup", n, 3) < 0) return NULL;
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    Py_XSETREF(h_ptr, a[0]);
    Py_XSETREF(h_i32, a[1]);
    Py_XSETREF(h_stream, a[2]);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))py_setup, METH_FASTCALL, NULL},
    {"window", (PyCFunction)(void (*)(void))py_window, METH_FASTCALL, NULL},
    {"window_q8", (PyCFunction)(void (*)(void))py_window_q8, METH_FASTCALL, NULL},
    {"beam", (PyCFunction)(void (*)(void))py_beam, METH_FASTCALL, NULL},
    {"reorder", (PyCFunction)(void (*)(void))py_reorder, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kdcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__kdcall(void) {
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    if (!s_is_contiguous || !s_data_ptr || !s_nbytes) return NULL;
    return PyModule_Create(&module);
}
