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

static PyObject *s_is_contiguous, *s_data_ptr, *s_nbytes, *s_shape, *s_stride, *s_dtype, *s_numel;
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

static int get_i64(PyObject* o, int64_t* out) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    *out = v;
    return 0;
}

/* torch's types, known once it is loaded (a tensor is at hand then). */
static PyObject *t_f32, *t_f16, *t_bf16, *t_i32;
static int find_types(void) {
    PyObject* torch;
    if (t_i32) return 0;
    torch = PyImport_ImportModule("torch");
    if (!torch) return -1;
    t_f32 = PyObject_GetAttrString(torch, "float32");
    t_f16 = PyObject_GetAttrString(torch, "float16");
    t_bf16 = PyObject_GetAttrString(torch, "bfloat16");
    t_i32 = PyObject_GetAttrString(torch, "int32");
    Py_DECREF(torch);
    return t_f32 && t_f16 && t_bf16 && t_i32 ? 0 : -1;
}

/* A tuple of n integers, the attribute `name` of o or what its method of that name returns (0: as many, -1: an error, 1: not n). */
static int get_sizes(PyObject* o, PyObject* name, int method, Py_ssize_t n, int64_t* out) {
    PyObject* v = method ? PyObject_CallMethodNoArgs(o, name) : PyObject_GetAttr(o, name);
    Py_ssize_t i;
    if (!v) return -1;
    if (!PyTuple_Check(v) || PyTuple_GET_SIZE(v) != n) {
        Py_DECREF(v);
        return 1;
    }
    for (i = 0; i < n; ++i)
        if (get_i64(PyTuple_GET_ITEM(v, i), &out[i]) < 0) {
            Py_DECREF(v);
            return -1;
        }
    Py_DECREF(v);
    return 0;
}
static int is_type(PyObject* o, PyObject* want) { /* the tensor's type; -1: an error */
    PyObject* v = PyObject_GetAttr(o, s_dtype);
    if (!v) return -1;
    Py_DECREF(v); /* torch keeps its types */
    return v == want;
}

/* A tensor [rows][heads][head_dim] whose heads lie one after another; rows may be further apart. */
typedef struct {
    void* p;
    int64_t ld, rows, heads, dim;
    int32_t dtype;
} Heads;
static int get_heads(PyObject* o, const char* what, Heads* h) {
    int64_t n[3], st[3];
    PyObject* v;
    int r;
    if (find_types() < 0) return -1;
    if ((r = get_sizes(o, s_shape, 0, 3, n)) < 0 || (!r && (r = get_sizes(o, s_stride, 1, 3, st)) < 0)) return -1;
    if (!r) {
        v = PyObject_GetAttr(o, s_dtype);
        if (!v) return -1;
        Py_DECREF(v);
        h->dtype = v == t_f32 ? KD_F32 : v == t_f16 ? KD_F16 : v == t_bf16 ? KD_BF16 : -1;
        r = h->dtype < 0 || (st[2] != 1 && n[2] > 1) || (st[1] != n[2] && n[1] > 1);
    }
    if (r) {
        PyErr_Format(PyExc_ValueError, "%s must be fp32, fp16 or bf16 [rows][heads][head_dim] with its heads one after another", what);
        return -1;
    }
    h->rows = n[0];
    h->heads = n[1];
    h->dim = n[2];
    h->ld = n[0] > 1 || st[0] > n[1] * n[2] ? st[0] : n[1] * n[2];
    v = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!v) return -1;
    h->p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return h->p == NULL && PyErr_Occurred() ? -1 : 0;
}
static int alike(const Heads* a, const Heads* b) {
    return a->rows == b->rows && a->heads == b->heads && a->dim == b->dim && a->dtype == b->dtype;
}

/* An int32 tensor [at least rows][pages]. */
static int get_table(PyObject* o, int32_t rows, void** p, int32_t* ld) {
    int64_t n[2];
    int r, ok;
    if (find_types() < 0 || (r = get_sizes(o, s_shape, 0, 2, n)) < 0 || (ok = is_type(o, t_i32)) < 0) return -1;
    if (r || !ok || n[0] < rows || n[1] > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "the page table must be int32 [sessions][pages], with %d sessions or more", (int)rows);
        return -1;
    }
    *ld = (int32_t)n[1];
    return get_ptr(o, p);
}

/* A kd_rope_table (a ctypes structure), or None. */
static int get_rope(PyObject* o, Py_buffer* b, const kd_rope_table** out) {
    *out = NULL;
    b->obj = NULL;
    if (o == Py_None) return 0;
    if (PyObject_GetBuffer(o, b, PyBUF_SIMPLE) < 0) return -1;
    if ((size_t)b->len < sizeof(kd_rope_table)) {
        PyBuffer_Release(b);
        PyErr_SetString(PyExc_TypeError, "expected the table that kd_rope_plan returns");
        return -1;
    }
    *out = b->buf;
    return 0;
}

/* plan, x, positions, out, stream */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    const kd_rope_table* table;
    Py_buffer plan;
    Heads x, out;
    PyObject *r = NULL, *v;
    void *pos, *st;
    int64_t count;
    int ok;
    kd_status s;
    (void)self;
    if (arity("kd_rope", n, 5) < 0 || get_rope(a[0], &plan, &table) < 0) return NULL;
    if (get_heads(a[1], "x", &x) < 0 || get_heads(a[3], "out", &out) < 0) goto done;
    if (!alike(&x, &out) || (table && x.dim != table->head_dim)) {
        PyErr_SetString(PyExc_ValueError, "x and out must be alike, in heads of the plan's head_dim");
        goto done;
    }
    if (x.rows > INT32_MAX || x.heads > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "too many rows");
        goto done;
    }
    v = PyObject_CallMethodNoArgs(a[2], s_numel);
    if (!v) goto done;
    ok = get_i64(v, &count);
    Py_DECREF(v);
    if (ok < 0 || (ok = is_type(a[2], t_i32)) < 0) goto done;
    if (!ok || count != x.rows) {
        PyErr_Format(PyExc_ValueError, "expected %lld int32 positions", (long long)x.rows);
        goto done;
    }
    if (get_ptr(a[2], &pos) < 0 || get_stream(a[4], &st) < 0) goto done;
    Py_BEGIN_ALLOW_THREADS
    s = kd_rope(table, x.p, x.dtype, x.ld, pos, (int32_t)x.rows, (int32_t)x.heads, out.p, out.ld, st);
    Py_END_ALLOW_THREADS
    r = PyLong_FromLong(s);
done:
    if (plan.obj) PyBuffer_Release(&plan);
    return r;
}

/* The planes of a cache, 2 (fp16 rows) or 4 (Q8_0). */
static int get_planes(PyObject* o, void** p) {
    Py_ssize_t i, n;
    PyObject* seq = PySequence_Fast(o, "planes must be a sequence");
    if (!seq) return -1;
    n = PySequence_Fast_GET_SIZE(seq);
    if (n != 2 && n != 4) {
        PyErr_SetString(PyExc_ValueError, "a cache has 2 or 4 planes");
        n = -1;
    }
    for (i = 0; i < n; ++i)
        if (get_ptr(PySequence_Fast_GET_ITEM(seq, i), &p[i]) < 0) {
            n = -1;
            break;
        }
    Py_DECREF(seq);
    return (int)n;
}

/* A tensor or array of `bytes` or more (addresses and None are taken as they are). */
static int check_size(PyObject* o, double bytes, const char* what) {
    size_t n;
    if (o == Py_None || PyLong_Check(o)) return 0;
    if (get_nbytes(o, &n) < 0) return -1;
    if ((double)n >= bytes) return 0;
    PyErr_Format(PyExc_ValueError, "%s is smaller than the call's sizes", what);
    return -1;
}
/* c: n_heads, n_kv_heads, head_dim, n_pages, page_size */
static int check_planes(PyObject* o, int planes, const int32_t* c) {
    const double rows = (double)c[3] * c[1] * c[4];
    PyObject* seq = PySequence_Fast(o, "planes must be a sequence");
    int i, r = 0;
    if (!seq) return -1;
    for (i = 0; i < planes && !r; ++i)
        r = check_size(PySequence_Fast_GET_ITEM(seq, i), rows * (planes == 2 ? 2.0 * c[2] : i & 1 ? 8 : 128), "a plane of the cache");
    Py_DECREF(seq);
    return r;
}

/* plan, k_new, v_new, planes, table, starts, counts, n_heads, n_kv_heads, head_dim, n_pages, page_size, q, q_out, fault,
 * stream */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    const kd_rope_table* rope;
    Py_buffer plan;
    Heads k, v, q = {.p = NULL}, q_out = {.p = NULL};
    void *p[4], *table, *fault, *st;
    int64_t sum = 0;
    int32_t table_ld, c[5], B = 0;
    Ints starts = {.held = 0}, counts = {.held = 0};
    PyObject* r = NULL;
    int i, planes, below = 0;
    kd_status s;
    (void)self;
    if (arity("kd_paged_append", n, 16) < 0 || get_rope(a[0], &plan, &rope) < 0) return NULL;
    if (get_heads(a[1], "k_new", &k) < 0 || get_heads(a[2], "v_new", &v) < 0 || (planes = get_planes(a[3], p)) < 0) goto done;
    for (i = 0; i < 5; ++i)
        if (get_i32(a[7 + i], &c[i]) < 0) goto done;
    if (check_planes(a[3], planes, c) < 0) goto done;
    if (!alike(&k, &v) || k.heads != c[1] || k.dim != c[2]) {
        PyErr_SetString(PyExc_ValueError, "k_new and v_new must be alike: [rows][n_kv_heads][head_dim]");
        goto done;
    }
    if (a[12] != Py_None) {
        if (get_heads(a[12], "q", &q) < 0 || get_heads(a[13], "q_out", &q_out) < 0) goto done;
        if (q.rows != k.rows || q.heads != c[0] || q.dim != c[2] || q.dtype != k.dtype || q_out.rows != k.rows ||
            q_out.heads != c[0] || q_out.dim != c[2] || q_out.dtype != KD_F32 || q_out.ld != q.heads * q.dim) {
            PyErr_SetString(PyExc_ValueError, "q must be [rows][n_heads][head_dim] of k_new's type, and q_out so in contiguous fp32");
            goto done;
        }
    }
    if (get_ints(a[5], &starts, -1, &B) < 0 || get_ints(a[6], &counts, B, NULL) < 0 || get_table(a[4], B, &table, &table_ld) < 0 ||
        get_ptr(a[14], &fault) < 0 || get_stream(a[15], &st) < 0)
        goto done;
    for (i = 0; i < B; ++i) {
        const int32_t count = ((const int32_t*)counts.b.buf)[i];
        below |= count < 0;
        sum += count;
    }
    if (!below && sum != k.rows) {
        PyErr_Format(PyExc_ValueError, "%lld new rows for counts of %lld in all", (long long)k.rows, (long long)sum);
        goto done;
    }
    Py_BEGIN_ALLOW_THREADS
    if (planes == 2)
        s = kd_paged_append(rope, k.p, k.ld, v.p, v.ld, q.p, q.ld, k.dtype, p[0], p[1], table, table_ld, starts.b.buf, counts.b.buf,
                            B, c[0], c[1], c[2], c[3], c[4], q_out.p, fault, st);
    else
        s = kd_paged_append_q8(rope, k.p, k.ld, v.p, v.ld, q.p, q.ld, k.dtype, p[0], p[1], p[2], p[3], table, table_ld,
                               starts.b.buf, counts.b.buf, B, c[0], c[1], c[3], c[4], q_out.p, fault, st);
    Py_END_ALLOW_THREADS
    r = PyLong_FromLong(s);
done:
    if (plan.obj) PyBuffer_Release(&plan);
    drop(&starts);
    drop(&counts);
    return r;
}

/* q, planes, table, lens, group_rows, group_prefix, n_heads, n_kv_heads, head_dim, n_pages, page_size, out,
 * workspace, fault, stream */
static PyObject* py_paged(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *q, *p[4], *table, *out, *ws, *fault, *st;
    int32_t table_ld, v[5], B = 0, G = 0;
    size_t bytes;
    Ints lens = {.held = 0}, rows = {.held = 0}, prefix = {.held = 0};
    PyObject* r = NULL;
    int i, planes;
    kd_status s;
    (void)self;
    if (arity("kd_attn_paged_decode", n, 15) < 0 || get_ptr(a[0], &q) < 0 || (planes = get_planes(a[1], p)) < 0) return NULL;
    if (get_ints(a[3], &lens, -1, &B) < 0 || get_table(a[2], B, &table, &table_ld) < 0) goto done;
    if (a[4] != Py_None && get_ints(a[4], &rows, -1, &G) < 0) goto done;
    if (a[5] != Py_None && get_ints(a[5], &prefix, G, NULL) < 0) goto done;
    if (a[5] == Py_None && G > 0) {
        PyErr_SetString(PyExc_ValueError, "groups without prefixes");
        goto done;
    }
    for (i = 0; i < 5; ++i)
        if (get_i32(a[6 + i], &v[i]) < 0) goto done;
    if (check_size(a[0], 4.0 * B * v[0] * v[2], "q") < 0 || check_planes(a[1], planes, v) < 0 ||
        check_size(a[11], 2.0 * B * v[0] * v[2], "out") < 0)
        goto done;
    if (get_ptr(a[11], &out) < 0 || get_ptr(a[12], &ws) < 0 || get_nbytes(a[12], &bytes) < 0 || get_ptr(a[13], &fault) < 0 ||
        get_stream(a[14], &st) < 0)
        goto done;
    Py_BEGIN_ALLOW_THREADS
    if (planes == 2)
        s = kd_attn_paged_decode(q, p[0], p[1], table, table_ld, lens.b.buf, B, G ? rows.b.buf : NULL, G ? prefix.b.buf : NULL,
                                 G, v[0], v[1], v[2], v[3], v[4], out, ws, bytes, fault, st);
    else
        s = kd_attn_paged_decode_q8(q, p[0], p[1], p[2], p[3], table, table_ld, lens.b.buf, B, G ? rows.b.buf : NULL,
                                    G ? prefix.b.buf : NULL, G, v[0], v[1], v[3], v[4], out, ws, bytes, fault, st);
    Py_END_ALLOW_THREADS
    r = PyLong_FromLong(s);
done:
    drop(&lens);
    drop(&rows);
    drop(&prefix);
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
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"paged", (PyCFunction)(void (*)(void))py_paged, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kdcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__kdcall(void) {
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_numel = PyUnicode_InternFromString("numel");
    if (!s_is_contiguous || !s_data_ptr || !s_nbytes || !s_shape || !s_stride || !s_dtype || !s_numel) return NULL;
    return PyModule_Create(&module);
}
