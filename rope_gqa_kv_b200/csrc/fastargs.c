/*
 * fastargs.c -- the argument checks of the Python binding, in C.
 *
 * A serving loop calls several entry points per layer and token; checking the ten or
 * so tensors of one call through their Python attributes (dtype, shape, device,
 * strides, pointer) takes 12 to 18 us, three times the launch itself.  This module
 * reads them through the DLPack exchange table that torch.Tensor offers to kernel
 * libraries, some 50 ns a tensor:
 *
 *   setup(capsule, types)   the table, and ((torch dtype, DLPack code, bits), ...)
 *   pointers(device, spec)  spec = (name, tensor, dtype, shape, name, tensor, ...):
 *       a tuple of the data pointers, 0 for None, with the device's current stream at
 *       the end; or None if any tensor is not a contiguous CUDA tensor of that device,
 *       dtype and shape (shape None: any of at least one element), or cannot be read.
 *
 *   append(..), backward(..), read_back(..), decode(..)   whole calls of the entry points,
 *       the shapes that belong to each other checked too: the gqa_status, or None if
 *       any argument is not plainly right (a dtype, a shape, a device, a layout; the
 *       tensors of a device that is not the current one).
 *
 * After a None the caller looks at the arguments one by one, to say which one does not
 * fit (or to accept what only that path can): nothing is refused here alone, and without
 * this module (a torch without that table) the caller takes that path for every call.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#include "gqa.h"

#define MAX_TYPES 8

static const DLPackExchangeAPI *g_api = NULL;
static PyObject *g_keep = NULL;          /* the capsule, which owns the table */
static PyObject *g_type[MAX_TYPES];
static int g_code[MAX_TYPES], g_bits[MAX_TYPES], g_types = 0;

static PyObject *setup(PyObject *self, PyObject *args) {
    PyObject *capsule, *types;
    if (!PyArg_ParseTuple(args, "OO!", &capsule, &PyTuple_Type, &types)) return NULL;
    const DLPackExchangeAPI *api =
        (const DLPackExchangeAPI *)PyCapsule_GetPointer(capsule, "dlpack_exchange_api");
    if (!api) return NULL;
    if (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync ||
        !api->current_work_stream) {
        PyErr_SetString(PyExc_RuntimeError, "torch's DLPack exchange table is of another version");
        return NULL;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(types);
    if (n > MAX_TYPES) {
        PyErr_SetString(PyExc_ValueError, "too many types");
        return NULL;
    }
    for (int i = 0; i < g_types; ++i) Py_CLEAR(g_type[i]);
    g_types = 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *t;
        int code, bits;
        if (!PyArg_ParseTuple(PyTuple_GET_ITEM(types, i), "Oii", &t, &code, &bits)) return NULL;
        Py_INCREF(t);
        g_type[i] = t;
        g_code[i] = code;
        g_bits[i] = bits;
        g_types = (int)i + 1;
    }
    Py_INCREF(capsule);
    Py_XSETREF(g_keep, capsule);
    g_api = api;
    Py_RETURN_NONE;
}

/* 1: t is as asked, *ptr is its data; 0: it is not, or could not be read. */
static int fits(PyObject *t, PyObject *dtype, PyObject *shape, long device, void **ptr) {
    DLTensor d;
    if (g_api->dltensor_from_py_object_no_sync(t, &d) != 0) {
        PyErr_Clear();
        return 0;
    }
    if (d.device.device_type != kDLCUDA || d.device.device_id != device) return 0;
    int k = 0;
    while (k < g_types && g_type[k] != dtype) ++k;
    if (k == g_types || d.dtype.code != g_code[k] || d.dtype.bits != g_bits[k] ||
        d.dtype.lanes != 1)
        return 0;
    if (shape != Py_None) {
        if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != d.ndim) return 0;
        for (int i = 0; i < d.ndim; ++i) {
            const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
            if (want == -1 && PyErr_Occurred()) {
                PyErr_Clear();
                return 0;
            }
            if (d.shape[i] != want) return 0;
        }
    }
    int64_t step = 1;
    for (int i = d.ndim - 1; i >= 0; --i) {
        if (d.shape[i] < 1) return 0;
        if (d.strides && d.shape[i] != 1 && d.strides[i] != step) return 0;
        step *= d.shape[i];
    }
    *ptr = (char *)d.data + d.byte_offset;
    return 1;
}

static PyObject *pointers(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs != 2 || !PyTuple_Check(args[1]) || PyTuple_GET_SIZE(args[1]) % 4) {
        PyErr_SetString(PyExc_TypeError, "pointers(device, (name, tensor, dtype, shape, ...))");
        return NULL;
    }
    const long device = PyLong_AsLong(args[0]);
    if (device == -1 && PyErr_Occurred()) return NULL;
    if (!g_api) Py_RETURN_NONE;
    PyObject *spec = args[1];
    const Py_ssize_t n = PyTuple_GET_SIZE(spec) / 4;
    PyObject *out = PyTuple_New(n + 1);
    if (!out) return NULL;
    for (Py_ssize_t i = 0; i <= n; ++i) {
        void *ptr = NULL;
        int ok = 1;
        if (i < n) {
            PyObject *t = PyTuple_GET_ITEM(spec, 4 * i + 1);
            if (t != Py_None)
                ok = fits(t, PyTuple_GET_ITEM(spec, 4 * i + 2), PyTuple_GET_ITEM(spec, 4 * i + 3),
                          device, &ptr);
        } else if (g_api->current_work_stream(kDLCUDA, (int32_t)device, &ptr) != 0) {
            PyErr_Clear();
            ok = 0;
        }
        if (!ok) {
            Py_DECREF(out);
            Py_RETURN_NONE;
        }
        PyObject *v = PyLong_FromVoidPtr(ptr);
        if (!v) {
            Py_DECREF(out);
            return NULL;
        }
        PyTuple_SET_ITEM(out, i, v);
    }
    return out;
}

/* ------------------------------------------------------------------------------- */
/* whole calls                                                                       */
/* ------------------------------------------------------------------------------- */
enum { F_APPEND, F_APPEND_Q4, F_BACKWARD, F_READ, F_DECODE, F_COUNT };
static void *g_fn[F_COUNT];

/* entries((address, ...)): the library's functions, in the order above. */
static PyObject *entries(PyObject *self, PyObject *args) {
    PyObject *t;
    if (!PyArg_ParseTuple(args, "O!", &PyTuple_Type, &t)) return NULL;
    if (PyTuple_GET_SIZE(t) != F_COUNT) {
        PyErr_SetString(PyExc_ValueError, "one address for each entry point");
        return NULL;
    }
    for (int i = 0; i < F_COUNT; ++i) {
        g_fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(t, i));
        if (!g_fn[i] && PyErr_Occurred()) return NULL;
    }
    Py_RETURN_NONE;
}

typedef struct {
    void *p;
    int nd, dev;
    const int64_t *shape;              /* the tensor's own, alive as long as it is */
} view;

enum { BF16, I32, U8, F32 };
static const int k_code[] = {kDLBfloat, kDLInt, kDLUInt, kDLFloat}, k_bits[] = {16, 32, 8, 32};

/* 1: t is a contiguous, non-empty CUDA tensor of that type; or None, where it may be. */
static int look(PyObject *t, int type, int may_be_none, view *v) {
    DLTensor d;
    if (t == Py_None) {
        v->p = NULL;
        v->nd = 0;
        v->dev = -1;
        v->shape = NULL;
        return may_be_none;
    }
    if (g_api->dltensor_from_py_object_no_sync(t, &d) != 0) {
        PyErr_Clear();
        return 0;
    }
    if (d.device.device_type != kDLCUDA || d.dtype.code != k_code[type] ||
        d.dtype.bits != k_bits[type] || d.dtype.lanes != 1)
        return 0;
    int64_t step = 1;
    for (int i = d.ndim - 1; i >= 0; --i) {
        if (d.shape[i] < 1 || d.shape[i] > 0x7fffffff) return 0;
        if (d.strides && d.shape[i] != 1 && d.strides[i] != step) return 0;
        step *= d.shape[i];
    }
    v->p = (char *)d.data + d.byte_offset;
    v->nd = d.ndim;
    v->dev = d.device.device_id;
    v->shape = d.shape;
    return 1;
}

/* None, or on device dev with n dims of these sizes (n < 0: any). */
static int is(const view *v, int dev, int n, int64_t a, int64_t b, int64_t c, int64_t d, int64_t e) {
    const int64_t want[5] = {a, b, c, d, e};
    if (!v->p) return 1;
    if (v->dev != dev) return 0;
    if (n < 0) return 1;
    if (v->nd != n) return 0;
    for (int i = 0; i < n; ++i)
        if (v->shape[i] != want[i]) return 0;
    return 1;
}

static int whole(PyObject *o, int *out) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return 0;
    }
    *out = (int)x;
    return x >= -0x7fffffffL && x <= 0x7fffffffL;
}

static int bytes_of(PyObject *o, void *out, size_t n) {
    if (!PyBytes_Check(o) || (size_t)PyBytes_GET_SIZE(o) != n) return 0;
    memcpy(out, PyBytes_AS_STRING(o), n);
    return 1;
}

/* The given stream's handle, or dev's current one. */
static int stream_of(PyObject *o, int dev, void **s) {
    if (o != Py_None) {
        *s = PyLong_AsVoidPtr(o);
        if (!*s && PyErr_Occurred()) {
            PyErr_Clear();
            return 0;
        }
        return 1;
    }
    if (g_api->current_work_stream(kDLCUDA, dev, s) != 0) {
        PyErr_Clear();
        return 0;
    }
    return 1;
}

/* Gains, positions and axes (None, or the bytes of a gqa_rope_inputs without pointers,
 * with the number of pairs that it covers).  *use: NULL where there is nothing. */
static int rope_of(PyObject *qg, PyObject *kg, PyObject *po, PyObject *axes, PyObject *n_pairs,
                   const gqa_rope_params *p, int dev, int64_t B, int64_t T, int64_t D,
                   gqa_rope_inputs *x, gqa_rope_inputs **use) {
    view g, h, v;
    int pairs;
    if (!look(qg, BF16, 1, &g) || !look(kg, BF16, 1, &h) || !look(po, I32, 1, &v)) return 0;
    if (!is(&g, dev, 1, D, 0, 0, 0, 0) || !is(&h, dev, 1, D, 0, 0, 0, 0)) return 0;
    if ((g.p || h.p) && !p->qk_norm) return 0;
    memset(x, 0, sizeof *x);
    x->n_axes = 1;
    if (axes != Py_None) {
        if (!v.p || !bytes_of(axes, x, sizeof *x) || !whole(n_pairs, &pairs) || pairs * 2 != D)
            return 0;
    }
    if (v.p) {
        const int64_t n = x->n_axes;
        const int two = v.nd == 2 && ((T == 1 && v.shape[0] == n && v.shape[1] == B) ||
                                      (n == 1 && v.shape[0] == B && v.shape[1] == T));
        if (v.dev != dev || (!two && !is(&v, dev, 3, n, B, T, 0, 0))) return 0;
    }
    x->q_gain = g.p;
    x->k_gain = h.p;
    x->pos = (const int32_t *)v.p;
    *use = g.p || h.p || v.p ? x : NULL;
    return 1;
}

#define STATUS(call)                          \
    do {                                      \
        int st;                               \
        Py_BEGIN_ALLOW_THREADS                \
        st = (int)(call);                     \
        Py_END_ALLOW_THREADS                  \
        return PyLong_FromLong(st);           \
    } while (0)

/* append(q4, current device, q, k, v, q_out, c0, c1, c2, c3, pos0, n_tok, new_len, status,
 *        q_gain, k_gain, pos, max_pos0, params, axes, pairs, stream) */
static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view q, k, v, qo, c[4], pos0, n_tok, new_len, status;
    int q4, dev, max_pos0;
    gqa_rope_params p;
    gqa_rope_inputs x, *use;
    void *s;
    if (n != 22 || !g_api || !whole(a[0], &q4) || !whole(a[1], &dev)) Py_RETURN_NONE;
    if (!look(a[2], BF16, 1, &q) || !look(a[3], BF16, 0, &k) || !look(a[4], BF16, 0, &v) ||
        !look(a[5], BF16, 1, &qo))
        Py_RETURN_NONE;
    if (k.dev != dev || (k.nd != 3 && k.nd != 4)) Py_RETURN_NONE;
    const int four = k.nd == 4;
    const int64_t B = k.shape[0], T = four ? k.shape[1] : 1, Hkv = k.shape[k.nd - 2],
                  D = k.shape[k.nd - 1], Hq = q.p && q.nd == k.nd ? q.shape[k.nd - 2] : 0;
    const int64_t d2 = four ? Hkv : D, d3 = four ? D : 0;
    if (!is(&v, dev, k.nd, B, four ? T : Hkv, d2, d3, 0) || !q.p != !qo.p) Py_RETURN_NONE;
    const int64_t e1 = four ? T : Hq, e2 = four ? Hq : D;
    if (!is(&q, dev, k.nd, B, e1, e2, d3, 0) || !is(&qo, dev, k.nd, B, e1, e2, d3, 0))
        Py_RETURN_NONE;
    int64_t L;
    if (q4) {
        for (int i = 0; i < 4; ++i)
            if (!look(a[6 + i], i % 2 ? BF16 : U8, 0, &c[i])) Py_RETURN_NONE;
        if (c[0].nd != 4) Py_RETURN_NONE;
        L = c[0].shape[2];
        for (int i = 0; i < 4; i += 2)
            if (!is(&c[i], dev, 4, B, Hkv, L, D / 2, 0) || D % 32 ||
                !is(&c[i + 1], dev, 5, B, Hkv, L, D / 32, 2))
                Py_RETURN_NONE;
    } else {
        for (int i = 0; i < 2; ++i)
            if (!look(a[6 + i], BF16, 0, &c[i])) Py_RETURN_NONE;
        if (c[0].nd != 4) Py_RETURN_NONE;
        L = c[0].shape[2];
        if (!is(&c[0], dev, 4, B, Hkv, L, D, 0) || !is(&c[1], dev, 4, B, Hkv, L, D, 0))
            Py_RETURN_NONE;
    }
    if (!look(a[10], I32, 1, &pos0) || !look(a[11], I32, 1, &n_tok) ||
        !look(a[12], I32, 1, &new_len) || !look(a[13], I32, 1, &status) ||
        !is(&pos0, dev, 1, B, 0, 0, 0, 0) || !is(&n_tok, dev, 1, B, 0, 0, 0, 0) ||
        !is(&new_len, dev, 1, B, 0, 0, 0, 0) || !is(&status, dev, -1, 0, 0, 0, 0, 0))
        Py_RETURN_NONE;
    if (!whole(a[17], &max_pos0) || !bytes_of(a[18], &p, sizeof p) ||
        !rope_of(a[14], a[15], a[16], a[19], a[20], &p, dev, B, T, D, &x, &use) ||
        !stream_of(a[21], dev, &s))
        Py_RETURN_NONE;
    if (q4)
        STATUS(((__typeof__(&gqa_norm_rope_append_q4))g_fn[F_APPEND_Q4])(
            q.p, k.p, v.p, qo.p, c[0].p, c[1].p, c[2].p, c[3].p, pos0.p, n_tok.p, max_pos0,
            new_len.p, (int)B, (int)T, (int)Hq, (int)Hkv, (int)D, (int)L, p, use, status.p, s));
    STATUS(((__typeof__(&gqa_norm_rope_append))g_fn[F_APPEND])(
        q.p, k.p, v.p, qo.p, c[0].p, c[1].p, pos0.p, n_tok.p, max_pos0, new_len.p, (int)B, (int)T,
        (int)Hq, (int)Hkv, (int)D, (int)L, p, use, status.p, s));
}

/* backward(current device, q, k, dq_out, dk_cache, dv_cache, dq, dk, dv, gains' gradients
 *          [2, D] or None, pos0, workspace, status, q_gain, k_gain, pos, max_pos0, params,
 *          axes, pairs, stream) */
static PyObject *backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view t[8], dg, pos0, ws, status;
    int dev, max_pos0;
    gqa_rope_params p;
    gqa_rope_inputs x, *use;
    void *s;
    if (n != 21 || !g_api || !whole(a[0], &dev)) Py_RETURN_NONE;
    for (int i = 0; i < 8; ++i)
        if (!look(a[1 + i], BF16, 0, &t[i]) || t[i].nd != 4) Py_RETURN_NONE;
    const int64_t B = t[0].shape[0], T = t[0].shape[1], Hq = t[0].shape[2], D = t[0].shape[3],
                  Hkv = t[1].shape[2], L = t[3].shape[2];
    for (int i = 0; i < 8; ++i) {
        const int q = i == 0 || i == 2 || i == 5, cache = i == 3 || i == 4;
        if (cache ? !is(&t[i], dev, 4, B, Hkv, L, D, 0) : !is(&t[i], dev, 4, B, T, q ? Hq : Hkv, D, 0))
            Py_RETURN_NONE;
    }
    if (!look(a[9], F32, 1, &dg) || !look(a[10], I32, 1, &pos0) || !look(a[11], U8, 1, &ws) ||
        !look(a[12], I32, 1, &status) || !is(&dg, dev, 2, 2, D, 0, 0, 0) ||
        !is(&pos0, dev, 1, B, 0, 0, 0, 0) || !is(&ws, dev, -1, 0, 0, 0, 0, 0) ||
        !is(&status, dev, -1, 0, 0, 0, 0, 0))
        Py_RETURN_NONE;
    size_t ws_bytes = ws.p ? 1 : 0;
    for (int i = 0; i < ws.nd; ++i) ws_bytes *= (size_t)ws.shape[i];
    if (!whole(a[16], &max_pos0) || !bytes_of(a[17], &p, sizeof p) ||
        !rope_of(a[13], a[14], a[15], a[18], a[19], &p, dev, B, T, D, &x, &use) ||
        !stream_of(a[20], dev, &s))
        Py_RETURN_NONE;
    float *g = dg.p;
    STATUS(((__typeof__(&gqa_norm_rope_append_backward))g_fn[F_BACKWARD])(
        t[0].p, t[1].p, t[2].p, t[3].p, t[4].p, t[5].p, t[6].p, t[7].p, g, g ? g + D : NULL,
        pos0.p, max_pos0, (int)B, (int)T, (int)Hq, (int)Hkv, (int)D, (int)L, p, use, ws.p, ws_bytes,
        status.p, s));
}

/* A 4-bit cache's four tensors a[0 .. 3]; sizes from the first. */
static int cache_of(PyObject *const *a, int dev, view *c, int64_t *B, int64_t *Hkv, int64_t *L,
                    int64_t *D) {
    for (int i = 0; i < 4; ++i)
        if (!look(a[i], i % 2 ? BF16 : U8, 0, &c[i])) return 0;
    if (c[0].nd != 4) return 0;
    *B = c[0].shape[0];
    *Hkv = c[0].shape[1];
    *L = c[0].shape[2];
    *D = 2 * c[0].shape[3];
    for (int i = 0; i < 4; i += 2)
        if (*D % 32 || !is(&c[i], dev, 4, *B, *Hkv, *L, *D / 2, 0) ||
            !is(&c[i + 1], dev, 5, *B, *Hkv, *L, *D / 32, 2))
            return 0;
    return 1;
}

/* cache(k_codes, k_scales, v_codes, v_scales): (B, Hkv, Lmax, D) of a 4-bit cache, or None. */
static PyObject *cache(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view c[4];
    int64_t B, Hkv, L, D;
    if (n != 4 || !g_api || !look(a[0], U8, 0, &c[0]) ||
        !cache_of(a, c[0].dev, c, &B, &Hkv, &L, &D) || (D != 64 && D != 96 && D != 128))
        Py_RETURN_NONE;
    return Py_BuildValue("(iiii)", (int)B, (int)Hkv, (int)L, (int)D);
}

/* read_back(current device, k_codes, k_scales, v_codes, v_scales, first, count, k_out, v_out,
 *      status, stream) */
static PyObject *read_back(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view c[4], first, count, ko, vo, status;
    int dev;
    int64_t B, Hkv, L, D;
    void *s;
    if (n != 11 || !g_api || !whole(a[0], &dev) || !cache_of(a + 1, dev, c, &B, &Hkv, &L, &D))
        Py_RETURN_NONE;
    if (!look(a[5], I32, 1, &first) || !look(a[6], I32, 1, &count) || !look(a[7], BF16, 0, &ko) ||
        !look(a[8], BF16, 0, &vo) || !look(a[9], I32, 1, &status) || ko.nd != 4)
        Py_RETURN_NONE;
    const int64_t Lout = ko.shape[2];
    if (!is(&first, dev, 1, B, 0, 0, 0, 0) || !is(&count, dev, 1, B, 0, 0, 0, 0) ||
        !is(&ko, dev, 4, B, Hkv, Lout, D, 0) || !is(&vo, dev, 4, B, Hkv, Lout, D, 0) ||
        !is(&status, dev, -1, 0, 0, 0, 0, 0) || !stream_of(a[10], dev, &s))
        Py_RETURN_NONE;
    STATUS(((__typeof__(&kv_cache_read_q4))g_fn[F_READ])(
        c[0].p, c[1].p, c[2].p, c[3].p, first.p, count.p, ko.p, vo.p, (int)B, (int)Hkv, (int)D,
        (int)L, (int)Lout, status.p, s));
}

/* decode(current device, k_codes, k_scales, v_codes, v_scales, q, lens, max_len, out, scale,
 *        workspace, status, stream) */
static PyObject *decode(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    view c[4], q, lens, out, ws, status;
    int dev, max_len;
    int64_t B, Hkv, L, D;
    void *s;
    if (n != 13 || !g_api || !whole(a[0], &dev) || !cache_of(a + 1, dev, c, &B, &Hkv, &L, &D))
        Py_RETURN_NONE;
    if (!look(a[5], BF16, 0, &q) || !look(a[6], I32, 0, &lens) || !whole(a[7], &max_len) ||
        !look(a[8], BF16, 0, &out) || !look(a[10], U8, 0, &ws) || !look(a[11], I32, 1, &status) ||
        q.nd != 3 || !PyFloat_Check(a[9]))
        Py_RETURN_NONE;
    const int64_t Hq = q.shape[1];
    if (!is(&q, dev, 3, B, Hq, D, 0, 0) || !is(&out, dev, 3, B, Hq, D, 0, 0) ||
        !is(&lens, dev, 1, B, 0, 0, 0, 0) || !is(&ws, dev, -1, 0, 0, 0, 0, 0) ||
        !is(&status, dev, -1, 0, 0, 0, 0, 0) || !stream_of(a[12], dev, &s))
        Py_RETURN_NONE;
    size_t ws_bytes = 1;
    for (int i = 0; i < ws.nd; ++i) ws_bytes *= (size_t)ws.shape[i];
    const float scale = (float)PyFloat_AS_DOUBLE(a[9]);
    STATUS(((__typeof__(&gqa_decode_q4))g_fn[F_DECODE])(
        q.p, c[0].p, c[1].p, c[2].p, c[3].p, lens.p, max_len, out.p, (int)B, (int)Hq, (int)Hkv,
        (int)D, (int)L, scale, ws.p, ws_bytes, status.p, s));
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "setup(capsule, ((dtype, code, bits), ...))"},
    {"pointers", (PyCFunction)(void (*)(void))pointers, METH_FASTCALL,
     "pointers(device, (name, tensor, dtype, shape, ...)) -> (ptr, ..., stream) or None"},
    {"entries", entries, METH_VARARGS, "entries((address, ...))"},
    FAST(append),
    FAST(backward),
    FAST(read_back),
    FAST(cache),
    FAST(decode),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastargs", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastargs(void) { return PyModule_Create(&module); }
