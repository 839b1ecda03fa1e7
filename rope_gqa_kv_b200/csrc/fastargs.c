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
 * The caller then looks at the tensors one by one, to say which one does not fit (or
 * to accept one that only this path could not read): nothing is refused or let through
 * here alone.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

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

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "setup(capsule, ((dtype, code, bits), ...))"},
    {"pointers", (PyCFunction)(void (*)(void))pointers, METH_FASTCALL,
     "pointers(device, (name, tensor, dtype, shape, ...)) -> (ptr, ..., stream) or None"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastargs", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastargs(void) { return PyModule_Create(&module); }
