/* CPython entry to the calls of a serving step (rotary positions and the 8-bit
 * cache), for which the conversion of some thirty arguments by ctypes would
 * take longer than a small kernel: the same C functions, their arguments in
 * the same order as integers (pointers; None is NULL) and floats, the
 * tg_status as the result. The library runs without the interpreter lock. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "tg_gemm.h"

static int64_t as_int(PyObject* x) { return x == Py_None ? 0 : (int64_t)PyLong_AsLongLong(x); }

static void* as_ptr(PyObject* x) {
    return x == Py_None ? NULL : (void*)(uintptr_t)PyLong_AsUnsignedLongLong(x);
}

static int take(const char* name, PyObject* const* args, Py_ssize_t n, Py_ssize_t want) {
    (void)args;
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
    return 0;
}

#define I(k) as_int(args[k])
#define N(k) (int)as_int(args[k])
#define P(k) as_ptr(args[k])
#define D(k) PyFloat_AsDouble(args[k])

#define ANSWER(call)                            \
    do {                                        \
        if (PyErr_Occurred()) return NULL;      \
        int status;                             \
        Py_BEGIN_ALLOW_THREADS status = (call); \
        Py_END_ALLOW_THREADS                    \
        return PyLong_FromLong(status);         \
    } while (0)

static PyObject* rope(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (!take("rope", args, n, 17)) return NULL;
    const void* x = P(0);
    const int64_t xt = I(1), xh = I(2);
    void* y = P(3);
    const int64_t yt = I(4), yh = I(5);
    const int32_t* pos = P(6);
    const int64_t tokens = I(7), heads = I(8), dim = I(9);
    const double* freq = P(10);
    const int64_t rotary = I(11);
    const double amplitude = D(12);
    const int layout = N(13), backward = N(14), dtype = N(15);
    tg_stream_t stream = P(16);
    ANSWER(tg_rope(x, xt, xh, y, yt, yh, pos, tokens, heads, dim, freq, rotary, amplitude, layout, backward, dtype, stream));
}

static PyObject* kv_append(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (!take("kv_append", args, n, 35)) return NULL;
    void *k = P(0), *v = P(1);
    float *ks = P(2), *vs = P(3);
    const int64_t pages = I(4), kv_heads = I(5), page = I(6), dim = I(7);
    const int format = N(8);
    const void* nk = P(9);
    const int64_t kt = I(10), kh = I(11);
    const void* nv = P(12);
    const int64_t vt = I(13), vh = I(14);
    const int32_t* table = P(15);
    const int64_t width = I(16);
    const int32_t *lens = P(17), *cu = P(18);
    const int64_t batch = I(19), total = I(20), max_new = I(21);
    const double* freq = P(22);
    const int64_t rotary = I(23);
    const double amplitude = D(24);
    const int layout = N(25);
    const void* q = P(26);
    const int64_t qt = I(27), qh = I(28);
    void* qo = P(29);
    const int64_t qot = I(30), qoh = I(31), heads = I(32);
    const int dtype = N(33);
    tg_stream_t stream = P(34);
    ANSWER(tg_kv_append(k, v, ks, vs, pages, kv_heads, page, dim, format, nk, kt, kh, nv, vt, vh, table, width, lens, cu, batch, total, max_new,
                        freq, rotary, amplitude, layout, q, qt, qh, qo, qot, qoh, heads, dtype, stream));
}

static PyObject* kv_read(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (!take("kv_read", args, n, 19)) return NULL;
    const void *k = P(0), *v = P(1);
    const float *ks = P(2), *vs = P(3);
    const int64_t pages = I(4), kv_heads = I(5), page = I(6), dim = I(7);
    const int format = N(8);
    const int32_t* table = P(9);
    const int64_t width = I(10);
    const int32_t *first = P(11), *cu = P(12);
    const int64_t batch = I(13), total = I(14);
    void *ok = P(15), *ov = P(16);
    const int dtype = N(17);
    tg_stream_t stream = P(18);
    ANSWER(tg_kv_read(k, v, ks, vs, pages, kv_heads, page, dim, format, table, width, first, cu, batch, total, ok, ov, dtype, stream));
}

static PyObject* attention_kv(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (!take("attention_kv", args, n, 30)) return NULL;
    const void* q = P(0);
    const int64_t qt = I(1), qh = I(2);
    void* o = P(3);
    float* lse = P(4);
    const void *k = P(5), *v = P(6);
    const float *ks = P(7), *vs = P(8);
    const int64_t pages = I(9), kv_heads = I(10), page = I(11), dim = I(12);
    const int format = N(13);
    const int32_t* table = P(14);
    const int64_t width = I(15);
    const int32_t *lens = P(16), *cu = P(17);
    const int64_t batch = I(18), total = I(19), heads = I(20), max_new = I(21), max_len = I(22);
    const int causal = N(23);
    const int64_t window = I(24);
    const double scale = D(25);
    const int dtype = N(26);
    void* work = P(27);
    const int64_t work_bytes = I(28);
    tg_stream_t stream = P(29);
    ANSWER(tg_attention_kv(q, qt, qh, o, lse, k, v, ks, vs, pages, kv_heads, page, dim, format, table, width, lens, cu, batch, total, heads, max_new,
                           max_len, causal, window, scale, dtype, work, work_bytes, stream));
}

static PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, "tg_rope"},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, "tg_kv_append"},
    {"kv_read", (PyCFunction)(void (*)(void))kv_read, METH_FASTCALL, "tg_kv_read"},
    {"attention_kv", (PyCFunction)(void (*)(void))attention_kv, METH_FASTCALL, "tg_attention_kv"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tg_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tg_binding(void) { return PyModule_Create(&module); }
