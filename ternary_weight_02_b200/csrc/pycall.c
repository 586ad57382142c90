/* pycall.c -- the entry points that a decode step calls per layer, as functions of a CPython
 * extension module (_bonsai_call): arguments in the order of bonsai.h, pointers as integers or
 * None, the status returned.  Converting 13 to 21 arguments takes about 0.2 us here against 1.3
 * to 2.1 us through ctypes, a third of such a call's host time. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/bonsai.h"

static void *ptr_of(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }

#define P(k) ptr_of(a[k])
#define Q(k) ((int64_t)PyLong_AsLongLong(a[k]))
#define I(k) ((int)PyLong_AsLongLong(a[k]))
#define F(k) ((float)PyFloat_AsDouble(a[k]))

/* One function: the number of arguments, its locals (converted before the call, with the
 * interpreter lock held), the call. */
#define ENTRY(name, count, locals, call)                                                     \
    static PyObject *py_##name(PyObject *self, PyObject *const *a, Py_ssize_t n) {           \
        int rc;                                                                              \
        (void)self;                                                                          \
        if (n != (count)) {                                                                  \
            PyErr_SetString(PyExc_TypeError, #name " takes " #count " arguments");           \
            return NULL;                                                                     \
        }                                                                                    \
        locals;                                                                              \
        if (PyErr_Occurred()) return NULL;                                                   \
        Py_BEGIN_ALLOW_THREADS;                                                              \
        rc = call;                                                                           \
        Py_END_ALLOW_THREADS;                                                                \
        return PyLong_FromLong(rc);                                                          \
    }

ENTRY(bonsai_ternary_linear, 9,
      const void *x = P(0); const void *w = P(1); const void *s = P(2); void *y = P(3);
      int64_t M = Q(4); int64_t N = Q(5); int64_t K = Q(6); int fmt = I(7); void *st = P(8),
      bonsai_ternary_linear(x, w, s, y, M, N, K, fmt, st))

ENTRY(bonsai_ternary_linear_swiglu, 9,
      const void *x = P(0); const void *w = P(1); const void *s = P(2); void *h = P(3);
      int64_t M = Q(4); int64_t N = Q(5); int64_t K = Q(6); int fmt = I(7); void *st = P(8),
      bonsai_ternary_linear_swiglu(x, w, s, h, M, N, K, fmt, st))

ENTRY(bonsai_ternary_linear_epilogue, 14,
      const void *x = P(0); const void *w = P(1); const void *s = P(2); const void *b = P(3);
      const void *r = P(4); void *y = P(5); int64_t M = Q(6); int64_t N = Q(7); int64_t K = Q(8);
      int fmt = I(9); int act = I(10); int algo = I(11); int split = I(12); void *st = P(13),
      bonsai_ternary_linear_epilogue(x, w, s, b, r, y, M, N, K, fmt, act, algo, split, st))

ENTRY(bonsai_rope, 13,
      const void *x = P(0); void *out = P(1); const void *f = P(2); const void *pos = P(3);
      int64_t T = Q(4); int64_t H = Q(5); int64_t D = Q(6); int64_t R = Q(7); int64_t lx = Q(8);
      int64_t lo = Q(9); float mag = F(10); int layout = I(11); void *st = P(12),
      bonsai_rope(x, out, f, pos, T, H, D, R, lx, lo, mag, layout, st))

ENTRY(bonsai_rope_append, 22,
      const void *x = P(0); void *q = P(1); void *k = P(2); void *v = P(3); const void *ks = P(4);
      const void *vs = P(5); const void *f = P(6); const void *pos = P(7); const void *slots = P(8);
      int64_t T = Q(9); int64_t Hq = Q(10); int64_t Hkv = Q(11); int64_t D = Q(12); int64_t R = Q(13);
      int64_t lx = Q(14); int64_t lq = Q(15); int64_t pages = Q(16); int64_t size = Q(17);
      float mag = F(18); int layout = I(19); int kind = I(20); void *st = P(21),
      bonsai_rope_append(x, q, k, v, ks, vs, f, pos, slots, T, Hq, Hkv, D, R, lx, lq, pages, size, mag, layout, kind, st))

ENTRY(bonsai_paged_attention, 22,
      const void *q = P(0); const void *k = P(1); const void *v = P(2); const void *ks = P(3);
      const void *vs = P(4); const void *table = P(5); const void *len = P(6); void *out = P(7);
      void *lse = P(8); int64_t B = Q(9); int64_t Hq = Q(10); int64_t Hkv = Q(11); int64_t D = Q(12);
      int64_t lq = Q(13); int64_t lo = Q(14); int64_t pages = Q(15); int64_t size = Q(16);
      int64_t width = Q(17); int64_t window = Q(18); float scale = F(19); int kind = I(20); void *st = P(21),
      bonsai_paged_attention(q, k, v, ks, vs, table, len, out, lse, B, Hq, Hkv, D, lq, lo, pages, size, width, window,
                             scale, kind, st))

#define DEF(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, "as in bonsai.h"}
static PyMethodDef methods[] = {DEF(bonsai_ternary_linear),          DEF(bonsai_ternary_linear_swiglu),
                                DEF(bonsai_ternary_linear_epilogue), DEF(bonsai_rope),
                                DEF(bonsai_rope_append),             DEF(bonsai_paged_attention),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bonsai_call", "Entry points of libbonsai.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__bonsai_call(void) { return PyModule_Create(&module); }
