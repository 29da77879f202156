/* Argument marshalling of the attention-side calls for Python: each function
 * takes the arguments of its namesake in tern.h, in order, and returns the
 * status.  A pointer argument is None, an address or an object with a
 * data_ptr() method (a tensor).
 *
 * These calls take 18 to 28 arguments and are made for single tokens, where the
 * GPU's part is 2 us: ctypes takes 1.8 us to convert the arguments and the
 * data_ptr() calls from Python another 0.9 us, against 0.5 us here. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "tern.h"

static PyObject* g_data_ptr;   /* interned "data_ptr" */

static int as_ptr(PyObject* o, void** out) {
    *out = NULL;
    if (o == Py_None) return 1;
    if (PyLong_Check(o)) {
        *out = PyLong_AsVoidPtr(o);
        return !(*out == NULL && PyErr_Occurred());
    }
    PyObject* p = PyObject_CallMethodNoArgs(o, g_data_ptr);
    if (p == NULL) return 0;
    *out = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return !(*out == NULL && PyErr_Occurred());
}

static int as_i64(PyObject* o, int64_t* out) {
    if (PyLong_Check(o)) {
        *out = PyLong_AsLongLong(o);
    } else {
        PyObject* i = PyNumber_Index(o);
        if (i == NULL) return 0;
        *out = PyLong_AsLongLong(i);
        Py_DECREF(i);
    }
    return !(*out == -1 && PyErr_Occurred());
}

static int as_int(PyObject* o, int* out) {
    int64_t v;
    if (!as_i64(o, &v)) return 0;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
        return 0;
    }
    *out = (int)v;
    return 1;
}

static int as_float(PyObject* o, float* out) {
    const double v = PyFloat_AsDouble(o);
    *out = (float)v;
    return !(v == -1.0 && PyErr_Occurred());
}

/* Arguments a[0..]: kinds 'i' int, 'q' int64, 'p' pointer, 'f' float into the
 * slots of the same index. */
typedef union {
    int i;
    int64_t q;
    void* p;
    float f;
} Slot;

static int parse(PyObject* const* a, Py_ssize_t n, const char* kinds, Slot* s) {
    const Py_ssize_t want = (Py_ssize_t)strlen(kinds);
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return 0;
    }
    for (Py_ssize_t k = 0; k < n; ++k) {
        int ok;
        switch (kinds[k]) {
            case 'i': ok = as_int(a[k], &s[k].i); break;
            case 'q': ok = as_i64(a[k], &s[k].q); break;
            case 'p': ok = as_ptr(a[k], &s[k].p); break;
            default: ok = as_float(a[k], &s[k].f); break;
        }
        if (!ok) return 0;
    }
    return 1;
}

/* Other threads run meanwhile: a launch may wait for a place in the queue. */
#define CALL_AND_RETURN(call)           \
    int status;                         \
    Py_BEGIN_ALLOW_THREADS              \
    status = (int)(call);               \
    Py_END_ALLOW_THREADS                \
    return PyLong_FromLong(status)

#define I(k) s[k].i
#define Q(k) s[k].q
#define P(k) s[k].p
#define F(k) s[k].f

static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Slot s[19];
    if (!parse(a, n, "iiqqqppfqpqpqqpqpqp", s)) return NULL;
    CALL_AND_RETURN(tern_rope(I(0), I(1), Q(2), Q(3), Q(4), P(5), P(6), F(7), Q(8), P(9), Q(10), P(11), Q(12),
                                     Q(13), P(14), Q(15), P(16), Q(17), P(18)));
}

static PyObject* py_kv_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Slot s[18];
    if (!parse(a, n, "iiqqqpqpqpqqpppppp", s)) return NULL;
    CALL_AND_RETURN(tern_kv_write(I(0), I(1), Q(2), Q(3), Q(4), P(5), Q(6), P(7), Q(8), P(9), Q(10), Q(11), P(12),
                                         P(13), P(14), P(15), P(16), P(17)));
}

static PyObject* py_rope_kv_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Slot s[28];
    if (!parse(a, n, "iiiqqqqqppfpqpqpqpqpqqpppppp", s)) return NULL;
    CALL_AND_RETURN(tern_rope_kv_write(I(0), I(1), I(2), Q(3), Q(4), Q(5), Q(6), Q(7), P(8), P(9), F(10), P(11),
                                              Q(12), P(13), Q(14), P(15), Q(16), P(17), Q(18), P(19), Q(20), Q(21),
                                              P(22), P(23), P(24), P(25), P(26), P(27)));
}

static PyObject* py_kv_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Slot s[17];
    if (!parse(a, n, "iiqqqpqqpppppqpqp", s)) return NULL;
    CALL_AND_RETURN(tern_kv_read(I(0), I(1), Q(2), Q(3), Q(4), P(5), Q(6), Q(7), P(8), P(9), P(10), P(11), P(12),
                                        Q(13), P(14), Q(15), P(16)));
}

static PyObject* py_attn_prompt(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Slot s[23];
    if (!parse(a, n, "iqppqqqqqifpqpqpqpqppqp", s)) return NULL;
    CALL_AND_RETURN(tern_attn_prompt(I(0), Q(1), P(2), P(3), Q(4), Q(5), Q(6), Q(7), Q(8), I(9), F(10), P(11),
                                            Q(12), P(13), Q(14), P(15), Q(16), P(17), Q(18), P(19), P(20),
                                            (size_t)Q(21), P(22)));
}

static PyObject* py_attn_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Slot s[24];
    if (!parse(a, n, "iiqqqqfpqqqpppppqppqppqp", s)) return NULL;
    CALL_AND_RETURN(tern_attn_decode(I(0), I(1), Q(2), Q(3), Q(4), Q(5), F(6), P(7), Q(8), Q(9), Q(10), P(11),
                                            P(12), P(13), P(14), P(15), Q(16), P(17), P(18), Q(19), P(20), P(21),
                                            (size_t)Q(22), P(23)));
}

#define CALL(name) {"tern_" #name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, "tern_" #name " of tern.h"}
static PyMethodDef g_methods[] = {CALL(rope),        CALL(kv_write),    CALL(rope_kv_write), CALL(kv_read),
                                  CALL(attn_prompt), CALL(attn_decode), {NULL, NULL, 0, NULL}};

static struct PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tern_python", "libtern's attention-side calls", -1, g_methods,
                                      NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tern_python(void) {
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (g_data_ptr == NULL) return NULL;
    return PyModule_Create(&g_module);
}
