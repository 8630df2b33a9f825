/* Calls of the C ABI from Python without ctypes: call(address, args...) for
 * functions whose arguments are integers and pointers and whose result is a
 * gemm_status_t.  An argument is an integer, None (NULL) or an object with a
 * data_ptr() method (a torch tensor).  The x86-64 calling convention passes
 * every such argument as one 64-bit word, of which a 32-bit parameter takes
 * the low half.  Against ctypes a call of twelve arguments, tensors among
 * them, takes 0.5 instead of 1.7 us (0.05 of it for letting other threads
 * run), which counts where a call is all there is (a decoder's few tokens). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

static PyObject *s_data_ptr;

/* 0 on success */
static int word(PyObject *o, uint64_t *out)
{
    PyObject *n;
    if (o == Py_None) {
        *out = 0;
        return 0;
    }
    if (PyLong_Check(o)) {
        *out = PyLong_AsUnsignedLongLongMask(o);
        return PyErr_Occurred() != NULL;
    }
    n = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!n) {
        if (!PyErr_ExceptionMatches(PyExc_AttributeError))
            return 1;
        PyErr_Clear();
        n = PyNumber_Index(o); /* raises TypeError for anything but an integer */
        if (!n)
            return 1;
    }
    *out = PyLong_AsUnsignedLongLongMask(n);
    Py_DECREF(n);
    return PyErr_Occurred() != NULL;
}

#define W1 uint64_t
#define W4 W1, W1, W1, W1
#define W8 W4, W4
#define A4(i) a[i], a[i + 1], a[i + 2], a[i + 3]
#define A8(i) A4(i), A4(i + 4)

static PyObject *call(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    uint64_t a[20] = {0};
    uintptr_t f;
    int r;
    Py_ssize_t i;
    (void)self;
    if (n < 1 || n > 21 || !PyLong_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "call(address, up to 20 arguments)");
        return NULL;
    }
    f = (uintptr_t)PyLong_AsUnsignedLongLongMask(args[0]);
    if (!f) {
        PyErr_SetString(PyExc_ValueError, "address is NULL");
        return NULL;
    }
    for (i = 1; i < n; ++i)
        if (word(args[i], &a[i - 1]))
            return NULL;
    /* A launch may wait (for room in a queue, for code to be loaded): other
     * threads run meanwhile.  The caller holds references to the arguments.
     * Words past a function's parameters are not read by it. */
    Py_BEGIN_ALLOW_THREADS
    if (n <= 9)
        r = ((int (*)(W8))f)(A8(0));
    else if (n <= 13)
        r = ((int (*)(W8, W4))f)(A8(0), A4(8));
    else
        r = ((int (*)(W8, W8, W4))f)(A8(0), A8(8), A4(16));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

static PyMethodDef methods[] = {
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(address, args...) -> status"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycall(void)
{
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    return s_data_ptr ? PyModule_Create(&module) : NULL;
}
