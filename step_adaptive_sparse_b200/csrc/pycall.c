/* The key/value cache's calls of libarea for CPython: arguments straight into
 * the C functions.  Their calls are short (a token's attention is 6 us on the GPU), so
 * that the time to marshal some 20 arguments counts: a token's call takes the host
 * 3.5 us, 2.9 of them the launch, and its workspace's size 0.2 us; through ctypes
 * 5.8 and 1.6.
 *
 * The functions' addresses come from the library that the binding has loaded
 * (bind).  Pointer arguments: None, an int address, or an object with
 * data_ptr(); the stream: None, an int, or an object with cuda_stream.  A call returns
 * its status, a size call the bytes or -status. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <string.h>

enum { SINK_WS, SINK, PREFIX_WS, PREFIX, CACHE_WS, CACHE, EVICT, FUNCTIONS };
static void *fn[FUNCTIONS];
static PyObject *s_data_ptr, *s_cuda_stream;

static int address_of(PyObject *x, void **out) {
  *out = PyLong_AsVoidPtr(x);
  return *out || !PyErr_Occurred();
}
static int pointer(PyObject *x, void **out) {
  if (x == Py_None) {
    *out = NULL;
    return 1;
  }
  if (PyLong_Check(x)) return address_of(x, out);
  PyObject *p = PyObject_CallMethodNoArgs(x, s_data_ptr);
  if (!p) return 0;
  const int ok = address_of(p, out);
  Py_DECREF(p);
  return ok;
}
static int stream(PyObject *x, void **out) {
  if (x == Py_None) {
    *out = NULL;
    return 1;
  }
  if (PyLong_Check(x)) return address_of(x, out);
  PyObject *p = PyObject_GetAttr(x, s_cuda_stream);
  if (!p) return 0;
  const int ok = address_of(p, out);
  Py_DECREF(p);
  return ok;
}
static int integer(PyObject *x, int *out) {
  const long v = PyLong_AsLong(x);
  if (v == -1 && PyErr_Occurred()) return 0;
  if (v < INT_MIN || v > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument outside a C int");
    return 0;
  }
  *out = (int)v;
  return 1;
}
static int size(PyObject *x, size_t *out) {
  const long long v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) return 0;
  if (v < 0) {
    PyErr_SetString(PyExc_OverflowError, "negative size");
    return 0;
  }
  *out = (size_t)v;
  return 1;
}

/* Arguments by a signature: P pointer, Z size, I int, F float, S stream. */
struct args {
  void *p[10];
  size_t z;
  int i[10];
  float f;
};
static int parse(int which, const char *sig, PyObject *const *a, Py_ssize_t n, struct args *out) {
  int np = 0, ni = 0;
  if (!fn[which]) {
    PyErr_SetString(PyExc_RuntimeError, "function not bound");
    return 0;
  }
  if ((size_t)n != strlen(sig)) {
    PyErr_Format(PyExc_TypeError, "%zu arguments expected, %zd given", strlen(sig), n);
    return 0;
  }
  for (Py_ssize_t k = 0; k < n; ++k) {
    int ok;
    switch (sig[k]) {
      case 'P': ok = pointer(a[k], &out->p[np++]); break;
      case 'S': ok = stream(a[k], &out->p[np++]); break;
      case 'Z': ok = size(a[k], &out->z); break;
      case 'I': ok = integer(a[k], &out->i[ni++]); break;
      default: {
        const double v = PyFloat_AsDouble(a[k]);
        ok = !(v == -1.0 && PyErr_Occurred());
        out->f = (float)v;
      }
    }
    if (!ok) return 0;
  }
  return 1;
}

#define STATUS(call)                 \
  int st;                            \
  Py_BEGIN_ALLOW_THREADS st = call;  \
  Py_END_ALLOW_THREADS return PyLong_FromLong(st)
#define BYTES(call)                  \
  size_t b = 0;                      \
  const int st = call;               \
  return st ? PyLong_FromLong(-st) : PyLong_FromSize_t(b)
#define P(k) x.p[k]
#define I(k) x.i[k]
typedef void *V;

static PyObject *sink_ws(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  struct args x;
  if (!parse(SINK_WS, "IIIIIIIII", a, n, &x)) return NULL;
  BYTES(((int (*)(int, int, int, int, int, int, int, int, int, size_t *))fn[SINK_WS])(
      I(0), I(1), I(2), I(3), I(4), I(5), I(6), I(7), I(8), &b));
}
static PyObject *prefix_ws(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  struct args x;
  if (!parse(PREFIX_WS, "IIIIIIII", a, n, &x)) return NULL;
  BYTES(((int (*)(int, int, int, int, int, int, int, int, size_t *))fn[PREFIX_WS])(
      I(0), I(1), I(2), I(3), I(4), I(5), I(6), I(7), &b));
}
static PyObject *cache_ws(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  struct args x;
  if (!parse(CACHE_WS, "IIIIIII", a, n, &x)) return NULL;
  BYTES(((int (*)(int, int, int, int, int, int, int, size_t *))fn[CACHE_WS])(
      I(0), I(1), I(2), I(3), I(4), I(5), I(6), &b));
}
static PyObject *sink(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  struct args x;
  if (!parse(SINK, "PPPPPPZIIIIIIIIFIS", a, n, &x)) return NULL;
  STATUS(((int (*)(V, V, V, V, V, V, size_t, int, int, int, int, int, int, int, int, float, int, V))
              fn[SINK])(P(0), P(1), P(2), P(3), P(4), P(5), x.z, I(0), I(1), I(2), I(3), I(4), I(5),
                        I(6), I(7), x.f, I(8), P(6)));
}
static PyObject *prefix(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  struct args x;
  if (!parse(PREFIX, "PPPPPPPPZIIIIIIIIFIS", a, n, &x)) return NULL;
  STATUS(((int (*)(V, V, V, V, V, V, V, V, size_t, int, int, int, int, int, int, int, int, float, int,
                   V))fn[PREFIX])(P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), x.z, I(0), I(1),
                                  I(2), I(3), I(4), I(5), I(6), I(7), x.f, I(8), P(8)));
}
static PyObject *cache(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  struct args x;
  if (!parse(CACHE, "PPPPPPPPZIIIIIIFIS", a, n, &x)) return NULL;
  STATUS(((int (*)(V, V, V, V, V, V, V, V, size_t, int, int, int, int, int, int, float, int, V))
              fn[CACHE])(P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), x.z, I(0), I(1), I(2), I(3),
                         I(4), I(5), x.f, I(6), P(8)));
}
static PyObject *evict(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  struct args x;
  if (!parse(EVICT, "PPPPPPPPPIIIIIIIIIS", a, n, &x)) return NULL;
  STATUS(((int (*)(V, V, V, V, V, V, V, V, V, int, int, int, int, int, int, int, int, int, V))
              fn[EVICT])(P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), P(8), I(0), I(1), I(2), I(3),
                         I(4), I(5), I(6), I(7), I(8), P(9)));
}

static const char *const names[FUNCTIONS] = {
    "area_sink_attn_ws_bytes",  "area_sink_attn",  "area_prefix_attn_ws_bytes", "area_prefix_attn",
    "area_cache_attn_ws_bytes", "area_cache_attn", "area_cache_evict"};
static PyObject *bind(PyObject *m, PyObject *args) {
  const char *name;
  PyObject *at;
  void *p;
  if (!PyArg_ParseTuple(args, "sO", &name, &at) || !address_of(at, &p)) return NULL;
  for (int k = 0; k < FUNCTIONS; ++k)
    if (!strcmp(name, names[k])) {
      fn[k] = p;
      Py_RETURN_NONE;
    }
  PyErr_SetString(PyExc_ValueError, name);
  return NULL;
}

#define FAST(f) (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL
static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(name, address) of a function of libarea"},
    {"area_sink_attn_ws_bytes", FAST(sink_ws)},     {"area_sink_attn", FAST(sink)},
    {"area_prefix_attn_ws_bytes", FAST(prefix_ws)}, {"area_prefix_attn", FAST(prefix)},
    {"area_cache_attn_ws_bytes", FAST(cache_ws)},   {"area_cache_attn", FAST(cache)},
    {"area_cache_evict", FAST(evict)},              {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_areacall", NULL, -1, methods};

PyMODINIT_FUNC PyInit__areacall(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  PyObject *m = PyModule_Create(&module);
  PyObject *all = m ? PyTuple_New(FUNCTIONS) : NULL;
  if (!all || !s_data_ptr || !s_cuda_stream) return NULL;
  for (int k = 0; k < FUNCTIONS; ++k) PyTuple_SET_ITEM(all, k, PyUnicode_FromString(names[k]));
  if (PyModule_AddObject(m, "FUNCTIONS", all) < 0) return NULL;
  return m;
}
