// CPython entries for the per-call public functions fd_decode_attn,
// fd_decode_attn_ex, fd_decode_attn_fp8 and fd_decode_attn_fp8_ex, and for those
// of the paged cache that a decode step calls: argument
// marshalling only (device addresses, the plan's host address and sizes as
// Python integers in, the library's status code out). They save the
// generic ctypes conversion on the host path of every call; the package falls
// back to ctypes when this module was not built.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "fd_decode_attn.h"
#include "fd_paged_attn.h"

static PyObject* py_decode_attn(PyObject* self, PyObject* args) {
  unsigned long long q, k, v, out, lens, stream;
  int B, NH, NKV, HS, capacity, window;
  double scale;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKKKiiiiiidK", &q, &k, &v, &out, &lens, &B, &NH, &NKV, &HS, &capacity, &window,
                        &scale, &stream))
    return NULL;
  const int rc = fd_decode_attn((const void*)(uintptr_t)q, (const void*)(uintptr_t)k, (const void*)(uintptr_t)v,
                                (void*)(uintptr_t)out, (const int*)(uintptr_t)lens, B, NH, NKV, HS, capacity, window,
                                (float)scale, (fd_stream_t)(uintptr_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* py_decode_attn_fp8(PyObject* self, PyObject* args) {
  unsigned long long q, k8, v8, ks, vs, out, lens, stream;
  int B, NH, NKV, HS, capacity, window;
  double scale;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKKKKKiiiiiidK", &q, &k8, &v8, &ks, &vs, &out, &lens, &B, &NH, &NKV, &HS, &capacity,
                        &window, &scale, &stream))
    return NULL;
  const int rc = fd_decode_attn_fp8((const void*)(uintptr_t)q, (const void*)(uintptr_t)k8, (const void*)(uintptr_t)v8,
                                    (const float*)(uintptr_t)ks, (const float*)(uintptr_t)vs, (void*)(uintptr_t)out,
                                    (const int*)(uintptr_t)lens, B, NH, NKV, HS, capacity, window, (float)scale,
                                    (fd_stream_t)(uintptr_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* py_decode_attn_ex(PyObject* self, PyObject* args) {
  unsigned long long plan, ws, ws_bytes, out32, q, k, v, out, lens, stream;
  int B, NH, NKV, HS, capacity, window;
  double scale;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKKKKKKKiiiiiidK", &plan, &ws, &ws_bytes, &out32, &q, &k, &v, &out, &lens, &B, &NH,
                        &NKV, &HS, &capacity, &window, &scale, &stream))
    return NULL;
  const int rc = fd_decode_attn_ex((const fd_plan_t*)(uintptr_t)plan, (void*)(uintptr_t)ws, (size_t)ws_bytes,
                                   (float*)(uintptr_t)out32, (const void*)(uintptr_t)q, (const void*)(uintptr_t)k,
                                   (const void*)(uintptr_t)v, (void*)(uintptr_t)out, (const int*)(uintptr_t)lens, B, NH,
                                   NKV, HS, capacity, window, (float)scale, (fd_stream_t)(uintptr_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* py_decode_attn_fp8_ex(PyObject* self, PyObject* args) {
  unsigned long long plan, ws, ws_bytes, out32, q, k8, v8, ks, vs, out, lens, stream;
  int B, NH, NKV, HS, capacity, window;
  double scale;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKKKKKKKKKiiiiiidK", &plan, &ws, &ws_bytes, &out32, &q, &k8, &v8, &ks, &vs, &out,
                        &lens, &B, &NH, &NKV, &HS, &capacity, &window, &scale, &stream))
    return NULL;
  const int rc = fd_decode_attn_fp8_ex(
      (const fd_plan_t*)(uintptr_t)plan, (void*)(uintptr_t)ws, (size_t)ws_bytes, (float*)(uintptr_t)out32,
      (const void*)(uintptr_t)q, (const void*)(uintptr_t)k8, (const void*)(uintptr_t)v8, (const float*)(uintptr_t)ks,
      (const float*)(uintptr_t)vs, (void*)(uintptr_t)out, (const int*)(uintptr_t)lens, B, NH, NKV, HS, capacity,
      window, (float)scale, (fd_stream_t)(uintptr_t)stream);
  return PyLong_FromLong(rc);
}

// The paged cache's entries take tensors (whose data_ptr() is called here),
// addresses or None where the C function takes a pointer. An array of
// `kinds`, one letter an argument: p pointer, i int, l long long, z size_t,
// f float.
typedef union {
  void* p;
  int i;
  long long l;
  size_t z;
  float f;
} Arg;

static PyObject* g_data_ptr;

static int parse(PyObject* const* args, Py_ssize_t nargs, const char* kinds, Arg* out) {
  const Py_ssize_t want = (Py_ssize_t)strlen(kinds);
  if (nargs != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, nargs);
    return 0;
  }
  for (Py_ssize_t k = 0; k < want; ++k) {
    PyObject* o = args[k];
    switch (kinds[k]) {
      case 'p':
        if (o == Py_None) {
          out[k].p = NULL;
        } else if (PyLong_Check(o)) {
          out[k].p = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(o);
        } else {
          PyObject* a = PyObject_CallMethodNoArgs(o, g_data_ptr);
          if (!a) return 0;
          out[k].p = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(a);
          Py_DECREF(a);
        }
        break;
      case 'i': {
        const long v = PyLong_AsLong(o);
        if (v != (long)(int)v) {
          PyErr_SetString(PyExc_OverflowError, "argument does not fit an int");
          return 0;
        }
        out[k].i = (int)v;
        break;
      }
      case 'l': out[k].l = PyLong_AsLongLong(o); break;
      case 'z': out[k].z = (size_t)PyLong_AsUnsignedLongLong(o); break;
      default: out[k].f = (float)PyFloat_AsDouble(o); break;
    }
    if (PyErr_Occurred()) return 0;
  }
  return 1;
}

static PyObject* py_paged_attn(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[19];
  (void)self;
  if (!parse(args, n, "ppppppppiiiiiiiifip", a)) return NULL;
  return PyLong_FromLong(fd_paged_attn(a[0].p, a[1].p, a[2].p, a[3].p, a[4].p, a[5].p, a[6].p, a[7].p, a[8].i, a[9].i,
                                       a[10].i, a[11].i, a[12].i, a[13].i, a[14].i, a[15].i, a[16].f, a[17].i,
                                       (fd_stream_t)a[18].p));
}

static PyObject* py_paged_attn_ex(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[22];
  (void)self;
  if (!parse(args, n, "ppzpppppppppiiiiiiiifp", a)) return NULL;
  return PyLong_FromLong(fd_paged_attn_ex((const fd_paged_plan_t*)a[0].p, a[1].p, a[2].z, a[3].p, a[4].p, a[5].p,
                                          a[6].p, a[7].p, a[8].p, a[9].p, a[10].p, a[11].p, a[12].i, a[13].i, a[14].i,
                                          a[15].i, a[16].i, a[17].i, a[18].i, a[19].i, a[20].f,
                                          (fd_stream_t)a[21].p));
}

static PyObject* py_paged_append(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[21];
  (void)self;
  if (!parse(args, n, "ppppppppppiiiiiiillip", a)) return NULL;
  return PyLong_FromLong(fd_paged_append(a[0].p, a[1].p, a[2].p, a[3].p, a[4].p, a[5].p, a[6].p, a[7].p, a[8].p, a[9].p,
                                         a[10].i, a[11].i, a[12].i, a[13].i, a[14].i, a[15].i, a[16].i, a[17].l,
                                         a[18].l, a[19].i, (fd_stream_t)a[20].p));
}

static PyObject* py_pages_reserve(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[13];
  (void)self;
  if (!parse(args, n, "pppppppziiiip", a)) return NULL;
  return PyLong_FromLong(fd_pages_reserve(a[0].p, a[1].p, a[2].p, a[3].p, a[4].p, a[5].p, a[6].p, a[7].z, a[8].i,
                                          a[9].i, a[10].i, a[11].i, (fd_stream_t)a[12].p));
}

static PyObject* py_pages_fork(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[11];
  (void)self;
  if (!parse(args, n, "ppppppiiiip", a)) return NULL;
  return PyLong_FromLong(fd_pages_fork(a[0].p, a[1].p, a[2].p, a[3].p, a[4].p, a[5].p, a[6].i, a[7].i, a[8].i, a[9].i,
                                       (fd_stream_t)a[10].p));
}

static PyObject* py_pages_free(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[10];
  (void)self;
  if (!parse(args, n, "ppppiiiiip", a)) return NULL;
  return PyLong_FromLong(fd_pages_free(a[0].p, a[1].p, a[2].p, a[3].p, a[4].i, a[5].i, a[6].i, a[7].i, a[8].i,
                                       (fd_stream_t)a[9].p));
}

static PyObject* py_pages_compact(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[9];
  (void)self;
  if (!parse(args, n, "ppppziiip", a)) return NULL;
  return PyLong_FromLong(fd_pages_compact(a[0].p, a[1].p, a[2].p, a[3].p, a[4].z, a[5].i, a[6].i, a[7].i,
                                          (fd_stream_t)a[8].p));
}

static PyObject* py_pages_copy(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[13];
  (void)self;
  if (!parse(args, n, "pppppiiiiiiip", a)) return NULL;
  return PyLong_FromLong(fd_pages_copy(a[0].p, a[1].p, a[2].p, a[3].p, a[4].p, a[5].i, a[6].i, a[7].i, a[8].i, a[9].i,
                                       a[10].i, a[11].i, (fd_stream_t)a[12].p));
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, "fd_" name "; returns the status code"}

static PyMethodDef kMethods[] = {
    FAST("paged_attn", py_paged_attn),
    FAST("paged_attn_ex", py_paged_attn_ex),
    FAST("paged_append", py_paged_append),
    FAST("pages_reserve", py_pages_reserve),
    FAST("pages_fork", py_pages_fork),
    FAST("pages_free", py_pages_free),
    FAST("pages_compact", py_pages_compact),
    FAST("pages_copy", py_pages_copy),
    {"decode_attn_ex", py_decode_attn_ex, METH_VARARGS, "fd_decode_attn_ex; returns the status code"},
    {"decode_attn_fp8_ex", py_decode_attn_fp8_ex, METH_VARARGS, "fd_decode_attn_fp8_ex; returns the status code"},
    {"decode_attn", py_decode_attn, METH_VARARGS, "fd_decode_attn; returns the status code"},
    {"decode_attn_fp8", py_decode_attn_fp8, METH_VARARGS, "fd_decode_attn_fp8; returns the status code"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fdfast", NULL, -1, kMethods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fdfast(void) {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  return g_data_ptr ? PyModule_Create(&kModule) : NULL;
}
