/* CPython module of the sequence operators' binding: one call checks the
 * tensors of a library call, writes its argument struct and makes it. The
 * same in Python took longer than a single token's kernel.
 *
 *   call(entry, stream, device, head, item, kind, shape, dtype, item, ...) -> int
 *
 * entry: the address of a conv_status (const void* args, void* stream)
 * function; device: the CUDA device that all tensors have to be on; head: the
 * first bytes of the struct; then four values for each further field of it, in
 * order. Returns the call's status (>= 0), or -1 - i where item i is not the
 * tensor that its kind, shape and dtype ask for, or is on another device (the
 * library is not called then).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

enum {
  DENSE = 0,        /* a contiguous tensor or None: its pointer */
  VIEW = 1,         /* [n, l, c], c contiguous, or None: pointer, strides of n and l */
  TOKEN = 2,        /* [n, c], c contiguous, or None: pointer, stride of n, 0 */
  GROUPS = 3,       /* [n, l, g, s], g and s dense, or None: as VIEW */
  TOKEN_GROUPS = 4, /* [n, g, s], g and s dense: as TOKEN */
  WORKSPACE = 5,    /* a contiguous tensor of any shape and type, or None: pointer, bytes */
  NUMBER = 6        /* an int */
};

enum { MAX_BYTES = 1024, MAX_DIMS = 8 };

static PyObject *s_dtype, *s_shape, *s_get_device, *s_stride, *s_data_ptr, *s_nbytes;

/* The ints of a tuple; their count, or -1. */
static int read_ints(PyObject* t, int64_t* v) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) > MAX_DIMS) return -1;
  const int n = (int)PyTuple_GET_SIZE(t);
  for (int i = 0; i < n; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (v[i] == -1 && PyErr_Occurred()) return -1;
  }
  return n;
}

/* The tensor's CUDA device (-1: it is not on one), or -2 with a Python error. */
static long device_of(PyObject* t) {
  PyObject* o = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!o) return -2;
  const long v = PyLong_AsLong(o);
  Py_DECREF(o);
  return v == -1 && PyErr_Occurred() ? -2 : v;
}

/* The tensor's shape and strides; the number of dimensions, or -1. */
static int layout(PyObject* t, int64_t* size, int64_t* stride) {
  PyObject* o = PyObject_GetAttr(t, s_shape);
  if (!o) return -1;
  const int n = read_ints(o, size);
  Py_DECREF(o);
  if (n < 0) return -1;
  o = PyObject_CallMethodNoArgs(t, s_stride);
  if (!o) return -1;
  const int m = read_ints(o, stride);
  Py_DECREF(o);
  return m == n ? n : -1;
}

static int64_t long_of(PyObject* o) {
  if (!o) return -1;
  const int64_t v = (int64_t)PyLong_AsUnsignedLongLong(o);
  Py_DECREF(o);
  return v;
}

/* Whether dimensions d .. n-1 are dense, with the last one's stride 1. */
static int dense_from(int d, int n, const int64_t* size, const int64_t* stride) {
  int64_t at = 1;
  for (int i = n - 1; i >= d; --i) {
    if (size[i] == 0) return 1;
    if (size[i] != 1 && stride[i] != at) return 0;
    at *= size[i];
  }
  return 1;
}

/* One item into `to`: the bytes written; 0 where it is not what is asked for;
 * -1 with a Python error. */
static int put(PyObject* t, long device, long kind, PyObject* shape, PyObject* dtype, uint8_t* to) {
  int64_t out[3] = {0, 0, 0};
  const int bytes = kind == DENSE || kind == NUMBER ? 8 : kind == WORKSPACE ? 16 : 24;
  if (kind == NUMBER) {
    out[0] = PyLong_AsLongLong(t);
    if (out[0] == -1 && PyErr_Occurred()) return -1;
  } else if (t != Py_None) {
    int64_t size[MAX_DIMS], stride[MAX_DIMS], want[MAX_DIMS];
    const long on = device_of(t);
    if (on == -2) return -1;
    if (on != device) return 0;
    const int n = layout(t, size, stride);
    if (n < 0) return PyErr_Occurred() ? -1 : 0;
    if (kind == WORKSPACE) {
      if (!dense_from(0, n, size, stride)) return 0;
      out[1] = long_of(PyObject_GetAttr(t, s_nbytes));
    } else {
      PyObject* d = PyObject_GetAttr(t, s_dtype);
      if (!d) return -1;
      const int same = d == dtype;
      Py_DECREF(d);
      if (!same) return 0;
      const int m = read_ints(shape, want);
      if (m < 0) return PyErr_Occurred() ? -1 : 0;
      if (m != n || memcmp(size, want, sizeof(int64_t) * (size_t)n) != 0) return 0;
      int lead = 0; /* dimensions whose strides are free */
      if (kind == VIEW || kind == GROUPS) lead = 2;
      if (kind == TOKEN || kind == TOKEN_GROUPS) lead = 1;
      if (n < lead + 1 && kind != DENSE) return 0;
      if (!dense_from(lead, n, size, stride)) return 0;
      if (lead > 0) out[1] = stride[0];
      if (lead > 1) out[2] = stride[1];
    }
    out[0] = long_of(PyObject_CallMethodNoArgs(t, s_data_ptr));
    if (PyErr_Occurred()) return -1;
  }
  memcpy(to, out, (size_t)bytes);
  return bytes;
}

static PyObject* seq_call(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  enum { FIRST = 4 }; /* of the items */
  if (n < FIRST || (n - FIRST) % 4 != 0 || !PyBytes_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "call(entry, stream, device, head, item, kind, shape, dtype, ...)");
    return NULL;
  }
  union {
    uint8_t bytes[MAX_BYTES];
    int64_t align;
  } buf;
  void* entry = PyLong_AsVoidPtr(args[0]);
  void* stream = PyLong_AsVoidPtr(args[1]);
  const long device = PyLong_AsLong(args[2]);
  if (PyErr_Occurred()) return NULL;
  Py_ssize_t at = PyBytes_GET_SIZE(args[3]);
  if (at > MAX_BYTES) at = MAX_BYTES + 1;
  else memcpy(buf.bytes, PyBytes_AS_STRING(args[3]), (size_t)at);
  for (Py_ssize_t i = FIRST; i < n; i += 4) {
    if (at + 24 > MAX_BYTES) {
      PyErr_SetString(PyExc_ValueError, "call: too many arguments");
      return NULL;
    }
    const long kind = PyLong_AsLong(args[i + 1]);
    if (kind == -1 && PyErr_Occurred()) return NULL;
    const int wrote = put(args[i], device, kind, args[i + 2], args[i + 3], buf.bytes + at);
    if (wrote < 0) return NULL;
    if (wrote == 0) return PyLong_FromLong(-1 - (long)((i - FIRST) / 4));
    at += wrote;
  }
  int (*fn)(const void*, void*);
  memcpy(&fn, &entry, sizeof fn);
  /* The launch may wait for room in the stream's queue, and what runs before
   * it for the interpreter (a host function of the caller's). */
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fn(buf.bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

static PyMethodDef methods[] = {
    {"call", (PyCFunction)(void (*)(void))seq_call, METH_FASTCALL, "Checks the items, packs them after head and calls entry."},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "seqcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_seqcall(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  if (!s_dtype || !s_shape || !s_get_device || !s_stride || !s_data_ptr || !s_nbytes) return NULL;
  return PyModule_Create(&module);
}
