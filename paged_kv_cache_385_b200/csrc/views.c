/* _views.pack: the pa_tensor views of a call's torch tensors, filled in one pass through the CPython API.
 *
 * The binding's calls take six to nine tensors. Reading a tensor's pointer, dtype, shape and strides
 * and packing them takes 0.9 to 1.3 us a tensor in Python, for a call more than a small kernel takes on the GPU;
 * here it takes 0.3 (a 64-token rope call 10.5 us of host time for 16.9, a commit 9.1 for 15.5). No torch header is used: the tensors are read through their public methods. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "pa.h"

static PyObject *s_data_ptr, *s_get_device, *s_dtype, *s_shape, *s_stride;

/* Sizes or strides (a tuple of ints) into out[4]: how many, or -1 (with a Python error unless they are
 * more than four). */
static int read_ints(PyObject* seq, int64_t* out) {
  if (!PyTuple_Check(seq)) {
    PyErr_SetString(PyExc_TypeError, "shape and stride must be tuples");
    return -1;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(seq);
  if (n > 4) return -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

/* One tensor's view: 1 done, 0 not a tensor the library takes (no Python error), -1 Python error. */
static int read_tensor(PyObject* t, PyObject* codes, long device, pa_tensor* out) {
  PyObject* x = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!x) return -1;
  const long on = PyLong_AsLong(x);
  Py_DECREF(x);
  if (on == -1 && PyErr_Occurred()) return -1;
  if (on != device) return 0;
  x = PyObject_GetAttr(t, s_dtype);
  if (!x) return -1;
  PyObject* code = PyDict_GetItemWithError(codes, x); /* borrowed */
  Py_DECREF(x);
  if (!code) return PyErr_Occurred() ? -1 : 0;
  out->dtype = (int32_t)PyLong_AsLong(code);
  x = PyObject_GetAttr(t, s_shape);
  if (!x) return -1;
  out->ndim = read_ints(x, out->shape);
  Py_DECREF(x);
  if (out->ndim < 0) return PyErr_Occurred() ? -1 : 0;
  x = PyObject_CallMethodNoArgs(t, s_stride);
  if (!x) return -1;
  const int n = read_ints(x, out->stride);
  Py_DECREF(x);
  if (n < 0) return PyErr_Occurred() ? -1 : 0;
  x = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!x) return -1;
  out->data = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return PyErr_Occurred() ? -1 : 1;
}

/* pack(tensors, codes, device) -> (buffer, addresses), or the index of the first tensor that is not one of
 * the dtypes in codes on that device with at most four dimensions. None in tensors gives None. The
 * addresses are valid while the buffer lives. */
static PyObject* pack(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 3 || !PyTuple_Check(args[0]) || !PyDict_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "pack(tensors: tuple, codes: dict, device: int)");
    return NULL;
  }
  const long device = PyLong_AsLong(args[2]);
  if (device == -1 && PyErr_Occurred()) return NULL;
  const Py_ssize_t n = PyTuple_GET_SIZE(args[0]);
  PyObject* buffer = PyBytes_FromStringAndSize(NULL, n * (Py_ssize_t)sizeof(pa_tensor));
  PyObject* refs = PyTuple_New(n);
  PyObject* done = NULL;
  if (!buffer || !refs) goto out;
  pa_tensor* views = (pa_tensor*)PyBytes_AS_STRING(buffer);
  memset(views, 0, (size_t)n * sizeof(pa_tensor));
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* t = PyTuple_GET_ITEM(args[0], i);
    PyObject* ref;
    if (t == Py_None) {
      Py_INCREF(Py_None);
      ref = Py_None;
    } else {
      const int r = read_tensor(t, args[1], device, &views[i]);
      if (r < 0) goto out;
      if (r == 0) {
        done = PyLong_FromSsize_t(i);
        goto out;
      }
      ref = PyLong_FromVoidPtr(&views[i]);
      if (!ref) goto out;
    }
    PyTuple_SET_ITEM(refs, i, ref);
  }
  done = PyTuple_Pack(2, buffer, refs);
out:
  Py_XDECREF(buffer);
  Py_XDECREF(refs);
  return done;
}

static PyMethodDef methods[] = {
    {"pack", (PyCFunction)(void (*)(void))pack, METH_FASTCALL, "pack(tensors, codes, device) -> (buffer, addresses) or index"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_views", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__views(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  if (!s_data_ptr || !s_get_device || !s_dtype || !s_shape || !s_stride) return NULL;
  return PyModule_Create(&module);
}
