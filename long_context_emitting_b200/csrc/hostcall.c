/* Calls of the decode step's small entry points from Python, by the vectorcall
 * convention: plain numbers in, a status out.  Through ctypes the same call costs
 * 2.1 to 2.5 us of argument conversion, more than the launch itself; here it is a
 * few tenths of one.  The addresses come from the loaded libkascade.so (bind), so
 * this module links to nothing of it; a call before that raises. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/kascade.h"

enum { kNormRope, kWrite, kRead, kAnchor, kReuse, kCalls };
static void* g_fn[kCalls][2]; /* [call][half precision] */

/* Arguments as whole numbers, but for number `real`, which is read where it is used:
 * None is a null pointer, and the ones in `small` must fit 32 bits. */
static int numbers(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, Py_ssize_t real, unsigned long long small,
                   long long* v) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
    return -1;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (i == real) continue;
    v[i] = args[i] == Py_None ? 0 : PyLong_AsLongLong(args[i]);
    if (v[i] == -1 && PyErr_Occurred()) return -1;
    if (((small >> i) & 1) && (v[i] < INT32_MIN || v[i] > INT32_MAX)) {
      PyErr_Format(PyExc_OverflowError, "argument %zd does not fit 32 bits", i);
      return -1;
    }
  }
  return 0;
}

#define PTR(type, i) ((type*)(intptr_t)v[i])
#define STRIDES(i) ((kascade_strides){v[i], v[(i) + 1], v[(i) + 2]})
#define SHAPE(i) ((kascade_shape){(int32_t)v[i], (int32_t)v[(i) + 1], (int32_t)v[(i) + 2], (int32_t)v[(i) + 3]})
#define CALL(expr)                                                               \
  int rc;                                                                        \
  if (!fn) {                                                                     \
    PyErr_SetString(PyExc_RuntimeError, "no addresses yet: bind() comes first"); \
    return NULL;                                                                 \
  }                                                                              \
  Py_BEGIN_ALLOW_THREADS;                                                        \
  rc = (expr);                                                                   \
  Py_END_ALLOW_THREADS;                                                          \
  return PyLong_FromLong(rc)

/* f16, B, Hq, Hkv, d, N, q, 3 strides, k, 3 strides, positions, inv_freq, q_weight, k_weight, eps,
 * interleaved, q_out, 3 strides, k_out, 3 strides, stream */
static PyObject* norm_rope(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  long long v[29];
  if (numbers(args, n, 29, 18, 0x8003full, v)) return NULL;
  const double eps = PyFloat_AsDouble(args[18]);
  if (eps == -1.0 && PyErr_Occurred()) return NULL;
  int (*fn)(kascade_shape, int32_t, const uint16_t*, kascade_strides, const uint16_t*, kascade_strides, const int32_t*,
            const float*, const uint16_t*, const uint16_t*, float, int32_t, uint16_t*, kascade_strides, uint16_t*,
            kascade_strides, void*) = g_fn[kNormRope][v[0] != 0];
  CALL(fn(SHAPE(1), (int32_t)v[5], PTR(const uint16_t, 6), STRIDES(7), PTR(const uint16_t, 10), STRIDES(11),
          PTR(const int32_t, 14), PTR(const float, 15), PTR(const uint16_t, 16), PTR(const uint16_t, 17), (float)eps,
          (int32_t)v[19], PTR(uint16_t, 20), STRIDES(21), PTR(uint16_t, 24), STRIDES(25), PTR(void, 28)));
}

/* f16, B, Hq, Hkv, d, N, k, 3 strides, v, 3 strides, pages, num_pages, block_table, max_pages, page_size, start,
 * count, stream */
static PyObject* kv_write(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  long long v[22];
  if (numbers(args, n, 22, -1, 0x6803full, v)) return NULL;
  int (*fn)(kascade_shape, int32_t, const uint16_t*, kascade_strides, const uint16_t*, kascade_strides, uint8_t*, int32_t,
            const int32_t*, int32_t, int32_t, const int32_t*, const int32_t*, void*) = g_fn[kWrite][v[0] != 0];
  CALL(fn(SHAPE(1), (int32_t)v[5], PTR(const uint16_t, 6), STRIDES(7), PTR(const uint16_t, 10), STRIDES(11),
          PTR(uint8_t, 14), (int32_t)v[15], PTR(const int32_t, 16), (int32_t)v[17], (int32_t)v[18],
          PTR(const int32_t, 19), PTR(const int32_t, 20), PTR(void, 21)));
}

/* f16, B, Hq, Hkv, d, N, pages, num_pages, block_table, max_pages, page_size, start, count, k, v, stream */
static PyObject* kv_read(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  long long v[16];
  if (numbers(args, n, 16, -1, 0x6bfull, v)) return NULL;
  int (*fn)(kascade_shape, int32_t, const uint8_t*, int32_t, const int32_t*, int32_t, int32_t, const int32_t*,
            const int32_t*, uint16_t*, uint16_t*, void*) = g_fn[kRead][v[0] != 0];
  CALL(fn(SHAPE(1), (int32_t)v[5], PTR(const uint8_t, 6), (int32_t)v[7], PTR(const int32_t, 8), (int32_t)v[9],
          (int32_t)v[10], PTR(const int32_t, 11), PTR(const int32_t, 12), PTR(uint16_t, 13), PTR(uint16_t, 14),
          PTR(void, 15)));
}

/* f16, B, Hq, Hkv, d, q, pages, num_pages, block_table, max_pages, page_size, seq_len, max_T, scale, out, lse, pooled,
 * ld_pooled, ws, ws_bytes, stream */
static PyObject* decode_anchor(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  long long v[21];
  if (numbers(args, n, 21, 13, 0x169full, v)) return NULL;
  const double scale = PyFloat_AsDouble(args[13]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  int (*fn)(kascade_shape, const uint16_t*, const uint8_t*, int32_t, const int32_t*, int32_t, int32_t, const int32_t*,
            int32_t, float, uint16_t*, float*, float*, int64_t, void*, size_t, void*) = g_fn[kAnchor][v[0] != 0];
  CALL(fn(SHAPE(1), PTR(const uint16_t, 5), PTR(const uint8_t, 6), (int32_t)v[7], PTR(const int32_t, 8), (int32_t)v[9],
          (int32_t)v[10], PTR(const int32_t, 11), (int32_t)v[12], (float)scale, PTR(uint16_t, 14), PTR(float, 15),
          PTR(float, 16), v[17], PTR(void, 18), (size_t)v[19], PTR(void, 20)));
}

/* f16, B, Hq, Hkv, d, q, pages, num_pages, block_table, max_pages, page_size, seq_len, idx, idx_k, k_max, head_map,
 * scale, out, lse, stream */
static PyObject* decode_reuse(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  long long v[20];
  if (numbers(args, n, 20, 16, 0x469full, v)) return NULL;
  const double scale = PyFloat_AsDouble(args[16]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  int (*fn)(kascade_shape, const uint16_t*, const uint8_t*, int32_t, const int32_t*, int32_t, int32_t, const int32_t*,
            const int32_t*, const int32_t*, int32_t, const int32_t*, float, uint16_t*, float*, void*) =
      g_fn[kReuse][v[0] != 0];
  CALL(fn(SHAPE(1), PTR(const uint16_t, 5), PTR(const uint8_t, 6), (int32_t)v[7], PTR(const int32_t, 8), (int32_t)v[9],
          (int32_t)v[10], PTR(const int32_t, 11), PTR(const int32_t, 12), PTR(const int32_t, 13), (int32_t)v[14],
          PTR(const int32_t, 15), (float)scale, PTR(uint16_t, 17), PTR(float, 18), PTR(void, 19)));
}

/* bind(addresses): bfloat16 and half entry point of each call, in the order of the enum. */
static PyObject* bind(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  long long v[2 * kCalls];
  if (numbers(args, n, 2 * kCalls, -1, 0, v)) return NULL;
  for (int i = 0; i < 2 * kCalls; ++i) {
    if (!v[i]) {
      PyErr_SetString(PyExc_ValueError, "null address");
      return NULL;
    }
    g_fn[i / 2][i % 2] = (void*)(intptr_t)v[i];
  }
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(bind),          METHOD(norm_rope),    METHOD(kv_write), METHOD(kv_read),
                                METHOD(decode_anchor), METHOD(decode_reuse), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hostcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__hostcall(void) { return PyModule_Create(&module); }
