/* The Python binding's checks and calls of the serving operators, as a CPython
 * extension: a decode step makes several calls a layer, and checking four
 * tensors and making the call takes 9 us in Python, of which the launch is 2.
 *
 * Each function takes the values that the method of the same name in bgtq.py
 * was given, checks them as that method does, and makes the library call.  It
 * returns the call's status, or None where anything is not as expected (the
 * method then goes its own way through the same checks and says what is wrong).
 * Nothing is kept from one call to the next but what a context holds: a
 * cache's device, types and sizes. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <string.h>

#include "../../include/bgtq.h"

typedef struct {
  PyObject *device, *rows, *i32, *f32; /* torch.device, torch.dtype */
  long index;                          /* the device's */
  long hkv, hq, width, pages;
  void* scratch;
} Ctx;

static const char kCtx[] = "bgtq.marshal";
static PyObject *s_dtype, *s_device, *s_shape, *s_is_contiguous, *s_data_ptr, *s_stride, *s_index, *s_type, *s_cuda;
static PyObject *g_stream, *g_device; /* torch._C's current raw stream of a device, current device */

static void free_ctx(PyObject* cap) {
  Ctx* c = PyCapsule_GetPointer(cap, kCtx);
  if (c == NULL) return;
  Py_XDECREF(c->device);
  Py_XDECREF(c->rows);
  Py_XDECREF(c->i32);
  Py_XDECREF(c->f32);
  PyMem_Free(c);
}

/* context(device, index, rows, i32, f32, hkv, hq, width, pages, scratch) */
static PyObject* context(PyObject* self, PyObject* args) {
  PyObject *device, *rows, *i32, *f32;
  long index, hkv, hq, width, pages;
  unsigned long long scratch;
  if (!PyArg_ParseTuple(args, "OlOOOllllK", &device, &index, &rows, &i32, &f32, &hkv, &hq, &width, &pages, &scratch))
    return NULL;
  Ctx* c = PyMem_Malloc(sizeof(Ctx));
  if (c == NULL) return PyErr_NoMemory();
  Py_INCREF(device);
  Py_INCREF(rows);
  Py_INCREF(i32);
  Py_INCREF(f32);
  c->device = device;
  c->rows = rows;
  c->i32 = i32;
  c->f32 = f32;
  c->index = index;
  c->hkv = hkv;
  c->hq = hq;
  c->width = width;
  c->pages = pages;
  c->scratch = (void*)(uintptr_t)scratch;
  PyObject* cap = PyCapsule_New(c, kCtx, free_ctx);
  if (cap == NULL) {
    Py_DECREF(device);
    Py_DECREF(rows);
    Py_DECREF(i32);
    Py_DECREF(f32);
    PyMem_Free(c);
  }
  return cap;
}

static PyObject* not_here(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

/* A tuple's integers into out[n]; 0 on success. */
static int sizes(PyObject* t, int n, int64_t* out) {
  if (t == NULL || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) != n) return -1;
  for (int i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return 0;
}

static int attr_is(PyObject* t, PyObject* name, PyObject* want) {
  PyObject* x = PyObject_GetAttr(t, name);
  if (x == NULL) return 0;
  const int same = x == want || PyObject_RichCompareBool(x, want, Py_EQ) == 1;
  Py_DECREF(x);
  return same;
}

static int shape_of(PyObject* t, int n, int64_t* out) {
  PyObject* x = PyObject_GetAttr(t, s_shape);
  const int r = sizes(x, n, out);
  Py_XDECREF(x);
  return r;
}

static int pointer_of(PyObject* t, void** out) {
  PyObject* x = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (x == NULL) return -1;
  *out = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* t: a contiguous tensor of dtype on device with n dims (shape: -1 any extent,
 * replaced by what it is); its address in out. */
static int tensor(PyObject* t, PyObject* dtype, PyObject* device, int n, int64_t* shape, void** out) {
  int64_t have[5];
  if (!attr_is(t, s_dtype, dtype) || !attr_is(t, s_device, device) || shape_of(t, n, have)) return -1;
  for (int i = 0; i < n; ++i) {
    if (shape[i] >= 0 && shape[i] != have[i]) return -1;
    shape[i] = have[i];
    if (have[i] > INT32_MAX) return -1;
  }
  PyObject* x = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (x == NULL) return -1;
  Py_DECREF(x);
  if (x != Py_True) return -1;
  return pointer_of(t, out);
}

static int row_tensor(const Ctx* c, PyObject* t, int64_t n, void** out) {
  int64_t s[1] = {n};
  return tensor(t, c->i32, c->device, 1, s, out);
}

static int table_tensor(const Ctx* c, PyObject* t, int64_t batch, void** out) {
  int64_t s[2] = {batch, c->width};
  return tensor(t, c->i32, c->device, 2, s, out);
}

/* An int argument that fits an int32. */
static int int_arg(PyObject* x, int32_t* out) {
  if (!PyLong_Check(x)) return -1;
  const long v = PyLong_AsLong(x);
  if ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX) return -1;
  *out = (int32_t)v;
  return 0;
}

static int state_arg(PyObject* x, bgtq_state** out) {
  if (!PyLong_Check(x)) return -1;
  *out = PyLong_AsVoidPtr(x);
  return *out == NULL ? -1 : 0;
}

static int stream_of(PyObject* index, void** out) {
  PyObject* x = PyObject_CallOneArg(g_stream, index);
  if (x == NULL) return -1;
  *out = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

static int stream_at(long index, void** out) {
  PyObject* i = PyLong_FromLong(index);
  if (i == NULL) return -1;
  const int r = stream_of(i, out);
  Py_DECREF(i);
  return r;
}

/* The library call, other threads running meanwhile: a launch waits where the
 * queue of launches is full. */
#define RELEASED(call)       \
  do {                       \
    Py_BEGIN_ALLOW_THREADS   \
    status = (call);         \
    Py_END_ALLOW_THREADS     \
  } while (0)

static const Ctx* ctx_arg(PyObject* x) { return PyCapsule_GetPointer(x, kCtx); }

/* append(ctx, state, layer, layer_count, k, v, start, count) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int status;
  bgtq_state* st;
  int32_t layer, layers;
  void *k, *v, *start, *count, *stream;
  if (n != 8) return not_here();
  const Ctx* c = ctx_arg(a[0]);
  if (c == NULL || state_arg(a[1], &st) || int_arg(a[2], &layer) || int_arg(a[3], &layers)) return not_here();
  int64_t s[5] = {layers, -1, -1, c->hkv, 128};
  if (tensor(a[4], c->rows, c->device, 5, s, &k) || tensor(a[5], c->rows, c->device, 5, s, &v) ||
      row_tensor(c, a[6], s[1], &start) || row_tensor(c, a[7], s[1], &count) || stream_at(c->index, &stream))
    return not_here();
  RELEASED(bgtq_byte_append(st, layer, layers, k, v, start, count, (int32_t)s[1], (int32_t)s[2], stream));
  return PyLong_FromLong(status);
}

/* decode_attn(ctx, state, layer, layer_count, q, seq_lens, out, scale, softcap, slopes, window, prefix, doc_start) */
static PyObject* decode_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int status;
  bgtq_state* st;
  int32_t layer, layers;
  void *q, *lens, *out, *slopes = NULL, *prefix = NULL, *docs = NULL, *stream;
  if (n != 13) return not_here();
  const Ctx* c = ctx_arg(a[0]);
  if (c == NULL || state_arg(a[1], &st) || int_arg(a[2], &layer) || int_arg(a[3], &layers)) return not_here();
  int64_t s[5] = {layers, -1, -1, c->hq, 128};
  if (tensor(a[4], c->rows, c->device, 5, s, &q) || tensor(a[6], c->rows, c->device, 5, s, &out) ||
      row_tensor(c, a[5], s[1], &lens))
    return not_here();
  bgtq_score score;
  memset(&score, 0, sizeof(score));
  if (a[7] != Py_None) {
    score.scale = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred() || !(score.scale > 0)) return not_here();
  }
  score.softcap = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred() || int_arg(a[10], &score.window)) return not_here();
  int64_t heads[1] = {c->hq}, per_query[2] = {s[1], s[2]};
  if ((a[9] != Py_None && tensor(a[9], c->f32, c->device, 1, heads, &slopes)) ||
      (a[11] != Py_None && row_tensor(c, a[11], s[1], &prefix)) ||
      (a[12] != Py_None && tensor(a[12], c->i32, c->device, 2, per_query, &docs)) || stream_at(c->index, &stream))
    return not_here();
  score.d_slopes = slopes;
  score.d_prefix = prefix;
  score.d_doc_start = docs;
  RELEASED(bgtq_byte_decode_attn(st, layer, layers, q, lens, (int32_t)s[1], (int32_t)s[2], &score, out, stream));
  return PyLong_FromLong(status);
}

/* copy_pages(ctx, state, src, dst) */
static PyObject* copy_pages(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int status;
  bgtq_state* st;
  void *src, *dst, *stream;
  int64_t s[1] = {-1};
  if (n != 4) return not_here();
  const Ctx* c = ctx_arg(a[0]);
  if (c == NULL || state_arg(a[1], &st) || tensor(a[2], c->i32, c->device, 1, s, &src) ||
      tensor(a[3], c->i32, c->device, 1, s, &dst) || stream_at(c->index, &stream))
    return not_here();
  if (s[0] == 0) return PyLong_FromLong(0);
  RELEASED(bgtq_copy_pages(st, src, dst, (int32_t)s[0], stream));
  return PyLong_FromLong(status);
}

/* fork_sequences(ctx, state, parent, table, refs, lens, table_out, refs_out, lens_out) */
static PyObject* fork_sequences(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int status;
  bgtq_state* st;
  void *parent, *table, *refs, *lens, *table_out, *refs_out, *lens_out, *stream;
  int64_t s[1] = {-1};
  if (n != 9) return not_here();
  const Ctx* c = ctx_arg(a[0]);
  if (c == NULL || state_arg(a[1], &st) || tensor(a[2], c->i32, c->device, 1, s, &parent) ||
      table_tensor(c, a[3], s[0], &table) || row_tensor(c, a[4], c->pages, &refs) || row_tensor(c, a[5], s[0], &lens) ||
      table_tensor(c, a[6], s[0], &table_out) || row_tensor(c, a[7], c->pages, &refs_out) ||
      row_tensor(c, a[8], s[0], &lens_out) || stream_at(c->index, &stream))
    return not_here();
  RELEASED(bgtq_fork_sequences(st, parent, table, refs, lens, (int32_t)s[0], table_out, refs_out, lens_out, c->scratch, stream));
  return PyLong_FromLong(status);
}

/* resize_sequences(ctx, state, table, refs, lens, new_lens, lens_out) */
static PyObject* resize_sequences(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int status;
  bgtq_state* st;
  void *table, *refs, *lens, *new_lens, *lens_out, *stream;
  int64_t s[1] = {-1};
  if (n != 7) return not_here();
  const Ctx* c = ctx_arg(a[0]);
  if (c == NULL || state_arg(a[1], &st) || tensor(a[4], c->i32, c->device, 1, s, &lens) ||
      table_tensor(c, a[2], s[0], &table) || row_tensor(c, a[3], c->pages, &refs) ||
      row_tensor(c, a[5], s[0], &new_lens) || row_tensor(c, a[6], s[0], &lens_out) || stream_at(c->index, &stream))
    return not_here();
  RELEASED(bgtq_resize_sequences(st, table, refs, lens, new_lens, (int32_t)s[0], lens_out, c->scratch, stream));
  return PyLong_FromLong(status);
}

/* compact_pages(ctx, state, table, refs, lens, table_out, refs_out, page_map, n_live) */
static PyObject* compact_pages(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int status;
  bgtq_state* st;
  void *table, *refs, *lens, *table_out, *refs_out, *map, *live, *stream;
  int64_t s[1] = {-1};
  if (n != 9) return not_here();
  const Ctx* c = ctx_arg(a[0]);
  if (c == NULL || state_arg(a[1], &st) || tensor(a[4], c->i32, c->device, 1, s, &lens) ||
      table_tensor(c, a[2], s[0], &table) || row_tensor(c, a[3], c->pages, &refs) ||
      table_tensor(c, a[5], s[0], &table_out) || row_tensor(c, a[6], c->pages, &refs_out) ||
      row_tensor(c, a[7], c->pages, &map) || row_tensor(c, a[8], 1, &live) || stream_at(c->index, &stream))
    return not_here();
  RELEASED(bgtq_compact_pages(st, table, refs, lens, (int32_t)s[0], table_out, refs_out, map, live, c->scratch, stream));
  return PyLong_FromLong(status);
}

/* Rows [tokens, heads, 128], heads contiguous: address and elements from a
 * token to the next. */
static int rope_rows(PyObject* t, PyObject* dtype, PyObject* device, int64_t* tokens, int64_t* heads, int32_t* stride,
                     void** out) {
  int64_t s[3], st[3];
  if (!attr_is(t, s_dtype, dtype) || !attr_is(t, s_device, device) || shape_of(t, 3, s)) return -1;
  PyObject* x = PyObject_CallMethodNoArgs(t, s_stride);
  const int bad = sizes(x, 3, st);
  Py_XDECREF(x);
  if (bad || s[2] != 128 || st[2] != 1 || (s[1] > 1 && st[1] != 128)) return -1;
  if ((*tokens >= 0 && s[0] != *tokens) || (*heads >= 0 && s[1] != *heads)) return -1;
  *tokens = s[0];
  *heads = s[1];
  if (s[0] <= 1) st[0] = s[1] * 128; /* there is no next token */
  if (s[0] > INT32_MAX || s[1] > INT32_MAX / 128 || st[0] > INT32_MAX || st[0] < 0) return -1;
  *stride = (int32_t)st[0];
  return pointer_of(t, out);
}

/* rope_axes(half, bfloat, i32, q, k, pos, axis, base, q_out, k_out, pairing); q or k and its output None */
static PyObject* rope_axes(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) return not_here();
  PyObject* one = a[3] != Py_None ? a[3] : a[4];
  if (one == Py_None || (a[3] == Py_None) != (a[8] == Py_None) || (a[4] == Py_None) != (a[9] == Py_None)) return not_here();
  bgtq_rope_config cfg;
  memset(&cfg, 0, sizeof(cfg));
  int64_t tokens = -1, hq = -1, hk = -1;
  int32_t sq = 0, sk = 0, sqo = 0, sko = 0;
  void *q = NULL, *k = NULL, *q_out = NULL, *k_out = NULL, *pos, *stream;
  PyObject* axis = NULL;
  PyObject* result = NULL;
  PyObject* dtype = PyObject_GetAttr(one, s_dtype);
  PyObject* device = PyObject_GetAttr(one, s_device);
  PyObject *index = NULL, *now = NULL;
  if (dtype == NULL || device == NULL || (dtype != a[0] && dtype != a[1])) goto done;
  if (!attr_is(device, s_type, s_cuda)) goto done;
  index = PyObject_GetAttr(device, s_index);
  now = PyObject_CallNoArgs(g_device);
  if (index == NULL || now == NULL || PyObject_RichCompareBool(index, now, Py_EQ) != 1) goto done;
  if (a[3] != Py_None && (rope_rows(a[3], dtype, device, &tokens, &hq, &sq, &q) ||
                          rope_rows(a[8], dtype, device, &tokens, &hq, &sqo, &q_out)))
    goto done;
  if (a[4] != Py_None && (rope_rows(a[4], dtype, device, &tokens, &hk, &sk, &k) ||
                          rope_rows(a[9], dtype, device, &tokens, &hk, &sko, &k_out)))
    goto done;
  int64_t ps[2] = {-1, tokens};
  if (tensor(a[5], a[2], device, 2, ps, &pos)) goto done;
  axis = PySequence_Fast(a[6], "axis");
  if (axis == NULL || PySequence_Fast_GET_SIZE(axis) != 64) goto done;
  for (int i = 0; i < 64; ++i) {
    PyObject* x = PySequence_Fast_GET_ITEM(axis, i);
    const long v = PyLong_Check(x) ? PyLong_AsLong(x) : -1;
    if (v < 0 || v > 255) goto done;
    cfg.axis[i] = (uint8_t)v;
  }
  cfg.base = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred() || int_arg(a[10], &cfg.pairing) || stream_of(index, &stream)) goto done;
  cfg.n_q_heads = hq < 0 ? 0 : (int32_t)hq;
  cfg.n_kv_heads = hk < 0 ? 0 : (int32_t)hk;
  cfg.head_dim = 128;
  cfg.dtype = dtype == a[1] ? BGTQ_DTYPE_BFLOAT : BGTQ_DTYPE_HALF;
  cfg.n_axes = (int32_t)ps[0];
  int status = 0;
  if (tokens != 0) RELEASED(bgtq_rope_axes(&cfg, q, sq, k, sk, pos, (int32_t)tokens, q_out, sqo, k_out, sko, stream));
  result = PyLong_FromLong(status);
done:
  Py_XDECREF(axis);
  Py_XDECREF(dtype);
  Py_XDECREF(device);
  Py_XDECREF(index);
  Py_XDECREF(now);
  return result != NULL ? result : not_here();
}

static PyMethodDef methods[] = {
    {"context", context, METH_VARARGS, NULL},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
    {"decode_attn", (PyCFunction)(void (*)(void))decode_attn, METH_FASTCALL, NULL},
    {"copy_pages", (PyCFunction)(void (*)(void))copy_pages, METH_FASTCALL, NULL},
    {"fork_sequences", (PyCFunction)(void (*)(void))fork_sequences, METH_FASTCALL, NULL},
    {"resize_sequences", (PyCFunction)(void (*)(void))resize_sequences, METH_FASTCALL, NULL},
    {"compact_pages", (PyCFunction)(void (*)(void))compact_pages, METH_FASTCALL, NULL},
    {"rope_axes", (PyCFunction)(void (*)(void))rope_axes, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_device = PyUnicode_InternFromString("device");
  s_shape = PyUnicode_InternFromString("shape");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_index = PyUnicode_InternFromString("index");
  s_type = PyUnicode_InternFromString("type");
  s_cuda = PyUnicode_InternFromString("cuda");
  PyObject* c = PyImport_ImportModule("torch._C");
  if (c == NULL) return NULL;
  g_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  g_device = PyObject_GetAttrString(c, "_cuda_getDevice");
  Py_DECREF(c);
  if (g_stream == NULL || g_device == NULL) return NULL;
  return PyModule_Create(&module);
}
