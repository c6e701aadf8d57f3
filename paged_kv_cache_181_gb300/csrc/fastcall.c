/* The serving calls' argument marshalling in C (a CPython extension over the C ABI).
 *
 * A decode step makes an append and an attention call per layer, each a few microseconds of GPU time; through ctypes a
 * call took 8 to 10 us of host time, more than the kernels.  The functions here check that the tensors are what the
 * call takes and make it: 4 to 6 us.  Where anything is not as it should be they return None without having done
 * anything, and the binding's careful path (_lib.py) runs instead: it raises the error, or takes the rarer forms (no
 * q, no rotation).  Otherwise they return the call's status.
 *
 * Only documented methods and attributes of the tensors are used (data_ptr, get_device, is_contiguous, dtype, shape,
 * stride), so nothing here depends on the build of torch.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "pagedkv.h"

static PyObject *s_data_ptr, *s_get_device, *s_is_contiguous, *s_dtype, *s_shape, *s_stride, *s_cuda_stream, *s_nbytes;
static PyObject *dt_code[3], *dt_u8, *dt_i32, *dt_i64; /* dt_code: by pkv_dtype */
static PyObject *current_device, *raw_stream, *scratch;

typedef struct {
  PyObject* shape; /* new reference */
  PyObject* dtype; /* new reference */
  void* ptr;
} Tensor;

static void drop(Tensor* t, int n) {
  for (int i = 0; i < n; ++i) {
    Py_XDECREF(t[i].shape);
    Py_XDECREF(t[i].dtype);
  }
}

static int method_long(PyObject* o, PyObject* name, long long* v) {
  PyObject* r = PyObject_CallMethodNoArgs(o, name);
  if (!r) return 0;
  *v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return !(*v == -1 && PyErr_Occurred());
}

/* Shape, type and address of a tensor on device `dev`; contiguous unless `strided`. */
static int load(PyObject* o, long long dev, int strided, Tensor* t) {
  long long d, p;
  t->shape = t->dtype = NULL;
  if (!method_long(o, s_get_device, &d) || d != dev) return 0;
  if (!strided) {
    PyObject* r = PyObject_CallMethodNoArgs(o, s_is_contiguous);
    if (!r) return 0;
    Py_DECREF(r);
    if (r != Py_True) return 0;
  }
  t->shape = PyObject_GetAttr(o, s_shape);
  t->dtype = PyObject_GetAttr(o, s_dtype);
  if (!t->shape || !t->dtype || !PyTuple_Check(t->shape) || !method_long(o, s_data_ptr, &p)) return 0;
  t->ptr = (void*)(intptr_t)p;
  return 1;
}

static int rank_of(const Tensor* t) { return (int)PyTuple_GET_SIZE(t->shape); }
static long long dim(const Tensor* t, int i) { return PyLong_AsLongLong(PyTuple_GET_ITEM(t->shape, i)); }
static int is_vector(const Tensor* t, long long n) { return rank_of(t) == 1 && dim(t, 0) == n; }
static int same_shape(const Tensor* a, const Tensor* b) {
  const int n = rank_of(a);
  if (rank_of(b) != n) return 0;
  for (int i = 0; i < n; ++i)
    if (dim(a, i) != dim(b, i)) return 0;
  return 1;
}
static int code_of(PyObject* dtype) {
  for (int i = 0; i < 3; ++i)
    if (dtype == dt_code[i]) return i;
  return -1;
}

/* Elements between the tokens of x [T, H, D] with contiguous heads and channels; -1: it has not. */
static long long token_stride(PyObject* o, const Tensor* t) {
  const long long T = dim(t, 0), h = dim(t, 1), d = dim(t, 2);
  PyObject* r = PyObject_CallMethodNoArgs(o, s_stride);
  long long st = -1;
  if (r && PyTuple_Check(r) && PyTuple_GET_SIZE(r) == 3) {
    const long long s0 = PyLong_AsLongLong(PyTuple_GET_ITEM(r, 0)), s1 = PyLong_AsLongLong(PyTuple_GET_ITEM(r, 1));
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(r, 2)) == 1 && (s1 == d || h <= 1)) st = T > 1 ? s0 : h * d;
  }
  Py_XDECREF(r);
  return st;
}

/* A plain int (no bool, no float) that fits 32 bits. */
static int as_int(PyObject* o, int* v) {
  if (!PyLong_CheckExact(o)) return 0;
  const long long x = PyLong_AsLongLong(o);
  *v = (int)x;
  return x == *v && !(x == -1 && PyErr_Occurred());
}

static int stream_of(PyObject* o, PyObject* dev, void** s) {
  PyObject* r = o == Py_None ? PyObject_CallOneArg(raw_stream, dev) : PyObject_GetAttr(o, s_cuda_stream);
  if (!r) return 0;
  const long long x = PyLong_AsLongLong(r);
  Py_DECREF(r);
  *s = (void*)(intptr_t)x;
  return !(x == -1 && PyErr_Occurred());
}

static PyObject* decline(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

/* attend(q4, q, key_pool, value_pool, block_table, query_start_loc, seq_lens, max_query_len, max_seq_len, scale, window,
 *        sinks, out, workspace, flags, block_size, stream) */
static PyObject* attend(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 17 || !raw_stream) return decline();
  const int q4 = a[0] == Py_True;
  PyObject* devo = PyObject_CallNoArgs(current_device);
  if (!devo) return decline();
  const long long dev = PyLong_AsLongLong(devo);
  Tensor t[8]; /* q, key_pool, value_pool, block_table, query_start_loc, seq_lens, out, workspace */
  PyObject* const objs[8] = {a[1], a[2], a[3], a[4], a[5], a[6], a[12], a[13]};
  const int count = a[13] == Py_None ? 7 : 8;
  int loaded = 0, status = -1;
  PyObject* owned = NULL; /* a workspace of this call */
  for (; loaded < count; ++loaded)
    if (!load(objs[loaded], dev, 0, &t[loaded])) {
      ++loaded;
      goto done;
    }
  {
    int mq, ml, window, sinks, flags, bs;
    if (!as_int(a[7], &mq) || !as_int(a[8], &ml) || !as_int(a[10], &window) || !as_int(a[11], &sinks) ||
        !as_int(a[14], &flags) || !as_int(a[15], &bs))
      goto done;
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) goto done;
    const int code = code_of(t[0].dtype);
    if (code < 0 || rank_of(&t[0]) != 3 || rank_of(&t[1]) != 3 || rank_of(&t[3]) != 2 || !same_shape(&t[0], &t[6]) ||
        !same_shape(&t[1], &t[2]) || t[6].dtype != t[0].dtype || bs != 16)
      goto done;
    PyObject* pool = q4 ? dt_u8 : t[0].dtype;
    if (t[1].dtype != pool || t[2].dtype != pool || t[3].dtype != dt_i32 || t[4].dtype != dt_i32 || t[5].dtype != dt_i32)
      goto done;
    const long long Tq = dim(&t[0], 0), hq = dim(&t[0], 1), d = dim(&t[0], 2), hkv = dim(&t[1], 1), B = dim(&t[3], 0),
                    W = dim(&t[3], 1);
    long long blocks = dim(&t[1], 0);
    if (dim(&t[1], 2) != (q4 ? 10 * d : d) || (!q4 && blocks % 16) || !is_vector(&t[4], B + 1) || !is_vector(&t[5], B) ||
        hq > INT32_MAX || hkv > INT32_MAX || d > INT32_MAX || B > INT32_MAX || W > INT32_MAX)
      goto done;
    if (!q4) blocks /= 16;
    void* ws = NULL;
    long long ws_bytes = 0;
    if (count == 8) {
      PyObject* r = PyObject_GetAttr(a[13], s_nbytes);
      if (!r) goto done;
      ws_bytes = PyLong_AsLongLong(r);
      Py_DECREF(r);
      if (ws_bytes < 0) goto done;
      ws = t[7].ptr;
    } else if (B * hkv < 256 && code && ml > 1024 && (window > 1024 || window == 0)) {
      /* Few sequences and heads over many keys: no other sizes take a workspace. */
      ws_bytes = (long long)paged_attn_window_workspace_size(blocks, (int)hq, (int)hkv, (int)d, (pkv_dtype)code, q4,
                                                             (int)B, mq, ml, window, sinks);
      if (ws_bytes) {
        PyObject* size = scratch ? PyLong_FromLongLong(ws_bytes) : NULL;
        long long at;
        if (!size) goto done;
        owned = PyObject_CallFunctionObjArgs(scratch, size, a[1], a[16], NULL);
        Py_DECREF(size);
        if (!owned || !method_long(owned, s_data_ptr, &at)) goto done;
        ws = (void*)(intptr_t)at;
      }
    }
    void* stream;
    if (!stream_of(a[16], devo, &stream)) goto done;
    status = (q4 ? paged_attn_q4 : paged_attn_window)(
        t[0].ptr, Tq, (int)hq, t[1].ptr, t[2].ptr, blocks, bs, (int)hkv, (int)d, (pkv_dtype)code, (const int32_t*)t[3].ptr,
        (int)B, (int)W, (const int32_t*)t[4].ptr, (const int32_t*)t[5].ptr, mq, ml, (float)scale, window, sinks, t[6].ptr,
        ws, (size_t)ws_bytes, (uint32_t)flags, stream);
  }
done:
  drop(t, loaded);
  Py_DECREF(devo);
  Py_XDECREF(owned); /* torch's allocator keeps the memory for this stream's order */
  return status < 0 ? decline() : PyLong_FromLong(status);
}

/* append(q4, q, k, v, positions, cos_sin, slot_mapping, key_pool, value_pool, interleaved, q_out, flags, stream) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 13 || !raw_stream || a[1] == Py_None || a[5] == Py_None || a[10] == Py_None) return decline();
  const int q4 = a[0] == Py_True;
  PyObject* devo = PyObject_CallNoArgs(current_device);
  if (!devo) return decline();
  const long long dev = PyLong_AsLongLong(devo);
  Tensor t[9]; /* q, k, v, positions, cos_sin, slot_mapping, key_pool, value_pool, q_out */
  PyObject* const objs[9] = {a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[10]};
  int loaded = 0, status = -1;
  for (; loaded < 9; ++loaded)
    if (!load(objs[loaded], dev, loaded < 3, &t[loaded])) {
      ++loaded;
      goto done;
    }
  {
    int flags;
    if (!as_int(a[11], &flags)) goto done;
    const int inter = PyObject_IsTrue(a[9]);
    const int code = code_of(t[1].dtype);
    if (inter < 0 || code < 0 || rank_of(&t[0]) != 3 || rank_of(&t[1]) != 3 || rank_of(&t[4]) != 2 || rank_of(&t[6]) != 3 ||
        !same_shape(&t[1], &t[2]) || !same_shape(&t[6], &t[7]) || !same_shape(&t[0], &t[8]))
      goto done;
    PyObject* pool = q4 ? dt_u8 : t[1].dtype;
    if (t[0].dtype != t[1].dtype || t[2].dtype != t[1].dtype || t[8].dtype != t[1].dtype || t[6].dtype != pool ||
        t[7].dtype != pool || t[3].dtype != dt_i32 || t[4].dtype != dt_code[PKV_F32] || t[5].dtype != dt_i64)
      goto done;
    const long long T = dim(&t[1], 0), hkv = dim(&t[1], 1), d = dim(&t[1], 2), hq = dim(&t[0], 1), rot = dim(&t[4], 1);
    if (dim(&t[0], 0) != T || dim(&t[0], 2) != d || dim(&t[6], 1) != hkv || dim(&t[6], 2) != (q4 ? 10 * d : d) ||
        !is_vector(&t[3], T) || !is_vector(&t[5], T) || rot <= 0 || rot > INT32_MAX || hq > INT32_MAX || hkv > INT32_MAX ||
        d > INT32_MAX)
      goto done;
    const long long qs = token_stride(a[1], &t[0]), ks = token_stride(a[2], &t[1]), vs = token_stride(a[3], &t[2]);
    void* stream;
    if (qs < 0 || ks < 0 || vs < 0 || !stream_of(a[12], devo, &stream)) goto done;
    status = (q4 ? paged_kv_append_q4 : paged_kv_append)(
        t[0].ptr, qs, t[1].ptr, ks, t[2].ptr, vs, (const int32_t*)t[3].ptr, (const float*)t[4].ptr, dim(&t[4], 0), (int)rot,
        (const int64_t*)t[5].ptr, T, (int)hq, t[8].ptr, t[6].ptr, t[7].ptr, dim(&t[6], 0), (int)hkv, (int)d,
        (pkv_dtype)code, (uint32_t)flags | (inter ? PKV_ROPE_INTERLEAVED : 0u), stream);
  }
done:
  drop(t, loaded);
  Py_DECREF(devo);
  return status < 0 ? decline() : PyLong_FromLong(status);
}

/* gather(key_pool, value_pool, block_table, stage_k, stage_v, first_block, n_blocks or None, flags, stream) */
static PyObject* gather(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 9 || !raw_stream) return decline();
  PyObject* devo = PyObject_CallNoArgs(current_device);
  if (!devo) return decline();
  const long long dev = PyLong_AsLongLong(devo);
  Tensor t[5];
  int loaded = 0, status = -1;
  for (; loaded < 5; ++loaded)
    if (!load(a[loaded], dev, 0, &t[loaded])) {
      ++loaded;
      goto done;
    }
  {
    int first, blocks = 0, flags;
    if (!as_int(a[5], &first) || !as_int(a[7], &flags) || (a[6] != Py_None && !as_int(a[6], &blocks))) goto done;
    const int code = code_of(t[3].dtype);
    if (code < 0 || rank_of(&t[0]) != 3 || rank_of(&t[2]) != 2 || rank_of(&t[3]) != 4 || !same_shape(&t[0], &t[1]) ||
        !same_shape(&t[3], &t[4]) || t[4].dtype != t[3].dtype || t[0].dtype != dt_u8 || t[1].dtype != dt_u8 ||
        t[2].dtype != dt_i32)
      goto done;
    const long long B = dim(&t[2], 0), W = dim(&t[2], 1), hkv = dim(&t[3], 2), d = dim(&t[3], 3);
    if (dim(&t[3], 0) != B || dim(&t[0], 1) != hkv || dim(&t[0], 2) != 10 * d || B > INT32_MAX || W > INT32_MAX ||
        hkv > INT32_MAX || d > INT32_MAX)
      goto done;
    if (a[6] == Py_None) blocks = (int)(W - first);
    void* stream;
    if (!stream_of(a[8], devo, &stream)) goto done;
    status = paged_kv_gather_q4(t[0].ptr, t[1].ptr, dim(&t[0], 0), (const int32_t*)t[2].ptr, (int)B, (int)W, first, blocks,
                                t[3].ptr, t[4].ptr, dim(&t[3], 1), (int)hkv, (int)d, (pkv_dtype)code, (uint32_t)flags,
                                stream);
  }
done:
  drop(t, loaded);
  Py_DECREF(devo);
  return status < 0 ? decline() : PyLong_FromLong(status);
}

/* setup((f32, bf16, f16), uint8, int32, int64, current_device, raw_stream[, scratch]) */
static PyObject* setup(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *f32, *bf16, *f16, *u8, *i32, *i64, *cur, *raw, *mem = NULL;
  if (!PyArg_ParseTuple(args, "(OOO)OOOOO|O", &f32, &bf16, &f16, &u8, &i32, &i64, &cur, &raw, &mem)) return NULL;
  PyObject* const v[8] = {f32, bf16, f16, u8, i32, i64, cur, raw};
  PyObject** const to[8] = {&dt_code[PKV_F32], &dt_code[PKV_BF16], &dt_code[PKV_F16], &dt_u8, &dt_i32, &dt_i64,
                            &current_device, &raw_stream};
  for (int i = 0; i < 8; ++i) {
    Py_INCREF(v[i]);
    Py_XSETREF(*to[i], v[i]);
  }
  Py_XINCREF(mem);
  Py_XSETREF(scratch, mem);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, "paged_attn_window / paged_attn_q4"},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, "paged_kv_append / paged_kv_append_q4"},
    {"gather", (PyCFunction)(void (*)(void))gather, METH_FASTCALL, "paged_kv_gather_q4"},
    {"setup", setup, METH_VARARGS, "dtypes, torch's device and stream queries, and the workspace allocation"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
  static const char* const names[8] = {"data_ptr", "get_device", "is_contiguous", "dtype",
                                       "shape",    "stride",     "cuda_stream",   "nbytes"};
  PyObject** const to[8] = {&s_data_ptr, &s_get_device, &s_is_contiguous, &s_dtype,
                            &s_shape,    &s_stride,     &s_cuda_stream,   &s_nbytes};
  for (int i = 0; i < 8; ++i)
    if (!(*to[i] = PyUnicode_InternFromString(names[i]))) return NULL;
  return PyModule_Create(&module);
}
