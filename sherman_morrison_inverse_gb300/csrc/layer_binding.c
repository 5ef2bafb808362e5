/* Argument checks and marshalling for Python of the state space layer's operators, and of the products and
 * layer norms around them.
 *
 * A decoding step of one sequence runs for a few microseconds on the GPU; checking a dozen tensors
 * and passing them through ctypes takes ten times that.  This module does the same work with the
 * CPython API: it reads each tensor's public attributes (shape, dtype, get_device(), stride(),
 * data_ptr()), checks them, allocates outputs through torch and calls the C entry points, whose
 * addresses layer.py hands over, without the interpreter's lock: a launch waits where the device's queue
 * is full.  It holds nothing from one call for the next.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "vla.h"

typedef vla_err_t (*conv_fn)(vla_handle_t, const void*, const float*, const float*, void*, void*, long long,
                             long long, long long, const int*, const int*, long long, long long, int,
                             const long long*, int, vla_dtype_t, void*);
typedef vla_err_t (*scan_fn)(vla_handle_t, const void*, const void*, const float*, const void*, const void*,
                             const float*, const void*, const float*, float*, void*, long long, long long,
                             long long, const int*, const int*, long long, long long, long long, long long,
                             long long, const long long*, int, vla_dtype_t, void*, size_t, void*);
typedef vla_err_t (*ws_fn)(vla_handle_t, long long, long long, long long, int, long long, long long, long long,
                           vla_dtype_t, size_t*);
typedef vla_err_t (*norm_fn)(vla_handle_t, const void*, const float*, void*, void*, float*, long long, long long,
                             long long, long long, long long, float, int, vla_out_t, vla_dtype_t, vla_dtype_t,
                             void*);

typedef vla_err_t (*linear_fn)(vla_handle_t, const void*, const void*, const float*, const float*, const float*,
                               const void*, void*, void*, long long, long long, long long, const long long*, vla_act_t,
                               vla_mat_t, vla_dtype_t, void*, size_t, void*);
typedef vla_err_t (*linear_ws_fn)(vla_handle_t, const void*, const void*, long long, long long, long long,
                                  const long long*, vla_mat_t, vla_dtype_t, size_t*);
typedef vla_err_t (*linear_back_fn)(vla_handle_t, const void*, const void*, const void*, const void*, void*, void*,
                                    float*, long long, long long, long long, const long long*, vla_act_t, vla_dtype_t,
                                    void*, size_t, void*);
typedef vla_err_t (*linear_back_ws_fn)(vla_handle_t, const void*, const void*, const void*, int, int, int, long long,
                                       long long, long long, const long long*, vla_act_t, vla_dtype_t, size_t*);
typedef vla_err_t (*lnorm_fn)(vla_handle_t, const void*, const float*, const float*, void*, void*, float*, long long,
                              long long, long long, long long, long long, float, vla_dtype_t, vla_dtype_t, void*);
typedef vla_err_t (*lnorm_back_fn)(vla_handle_t, const void*, const void*, const float*, const float*, const void*, void*,
                                   float*, float*, long long, long long, const long long*, vla_dtype_t, vla_dtype_t,
                                   void*, size_t, void*);
typedef vla_err_t (*lnorm_back_ws_fn)(vla_handle_t, long long, long long, size_t*);

static conv_fn f_conv;
static scan_fn f_scan;
static ws_fn f_ws;
static norm_fn f_norm;
static linear_fn f_linear;
static linear_ws_fn f_linear_ws;
static linear_back_fn f_linear_back;
static linear_back_ws_fn f_linear_back_ws;
static lnorm_fn f_lnorm;
static lnorm_back_fn f_lnorm_back;
static lnorm_back_ws_fn f_lnorm_back_ws;
static PyObject *c_new, *t_u8, *s_device, *k_new;                 /* torch.empty; names of its dtype and device */
static PyObject *c_grad, *s_requires;                             /* torch.is_grad_enabled, and what it is asked for */
static PyObject *c_strided, *c_at, *c_modes;                      /* see read_allocator; None where torch has them not */
static PyObject *t_f32, *t_bf16, *t_i32, *t_e4m3, *t_i8;          /* torch dtypes */
static PyObject *c_like, *c_dense, *c_empty, *c_bytes, *c_stream; /* allocators and the current stream */
static PyObject *s_shape, *s_dtype, *s_get_device, *s_stride, *s_data_ptr, *s_ptr, *s_index, *s_fail, *k_dtype;

enum { MAXD = 8 };
typedef struct {
  PyObject* obj;
  const char* name;
  int nd;
  long long shape[MAXD], stride[MAXD];
  void* ptr;
} Tensor;

enum { DENSE = 0, PACKED = 1, TOKEN = 2 };   /* [S, T, ...], [tokens, ...] with offsets, [S, ...] */

static int read_ints(PyObject* tuple, long long* out, int most, int* n) {
  if (!tuple) return -1;
  Py_ssize_t size = PyTuple_Check(tuple) ? PyTuple_GET_SIZE(tuple) : -1;
  if (size < 0 || size > most) {
    Py_DECREF(tuple);
    PyErr_SetString(PyExc_ValueError, "tensors of at most 8 dimensions are supported");
    return -1;
  }
  for (Py_ssize_t i = 0; i < size; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
  Py_DECREF(tuple);
  *n = (int)size;
  return PyErr_Occurred() ? -1 : 0;
}

static PyObject* call0(PyObject* self, PyObject* method) {
  PyObject* args[1] = {self};
  return PyObject_VectorcallMethod(method, args, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}

/* Reads a tensor; 0 on success. */
static int read_tensor(Tensor* t, PyObject* obj, const char* name) {
  t->obj = obj;
  t->name = name;
  int n;
  if (read_ints(PyObject_GetAttr(obj, s_shape), t->shape, MAXD, &t->nd)) return -1;
  if (read_ints(call0(obj, s_stride), t->stride, MAXD, &n)) return -1;
  PyObject* p = call0(obj, s_data_ptr);
  if (!p) return -1;
  t->ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return PyErr_Occurred() ? -1 : 0;
}

static PyObject* shape_tuple(const long long* shape, int nd) {
  PyObject* r = PyTuple_New(nd);
  for (int i = 0; r && i < nd; ++i) PyTuple_SET_ITEM(r, i, PyLong_FromLongLong(shape[i]));
  return r;
}

static int check_dtype(const Tensor* t, PyObject* dtype) {
  PyObject* d = PyObject_GetAttr(t->obj, s_dtype);
  if (!d) return -1;
  int ok = d == dtype;
  if (!ok) PyErr_Format(PyExc_ValueError, "%s has dtype %R, expected %R", t->name, d, dtype);
  Py_DECREF(d);
  return ok ? 0 : -1;
}

static int check_device(const Tensor* t, long device) {
  PyObject* d = call0(t->obj, s_get_device);
  if (!d) return -1;
  long at = PyLong_AsLong(d);
  Py_DECREF(d);
  if (at == -1 && PyErr_Occurred()) return -1;
  if (at == device) return 0;
  if (at < 0) PyErr_Format(PyExc_ValueError, "%s is not on a CUDA device, the handle is on cuda:%ld", t->name, device);
  else PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, the handle is on cuda:%ld", t->name, at, device);
  return -1;
}

static int check(const Tensor* t, const long long* shape, int nd, PyObject* dtype, long device) {
  int same = t->nd == nd;
  for (int i = 0; same && i < nd; ++i) same = t->shape[i] == shape[i];
  if (!same) {
    PyObject *got = shape_tuple(t->shape, t->nd), *want = shape_tuple(shape, nd);
    if (got && want) PyErr_Format(PyExc_ValueError, "%s has shape %R, expected %R", t->name, got, want);
    Py_XDECREF(got);
    Py_XDECREF(want);
    return -1;
  }
  return check_dtype(t, dtype) || check_device(t, device) ? -1 : 0;
}

/* A contiguous tensor, or None where `optional`: *ptr is then NULL. */
static int dense(PyObject* obj, const char* name, const long long* shape, int nd, PyObject* dtype, long device,
                 void** ptr) {
  Tensor t;
  *ptr = NULL;
  if (obj == Py_None) return 0;
  if (read_tensor(&t, obj, name) || check(&t, shape, nd, dtype, device)) return -1;
  long long want = 1;
  int empty = 0;
  for (int i = 0; i < nd; ++i) empty |= shape[i] == 0;
  for (int i = nd - 1; i >= 0 && !empty; --i) {
    if (shape[i] != 1 && t.stride[i] != want) {
      PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
      return -1;
    }
    want *= shape[i];
  }
  *ptr = t.ptr;
  return 0;
}

/* Strides {sequence, token} of token rows whose values within a token are adjacent. */
static int row_strides(const Tensor* t, int lead, int form, long long* out) {
  long long width = 1;
  int empty = 0;
  for (int i = 0; i < t->nd; ++i) empty |= t->shape[i] == 0;
  for (int i = t->nd - 1; i >= lead && !empty; --i) {
    if (t->shape[i] != 1 && t->stride[i] != width) {
      PyErr_Format(PyExc_ValueError, "%s: the values of a token must be adjacent", t->name);
      return -1;
    }
    width *= t->shape[i];
  }
  out[0] = form == PACKED ? 0 : t->stride[0];
  out[1] = form == DENSE ? t->stride[1] : form == PACKED ? t->stride[0] : width;
  return 0;
}

static int rows(Tensor* t, PyObject* obj, const char* name, const long long* shape, int nd, PyObject* dtype,
                long device, int form, long long* out) {
  if (read_tensor(t, obj, name) || check(t, shape, nd, dtype, device)) return -1;
  return row_strides(t, form == DENSE ? 2 : 1, form, out);
}

typedef struct {
  vla_handle_t h;
  long device;
  void* stream;
  int direct;   /* see read_allocator; -1: not asked yet */
} Call;

/* The handle's pointer and device, and the stream (an int; None: torch's current one). */
static int read_call(Call* c, PyObject* self, PyObject* stream) {
  PyObject *p = PyObject_GetAttr(self, s_ptr), *d = PyObject_GetAttr(self, s_index);
  c->direct = -1;
  if (p && d) {
    c->h = (vla_handle_t)PyLong_AsVoidPtr(p);
    c->device = PyLong_AsLong(d);
    if (stream == Py_None) {
      PyObject* s = PyObject_CallOneArg(c_stream, d);
      if (s) c->stream = PyLong_AsVoidPtr(s);
      Py_XDECREF(s);
    } else {
      c->stream = PyLong_AsVoidPtr(stream);
    }
  }
  Py_XDECREF(p);
  Py_XDECREF(d);
  return PyErr_Occurred() ? -1 : 0;
}

static int read_io(const Tensor* x, PyObject** dtype, vla_dtype_t* io) {
  PyObject* d = PyObject_GetAttr(x->obj, s_dtype);
  if (!d) return -1;
  Py_DECREF(d);   /* torch keeps its dtypes */
  *dtype = d;
  if (d == t_f32) *io = VLA_F32;
  else if (d == t_bf16) *io = VLA_BF16;
  else {
    PyErr_Format(PyExc_ValueError, "%s must be float32 or bfloat16", x->name);
    return -1;
  }
  return 0;
}

typedef struct {
  long long n_seq, T, max_len, n_slots;
  void *offsets, *slots;
  int form;
} Batch;

/* The sequences of a batch.  form: TOKEN, or DENSE which offsets turn into PACKED. */
static int read_batch(Batch* b, const Tensor* x, PyObject* offsets, PyObject* slots, PyObject* state,
                      PyObject* max_len, long device) {
  long long shape[1];
  b->offsets = NULL;
  if (b->form == PACKED) {
    Tensor o;
    if (read_tensor(&o, offsets, "offsets")) return -1;
    if (o.nd != 1 || o.shape[0] < 1) {
      PyErr_SetString(PyExc_ValueError, "offsets must be [sequences + 1]");
      return -1;
    }
    if (dense(offsets, "offsets", o.shape, 1, t_i32, device, &b->offsets)) return -1;
    b->n_seq = o.shape[0] - 1;
    b->T = b->max_len = x->shape[0];
    if (max_len != Py_None) b->max_len = PyLong_AsLongLong(max_len);
    if (PyErr_Occurred()) return -1;
  } else {
    b->n_seq = x->shape[0];
    b->T = b->max_len = b->form == DENSE ? x->shape[1] : 1;
  }
  if (slots != Py_None && state == Py_None) {
    PyErr_SetString(PyExc_ValueError, "slots need a state");
    return -1;
  }
  shape[0] = b->n_seq;
  return dense(slots, "slots", shape, 1, t_i32, device, &b->slots);
}

/* The pool's size: the first dimension of the state. */
static int read_slots(Batch* b, PyObject* state, Tensor* t) {
  b->n_slots = 0;
  if (state == Py_None) return 0;
  if (read_tensor(t, state, "state")) return -1;
  b->n_slots = t->nd > 0 ? t->shape[0] : 0;
  return 0;
}

static PyObject* failed(PyObject* self, vla_err_t code, PyObject* y) {
  Py_XDECREF(y);
  PyObject* c = PyLong_FromLong(code);
  if (!c) return NULL;
  PyObject* r = PyObject_CallMethodOneArg(self, s_fail, c);   /* raises */
  Py_DECREF(c);
  return r;
}

/* A new contiguous tensor of x's shape; dtype NULL: x's.  torch.empty_like keeps the strides of a
 * contiguous x, and costs a fifth of the call that asks for a layout. */
static PyObject* like(const Tensor* x, PyObject* dtype) {
  long long step = 1;
  int dense = 1;
  for (int i = x->nd - 1; i >= 0; --i) {
    if (x->shape[i] != 1 && x->stride[i] != step) dense = 0;
    step *= x->shape[i];
  }
  PyObject* args[2] = {x->obj, dtype};
  if (!dense) return PyObject_Vectorcall(c_dense, args, dtype ? 2 : 1, NULL);
  return PyObject_Vectorcall(c_like, args, 1, dtype ? k_dtype : NULL);
}

/* y as given, or a new contiguous tensor like x. */
static PyObject* output(PyObject* y, const Tensor* x) {
  if (y == Py_None) return like(x, NULL);
  Py_INCREF(y);
  return y;
}

static PyObject* want(const char* text) {
  PyErr_SetString(PyExc_ValueError, text);
  return NULL;
}

static int truth(PyObject* o) { return PyObject_IsTrue(o); }

/* A workspace of `need` bytes (none for 0) from the allocator of the tensor `like`. */
static int workspace(PyObject* like, size_t need, PyObject** ws, void** ptr) {
  *ws = NULL;
  *ptr = NULL;
  if (!need) return 0;
  PyObject* size = PyLong_FromSize_t(need);
  PyObject* args[2] = {like, size};
  *ws = size ? PyObject_Vectorcall(c_bytes, args, 2, NULL) : NULL;
  Py_XDECREF(size);
  PyObject* p = *ws ? call0(*ws, s_data_ptr) : NULL;
  if (p) *ptr = PyLong_AsVoidPtr(p);
  Py_XDECREF(p);
  if (p && !PyErr_Occurred()) return 0;
  Py_CLEAR(*ws);
  return -1;
}

/* conv(handle, x, w, bias, state, y, silu, offsets, slots, max_len, token, stream) */
static PyObject* py_conv(PyObject* mod, PyObject* const* a, Py_ssize_t n) {
  (void)mod;
  if (n != 12) return want("conv takes 12 arguments");
  PyObject *self = a[0], *y = NULL;
  Call c;
  Tensor x, w, st, yt;
  Batch b;
  PyObject* dtype;
  vla_dtype_t io;
  long long strides[4], shape[3];
  void *bias, *wp, *sp;
  if (read_call(&c, self, a[11]) || read_tensor(&x, a[1], "x") || read_tensor(&w, a[2], "w")) return NULL;
  b.form = truth(a[10]) ? TOKEN : a[7] == Py_None ? DENSE : PACKED;
  if (x.nd != (b.form == DENSE ? 3 : 2))
    return want(b.form == TOKEN ? "x must be [S, C]" : "x must be [S, T, C], or [tokens, C] with offsets");
  if (read_io(&x, &dtype, &io) || check_device(&x, c.device)) return NULL;
  if (w.nd != 2 || w.shape[0] != x.shape[x.nd - 1]) return want("w must be [C, K]");
  const long long C = w.shape[0], K = w.shape[1];
  if (read_batch(&b, &x, a[7], a[8], a[4], a[9], c.device) || read_slots(&b, a[4], &st)) return NULL;
  if (row_strides(&x, x.nd - 1, b.form, strides)) return NULL;
  if (dense(a[2], "w", w.shape, 2, t_f32, c.device, &wp)) return NULL;
  shape[0] = C;
  if (dense(a[3], "bias", shape, 1, t_f32, c.device, &bias)) return NULL;
  shape[0] = b.n_slots; shape[1] = K - 1; shape[2] = C;
  if (dense(a[4], "state", shape, 3, dtype, c.device, &sp)) return NULL;
  if (!(y = output(a[5], &x))) return NULL;
  if (rows(&yt, y, "y", x.shape, x.nd, dtype, c.device, b.form, strides + 2)) {
    Py_DECREF(y);
    return NULL;
  }
  const int silu = truth(a[6]);
  vla_err_t code;
  Py_BEGIN_ALLOW_THREADS
  code = f_conv(c.h, x.ptr, (const float*)wp, (const float*)bias, sp, yt.ptr, b.n_seq, b.T, b.max_len,
                (const int*)b.offsets, (const int*)b.slots, b.n_slots, C, K > 100 ? 100 : (int)K, strides, silu, io,
                c.stream);
  Py_END_ALLOW_THREADS
  return code ? failed(self, code, y) : y;
}

/* scan(handle, x, dt, A, B, C, state, y, D, z, dt_bias, softplus, offsets, slots, max_len, token, stream) */
static PyObject* py_scan(PyObject* mod, PyObject* const* a, Py_ssize_t n) {
  (void)mod;
  if (n != 17) return want("scan takes 17 arguments");
  PyObject *self = a[0], *y = NULL, *ws = NULL;
  Call c;
  Tensor x, dt, B, Ct, z, st, yt;
  Batch b;
  PyObject* dtype;
  vla_dtype_t io;
  long long strides[12] = {0}, shape[4];
  void *A, *D, *bias, *sp, *zp = NULL, *wsp = NULL;
  if (read_call(&c, self, a[16]) || read_tensor(&x, a[1], "x") || read_tensor(&B, a[4], "B")) return NULL;
  b.form = truth(a[15]) ? TOKEN : a[12] == Py_None ? DENSE : PACKED;
  const int lead = b.form == DENSE ? 2 : 1;
  if (x.nd != lead + 2)
    return want(b.form == TOKEN ? "x must be [S, H, P]" : "x must be [S, T, H, P], or [tokens, H, P] with offsets");
  if (read_io(&x, &dtype, &io) || check_device(&x, c.device)) return NULL;
  if (B.nd != x.nd)
    return want(b.form == TOKEN ? "B must be [S, G, N]" : "B must be [S, T, G, N], or [tokens, G, N] with offsets");
  const long long H = x.shape[lead], P = x.shape[lead + 1], G = B.shape[lead], N = B.shape[lead + 1];
  if (read_batch(&b, &x, a[12], a[13], a[6], a[14], c.device) || read_slots(&b, a[6], &st)) return NULL;
  if (row_strides(&x, lead, b.form, strides)) return NULL;
  for (int i = 0; i < lead; ++i) shape[i] = x.shape[i];
  shape[lead] = H;
  if (rows(&dt, a[2], "dt", shape, lead + 1, dtype, c.device, b.form, strides + 2)) return NULL;
  shape[lead] = G;
  shape[lead + 1] = N;
  if (check(&B, shape, lead + 2, dtype, c.device) || row_strides(&B, lead, b.form, strides + 4)) return NULL;
  if (rows(&Ct, a[5], "C", shape, lead + 2, dtype, c.device, b.form, strides + 6)) return NULL;
  if (a[9] != Py_None) {
    if (rows(&z, a[9], "z", x.shape, x.nd, dtype, c.device, b.form, strides + 8)) return NULL;
    zp = z.ptr;
  }
  if (a[3] == Py_None) return want("A must be [H] float32");
  if (dense(a[3], "A", &H, 1, t_f32, c.device, &A) || dense(a[8], "D", &H, 1, t_f32, c.device, &D) ||
      dense(a[10], "dt_bias", &H, 1, t_f32, c.device, &bias))
    return NULL;
  shape[0] = b.n_slots; shape[1] = H; shape[2] = P; shape[3] = N;
  if (dense(a[6], "state", shape, 4, t_f32, c.device, &sp)) return NULL;
  size_t need = 0;
  vla_err_t code = f_ws(c.h, b.n_seq, b.T, b.max_len, b.form == PACKED, H, P, N, io, &need);
  if (code) return failed(self, code, NULL);
  if (!(y = output(a[7], &x))) return NULL;
  if (rows(&yt, y, "y", x.shape, x.nd, dtype, c.device, b.form, strides + 10)) {
    Py_DECREF(y);
    return NULL;
  }
  if (workspace(a[1], need, &ws, &wsp)) {
    Py_DECREF(y);
    return NULL;
  }
  const int softplus = truth(a[11]);
  Py_BEGIN_ALLOW_THREADS
  code = f_scan(c.h, x.ptr, dt.ptr, (const float*)A, B.ptr, Ct.ptr, (const float*)D, zp, (const float*)bias,
                (float*)sp, yt.ptr, b.n_seq, b.T, b.max_len, (const int*)b.offsets, (const int*)b.slots, b.n_slots,
                H, P, G, N, strides, softplus, io, wsp, need, c.stream);
  Py_END_ALLOW_THREADS
  Py_XDECREF(ws);   /* the caching allocator hands it on in stream order */
  return code ? failed(self, code, y) : y;
}

/* Rows of evenly spaced values: their number and distance. */
static int even(const Tensor* t, long long* n_rows, long long* step) {
  int started = 0, empty = 0;
  long long count = 1, gap = t->shape[t->nd - 1];
  for (int i = 0; i < t->nd; ++i) empty |= t->shape[i] == 0;
  if (empty) {
    *n_rows = 0;
    *step = gap;
    return 0;
  }
  if (t->shape[t->nd - 1] > 1 && t->stride[t->nd - 1] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: the values of a row must be adjacent", t->name);
    return -1;
  }
  for (int i = t->nd - 2; i >= 0; --i) {
    if (t->shape[i] == 1) continue;
    if (!started) {
      started = 1;
      gap = t->stride[i];
    } else if (t->stride[i] != gap * count) {
      PyErr_Format(PyExc_ValueError, "%s: rows must be evenly spaced", t->name);
      return -1;
    }
    count *= t->shape[i];
  }
  *n_rows = count;
  *step = gap;
  return 0;
}

/* norm(handle, x, w, residual, y, eps, out, group, scale, stream); out: 0 io, 1 e4m3, 2 int8 */
static PyObject* py_norm(PyObject* mod, PyObject* const* a, Py_ssize_t n) {
  (void)mod;
  if (n != 10) return want("norm takes 10 arguments");
  PyObject *self = a[0], *y = NULL, *scale = NULL, *dtype, *rdtype, *odtype, *made;
  Call c;
  Tensor x, r, yt;
  vla_dtype_t io, rio = VLA_F32;
  long long count, x_row, r_row = 0, y_row, ignored;
  void *w, *rp = NULL, *sp = NULL;
  const double eps = PyFloat_AsDouble(a[5]);
  const long out = PyLong_AsLong(a[6]), group = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) return NULL;
  if (group != 0 && group != 128) return want("group must be 0 or 128");
  if (read_call(&c, self, a[9]) || read_tensor(&x, a[1], "x")) return NULL;
  if (x.nd < 1) return want("x must be [..., D]");
  if (read_io(&x, &dtype, &io) || check_device(&x, c.device) || even(&x, &count, &x_row)) return NULL;
  const long long D = x.shape[x.nd - 1];
  if (a[2] == Py_None) return want("w must be [D] float32");
  if (dense(a[2], "w", &D, 1, t_f32, c.device, &w)) return NULL;
  if (a[3] != Py_None) {
    if (read_tensor(&r, a[3], "residual") || read_io(&r, &rdtype, &rio) ||
        check(&r, x.shape, x.nd, rdtype, c.device) || even(&r, &ignored, &r_row))
      return NULL;
    rp = r.ptr;
  }
  odtype = out == 0 ? dtype : out == 1 ? t_e4m3 : t_i8;
  if (a[4] != Py_None) {
    y = a[4];
    Py_INCREF(y);
  } else {
    y = like(&x, out == 0 ? NULL : odtype);
  }
  if (!y) return NULL;
  if (read_tensor(&yt, y, "y") || check(&yt, x.shape, x.nd, odtype, c.device) || even(&yt, &ignored, &y_row)) goto bad;
  if (out != 0) {
    long long shape[MAXD];
    int nd = x.nd - 1;
    for (int i = 0; i < nd; ++i) shape[i] = x.shape[i];
    if (group) shape[nd++] = (D + 127) / 128;
    if (a[8] != Py_None) {
      scale = a[8];
      Py_INCREF(scale);
    } else {
      PyObject* size = shape_tuple(shape, nd);
      PyObject* args[2] = {a[1], size};
      scale = size ? PyObject_Vectorcall(c_empty, args, 2, NULL) : NULL;
      Py_XDECREF(size);
    }
    if (!scale || dense(scale, "scale", shape, nd, t_f32, c.device, &sp)) goto bad;
  }
  {
    vla_err_t code;
    Py_BEGIN_ALLOW_THREADS
    code = f_norm(c.h, x.ptr, (const float*)w, rp, yt.ptr, (float*)sp, count, D, x_row, r_row, y_row, (float)eps,
                  (int)group, (vla_out_t)out, io, rio, c.stream);
    Py_END_ALLOW_THREADS
    if (code) {
      Py_XDECREF(scale);
      return failed(self, code, y);
    }
  }
  if (out == 0) return y;
  made = PyTuple_Pack(2, y, scale);
  Py_DECREF(y);
  Py_DECREF(scale);
  return made;
bad:
  Py_XDECREF(y);
  Py_XDECREF(scale);
  return NULL;
}

/* Whether the call's outputs can come from torch's allocator without its dispatcher: where torch offers that (c_strided:
 * sizes, strides, dtype, on the current device, which c_at says), the handle's device is the current one, and no
 * dispatch mode (c_modes counts them) watches or replaces what is allocated.  Behind a launch torch.empty takes 3.3 us
 * (new_empty 6.3, empty_like 3.2), that 1.5. */
static int read_allocator(Call* c) {
  c->direct = 0;
  if (c_strided == Py_None) return 0;
  PyObject *modes = PyObject_CallNoArgs(c_modes), *at = modes ? PyObject_CallNoArgs(c_at) : NULL;
  if (at) c->direct = PyLong_AsLong(modes) == 0 && PyLong_AsLong(at) == c->device;
  Py_XDECREF(modes);
  Py_XDECREF(at);
  return PyErr_Occurred() ? -1 : 0;
}

/* A new contiguous tensor on the device of `like`. */
static PyObject* fresh(Call* c, PyObject* like, const long long* shape, int nd, PyObject* dtype) {
  PyObject *size, *r = NULL;
  if ((c->direct < 0 && read_allocator(c)) || !(size = shape_tuple(shape, nd))) return NULL;
  if (c->direct) {
    long long stride[MAXD], step = 1;
    for (int i = nd - 1; i >= 0; --i) {
      stride[i] = step;
      step *= shape[i] > 1 ? shape[i] : 1;
    }
    PyObject* strides = shape_tuple(stride, nd);
    PyObject* args[3] = {size, strides, dtype};
    r = strides ? PyObject_Vectorcall(c_strided, args, 3, NULL) : NULL;
    Py_XDECREF(strides);
  } else {
    PyObject* dev = PyObject_GetAttr(like, s_device);
    PyObject* args[3] = {size, dtype, dev};
    r = dev ? PyObject_Vectorcall(c_new, args, 1, k_new) : NULL;
    Py_XDECREF(dev);
  }
  Py_DECREF(size);
  return r;
}

/* The tensor given, or a new contiguous one. */
static PyObject* given_or_new(Call* c, PyObject* given, PyObject* like, const long long* shape, int nd, PyObject* dtype) {
  if (given == Py_None) return fresh(c, like, shape, nd, dtype);
  Py_INCREF(given);
  return given;
}

/* A workspace of `need` bytes (none for 0). */
static int scratch(Call* c, PyObject* like, size_t need, PyObject** ws, void** ptr) {
  const long long size = (long long)need;
  *ws = NULL;
  *ptr = NULL;
  if (!need) return 0;
  PyObject* p = (*ws = fresh(c, like, &size, 1, t_u8)) ? call0(*ws, s_data_ptr) : NULL;
  if (p) *ptr = PyLong_AsVoidPtr(p);
  Py_XDECREF(p);
  if (p && !PyErr_Occurred()) return 0;
  Py_CLEAR(*ws);
  return -1;
}

/* The products and norms record no gradient: a tensor that wants one is refused, where gradients are recorded at all.
 * (0.2 us of a call.) */
static int no_gradient(PyObject* const* a, const char* const* names, int n) {
  PyObject* on = PyObject_CallNoArgs(c_grad);
  if (!on) return -1;
  Py_DECREF(on);   /* a singleton */
  for (int i = 0; i < n && on == Py_True; ++i) {
    if (!names[i] || a[i] == Py_None || PyBool_Check(a[i])) continue;
    PyObject* r = PyObject_GetAttr(a[i], s_requires);
    if (!r) return -1;
    Py_DECREF(r);
    if (r != Py_True) continue;
    PyErr_Format(PyExc_ValueError,
                 "%s requires a gradient, and the call would not record one: make it under torch.no_grad() or in an "
                 "autograd.Function that calls the gradient's operator",
                 names[i]);
    return -1;
  }
  return 0;
}

/* Reads and checks a tensor of evenly spaced rows, [..., width]. */
static int even_rows(Tensor* t, PyObject* obj, const char* name, const long long* shape, int nd, PyObject* dtype,
                     long device, long long* step) {
  long long ignored;
  return read_tensor(t, obj, name) || check(t, shape, nd, dtype, device) || even(t, &ignored, step) ? -1 : 0;
}

/* linear(handle, x, w, bias, residual, y, act, pre, x_scale, w_scale, dtype, stream); act: 0 none, 1 silu, 2 gelu */
static PyObject* py_linear(PyObject* mod, PyObject* const* a, Py_ssize_t n) {
  (void)mod;
  static const char* const names[] = {"x", "w", "bias", "residual", "y", NULL, "pre", "x_scale", "w_scale"};
  if (n != 12) return want("linear takes 12 arguments");
  if (no_gradient(a + 1, names, 9)) return NULL;
  PyObject *self = a[0], *y = NULL, *ws = NULL, *dtype, *odtype;
  Call c;
  Tensor x, w, t;
  vla_mat_t in;
  vla_dtype_t out;
  long long M, N, K, ignored, rows[5] = {0}, shape[MAXD], wshape[2];
  void *bias, *xs, *wsc, *res = NULL, *pre = NULL, *yp, *wsp = NULL;
  const long act = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return NULL;
  if (read_call(&c, self, a[11]) || read_tensor(&x, a[1], "x") || read_tensor(&w, a[2], "w")) return NULL;
  if (x.nd < 1) return want("x must be [..., K]");
  if (w.nd != 2) return want("w must be [N, K]");
  if (!(dtype = PyObject_GetAttr(a[1], s_dtype))) return NULL;
  Py_DECREF(dtype);   /* torch keeps its dtypes */
  if (dtype == t_f32) in = VLA_MAT_F32;
  else if (dtype == t_bf16) in = VLA_MAT_BF16;
  else if (dtype == t_e4m3) in = VLA_MAT_E4M3;
  else return want("x must be float32, bfloat16 or float8_e4m3fn");
  if (check_device(&x, c.device) || even(&x, &M, &rows[0])) return NULL;
  K = x.shape[x.nd - 1];
  N = w.shape[0];
  wshape[0] = N; wshape[1] = K;
  if (check(&w, wshape, 2, dtype, c.device) || even(&w, &ignored, &rows[1])) return NULL;
  odtype = a[10] != Py_None ? a[10] : dtype == t_e4m3 ? t_bf16 : dtype;
  if (odtype == t_f32) out = VLA_F32;
  else if (odtype == t_bf16) out = VLA_BF16;
  else return want("dtype must be float32 or bfloat16");
  if (dense(a[3], "bias", &N, 1, t_f32, c.device, &bias) || dense(a[9], "w_scale", &N, 1, t_f32, c.device, &wsc) ||
      dense(a[8], "x_scale", x.shape, x.nd - 1, t_f32, c.device, &xs))
    return NULL;
  for (int i = 0; i < x.nd - 1; ++i) shape[i] = x.shape[i];
  shape[x.nd - 1] = N;
  if (a[4] != Py_None) {
    if (even_rows(&t, a[4], "residual", shape, x.nd, odtype, c.device, &rows[2])) return NULL;
    res = t.ptr;
  }
  if (a[7] != Py_None) {
    if (even_rows(&t, a[7], "pre", shape, x.nd, odtype, c.device, &rows[3])) return NULL;
    pre = t.ptr;
  }
  if (!(y = given_or_new(&c, a[5], a[1], shape, x.nd, odtype))) return NULL;
  if (even_rows(&t, y, "y", shape, x.nd, odtype, c.device, &rows[4])) goto bad;
  yp = t.ptr;
  M = 1;   /* x without columns has its rows all the same */
  for (int i = 0; i < x.nd - 1; ++i) M *= x.shape[i];
  size_t need = 0;
  vla_err_t code = f_linear_ws(c.h, x.ptr, w.ptr, M, N, K, rows, in, out, &need);
  if (code) return failed(self, code, y);
  if (scratch(&c, a[1], need, &ws, &wsp)) goto bad;
  Py_BEGIN_ALLOW_THREADS
  code = f_linear(c.h, x.ptr, w.ptr, (const float*)xs, (const float*)wsc, (const float*)bias, res, pre, yp, M, N, K, rows,
                  (vla_act_t)act, in, out, wsp, need, c.stream);
  Py_END_ALLOW_THREADS
  Py_XDECREF(ws);   /* the caching allocator hands it on in stream order */
  return code ? failed(self, code, y) : y;
bad:
  Py_DECREF(y);
  return NULL;
}

/* linear_back(handle, dy, x, w, pre, act, dx, dw, db, stream); dx, dw, db: a tensor, None (a new one) or False (not
 * computed) */
static PyObject* py_linear_back(PyObject* mod, PyObject* const* a, Py_ssize_t n) {
  (void)mod;
  static const char* const names[] = {"dy", "x", "w", "pre", NULL, "dx", "dw", "db"};
  if (n != 10) return want("linear_back takes 10 arguments");
  if (no_gradient(a + 1, names, 8)) return NULL;
  PyObject *self = a[0], *ws = NULL, *dtype, *got[3] = {NULL, NULL, NULL}, *made;
  Call c;
  Tensor dy, x, w, t;
  vla_dtype_t io;
  long long M, N, K, ignored, rows[6] = {0}, shape[MAXD];
  void *pre = NULL, *out[3] = {NULL, NULL, NULL}, *wsp = NULL;
  const long act = PyLong_AsLong(a[5]);
  if (PyErr_Occurred()) return NULL;
  if (read_call(&c, self, a[9]) || read_tensor(&dy, a[1], "dy") || read_tensor(&x, a[2], "x") || read_tensor(&w, a[3], "w"))
    return NULL;
  if (dy.nd < 1 || x.nd != dy.nd) return want("dy must be [..., N] and x [..., K] with the same rows");
  if (w.nd != 2) return want("w must be [N, K]");
  if (read_io(&dy, &dtype, &io) || check_device(&dy, c.device)) return NULL;
  N = w.shape[0];
  K = w.shape[1];
  M = 1;
  for (int i = 0; i < dy.nd - 1; ++i) M *= shape[i] = dy.shape[i];
  shape[dy.nd - 1] = K;
  if (check(&x, shape, x.nd, dtype, c.device) || even(&x, &ignored, &rows[1])) return NULL;
  if (check(&w, w.shape, 2, dtype, c.device) || even(&w, &ignored, &rows[2])) return NULL;
  shape[dy.nd - 1] = N;
  if (check(&dy, shape, dy.nd, dtype, c.device) || even(&dy, &ignored, &rows[0])) return NULL;
  if (act != 0) {
    if (a[4] == Py_None) return want("pre is needed behind an activation");
    if (even_rows(&t, a[4], "pre", shape, dy.nd, dtype, c.device, &rows[3])) return NULL;
    pre = t.ptr;
  }
  for (int i = 0; i < 3; ++i) {
    if (a[6 + i] == Py_False) {
      Py_INCREF(Py_None);
      got[i] = Py_None;
      continue;
    }
    const char* name = i == 0 ? "dx" : i == 1 ? "dw" : "db";
    const long long* sh = i == 0 ? x.shape : i == 1 ? w.shape : &N;
    const int nd = i == 0 ? x.nd : i == 1 ? 2 : 1;
    PyObject* dt = i == 2 ? t_f32 : dtype;
    if (!(got[i] = given_or_new(&c, a[6 + i], a[1], sh, nd, dt))) goto bad;
    if (i == 2) {
      if (dense(got[2], name, sh, 1, dt, c.device, &out[2])) goto bad;
    } else {
      if (even_rows(&t, got[i], name, sh, nd, dt, c.device, &rows[4 + i])) goto bad;
      out[i] = t.ptr;
    }
  }
  {
    size_t need = 0;
    vla_err_t code = f_linear_back_ws(c.h, dy.ptr, x.ptr, w.ptr, got[0] != Py_None, got[1] != Py_None, got[2] != Py_None,
                                      M, N, K, rows, (vla_act_t)act, io, &need);
    if (!code) {
      if (scratch(&c, a[1], need, &ws, &wsp)) goto bad;
      Py_BEGIN_ALLOW_THREADS
      code = f_linear_back(c.h, dy.ptr, x.ptr, w.ptr, pre, out[0], out[1], (float*)out[2], M, N, K, rows, (vla_act_t)act,
                           io, wsp, need, c.stream);
      Py_END_ALLOW_THREADS
      Py_XDECREF(ws);
    }
    if (code) {
      Py_DECREF(got[0]);
      Py_DECREF(got[1]);
      return failed(self, code, got[2]);
    }
  }
  made = PyTuple_Pack(3, got[0], got[1], got[2]);
  for (int i = 0; i < 3; ++i) Py_DECREF(got[i]);
  return made;
bad:
  for (int i = 0; i < 3; ++i) Py_XDECREF(got[i]);
  return NULL;
}

/* layer_norm(handle, x, w, b, residual, y, eps, stats, stream); stats: a tensor, True (a new one) or False */
static PyObject* py_layer_norm(PyObject* mod, PyObject* const* a, Py_ssize_t n) {
  (void)mod;
  static const char* const names[] = {"x", "w", "b", "residual", "y", NULL, "stats"};
  if (n != 9) return want("layer_norm takes 9 arguments");
  if (no_gradient(a + 1, names, 7)) return NULL;
  PyObject *self = a[0], *y = NULL, *stats = NULL, *dtype, *rdtype, *made;
  Call c;
  Tensor x, r, t;
  vla_dtype_t io, rio = VLA_F32;
  long long count, x_row, r_row = 0, y_row, ignored, shape[MAXD];
  void *w, *b, *rp = NULL, *sp = NULL;
  const double eps = PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred()) return NULL;
  if (read_call(&c, self, a[8]) || read_tensor(&x, a[1], "x")) return NULL;
  if (x.nd < 1) return want("x must be [..., D]");
  if (read_io(&x, &dtype, &io) || check_device(&x, c.device) || even(&x, &count, &x_row)) return NULL;
  const long long D = x.shape[x.nd - 1];
  if (a[2] == Py_None) return want("w must be [D] float32");
  if (dense(a[2], "w", &D, 1, t_f32, c.device, &w) || dense(a[3], "b", &D, 1, t_f32, c.device, &b)) return NULL;
  if (a[4] != Py_None) {
    if (read_tensor(&r, a[4], "residual") || read_io(&r, &rdtype, &rio) ||
        check(&r, x.shape, x.nd, rdtype, c.device) || even(&r, &ignored, &r_row))
      return NULL;
    rp = r.ptr;
  }
  if (!(y = given_or_new(&c, a[5], a[1], x.shape, x.nd, dtype))) return NULL;
  if (even_rows(&t, y, "y", x.shape, x.nd, dtype, c.device, &y_row)) goto bad;
  if (a[7] != Py_False) {
    if (x.nd >= MAXD) {
      want("statistics are kept of tensors of at most 7 dimensions");
      goto bad;
    }
    for (int i = 0; i < x.nd - 1; ++i) shape[i] = x.shape[i];
    shape[x.nd - 1] = 2;
    if (!(stats = given_or_new(&c, a[7] == Py_True ? Py_None : a[7], a[1], shape, x.nd, t_f32))) goto bad;
    if (dense(stats, "stats", shape, x.nd, t_f32, c.device, &sp)) goto bad;
  }
  {
    vla_err_t code;
    Py_BEGIN_ALLOW_THREADS
    code = f_lnorm(c.h, x.ptr, (const float*)w, (const float*)b, rp, t.ptr, (float*)sp, count, D, x_row, r_row, y_row,
                   (float)eps, io, rio, c.stream);
    Py_END_ALLOW_THREADS
    if (code) {
      Py_XDECREF(stats);
      return failed(self, code, y);
    }
  }
  if (!stats) return y;
  made = PyTuple_Pack(2, y, stats);
  Py_DECREF(y);
  Py_DECREF(stats);
  return made;
bad:
  Py_XDECREF(y);
  Py_XDECREF(stats);
  return NULL;
}

/* layer_norm_back(handle, dy, x, w, stats, dresidual, dx, dw, db, stream); db: a tensor, None (a new one) or False (not
 * computed) */
static PyObject* py_layer_norm_back(PyObject* mod, PyObject* const* a, Py_ssize_t n) {
  (void)mod;
  static const char* const names[] = {"dy", "x", "w", "stats", "dresidual", "dx", "dw", "db"};
  if (n != 10) return want("layer_norm_back takes 10 arguments");
  if (no_gradient(a + 1, names, 8)) return NULL;
  PyObject *self = a[0], *dx = NULL, *dw = NULL, *db = NULL, *ws = NULL, *gtype, *dtype, *made;
  Call c;
  Tensor dy, x, t;
  vla_dtype_t gio, io;
  long long count, strides[4] = {0}, shape[MAXD];
  void *w, *sp, *res = NULL, *dxp, *dwp = NULL, *dbp = NULL, *wsp = NULL;
  if (read_call(&c, self, a[9]) || read_tensor(&dy, a[1], "dy") || read_tensor(&x, a[2], "x")) return NULL;
  if (x.nd < 1) return want("x must be [..., D]");
  if (read_io(&x, &dtype, &io) || check_device(&x, c.device) || even(&x, &count, &strides[1])) return NULL;
  if (read_io(&dy, &gtype, &gio) || check(&dy, x.shape, x.nd, gtype, c.device) || even(&dy, &count, &strides[0])) return NULL;
  const long long D = x.shape[x.nd - 1];
  if (a[3] == Py_None) return want("w must be [D] float32");
  if (a[4] == Py_None) return want("stats must be [..., 2] float32");
  if (dense(a[3], "w", &D, 1, t_f32, c.device, &w)) return NULL;
  for (int i = 0; i < x.nd - 1; ++i) shape[i] = x.shape[i];
  shape[x.nd - 1] = 2;
  if (dense(a[4], "stats", shape, x.nd, t_f32, c.device, &sp)) return NULL;
  if (a[5] != Py_None) {
    if (even_rows(&t, a[5], "dresidual", x.shape, x.nd, dtype, c.device, &strides[2])) return NULL;
    res = t.ptr;
  }
  if (!(dx = given_or_new(&c, a[6], a[1], x.shape, x.nd, dtype)) || even_rows(&t, dx, "dx", x.shape, x.nd, dtype, c.device, &strides[3])) goto bad;
  dxp = t.ptr;
  if (!(dw = given_or_new(&c, a[7], a[1], &D, 1, t_f32)) || dense(dw, "dw", &D, 1, t_f32, c.device, &dwp)) goto bad;
  if (a[8] == Py_False) {
    Py_INCREF(Py_None);
    db = Py_None;
  } else if (!(db = given_or_new(&c, a[8], a[1], &D, 1, t_f32)) || dense(db, "db", &D, 1, t_f32, c.device, &dbp)) {
    goto bad;
  }
  {
    size_t need = 0;
    vla_err_t code = f_lnorm_back_ws(c.h, count, D, &need);
    if (!code) {
      if (scratch(&c, a[1], need, &ws, &wsp)) goto bad;
      Py_BEGIN_ALLOW_THREADS
      code = f_lnorm_back(c.h, dy.ptr, x.ptr, (const float*)w, (const float*)sp, res, dxp, (float*)dwp, (float*)dbp, count,
                          D, strides, gio, io, wsp, need, c.stream);
      Py_END_ALLOW_THREADS
      Py_XDECREF(ws);
    }
    if (code) {
      Py_DECREF(dx);
      Py_DECREF(dw);
      return failed(self, code, db);
    }
  }
  made = PyTuple_Pack(3, dx, dw, db);
  Py_DECREF(dx);
  Py_DECREF(dw);
  Py_DECREF(db);
  return made;
bad:
  Py_XDECREF(dx);
  Py_XDECREF(dw);
  Py_XDECREF(db);
  return NULL;
}

/* setup_dense(addresses of the entry points and workspace queries, torch.is_grad_enabled, torch.empty, torch.uint8, and for
 * read_allocator either three callables or None): after setup */
static PyObject* py_setup_dense(PyObject* mod, PyObject* args) {
  (void)mod;
  unsigned long long p[7];
  PyObject* o[6];
  if (!PyArg_ParseTuple(args, "KKKKKKKOOOOOO", p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6, o, o + 1, o + 2, o + 3, o + 4, o + 5))
    return NULL;
  f_linear = (linear_fn)(uintptr_t)p[0];
  f_linear_ws = (linear_ws_fn)(uintptr_t)p[1];
  f_linear_back = (linear_back_fn)(uintptr_t)p[2];
  f_linear_back_ws = (linear_back_ws_fn)(uintptr_t)p[3];
  f_lnorm = (lnorm_fn)(uintptr_t)p[4];
  f_lnorm_back = (lnorm_back_fn)(uintptr_t)p[5];
  f_lnorm_back_ws = (lnorm_back_ws_fn)(uintptr_t)p[6];
  PyObject** slot[6] = {&c_grad, &c_new, &t_u8, &c_strided, &c_at, &c_modes};
  for (int i = 0; i < 6; ++i) {
    Py_INCREF(o[i]);
    Py_XDECREF(*slot[i]);
    *slot[i] = o[i];
  }
  Py_RETURN_NONE;
}

/* setup(addresses of the four entry points, dtypes f32 bf16 i32 e4m3 i8, like, dense, empty, bytes, stream) */
static PyObject* py_setup(PyObject* mod, PyObject* args) {
  (void)mod;
  unsigned long long p[4];
  PyObject* o[10];
  if (!PyArg_ParseTuple(args, "KKKKOOOOOOOOOO", p, p + 1, p + 2, p + 3, o, o + 1, o + 2, o + 3, o + 4, o + 5, o + 6,
                        o + 7, o + 8, o + 9))
    return NULL;
  f_conv = (conv_fn)(uintptr_t)p[0];
  f_scan = (scan_fn)(uintptr_t)p[1];
  f_ws = (ws_fn)(uintptr_t)p[2];
  f_norm = (norm_fn)(uintptr_t)p[3];
  PyObject** slot[10] = {&t_f32, &t_bf16, &t_i32, &t_e4m3, &t_i8, &c_like, &c_dense, &c_empty, &c_bytes, &c_stream};
  for (int i = 0; i < 10; ++i) {
    Py_INCREF(o[i]);
    Py_XDECREF(*slot[i]);
    *slot[i] = o[i];
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, NULL},
    {"conv", (PyCFunction)(void (*)(void))py_conv, METH_FASTCALL, NULL},
    {"scan", (PyCFunction)(void (*)(void))py_scan, METH_FASTCALL, NULL},
    {"norm", (PyCFunction)(void (*)(void))py_norm, METH_FASTCALL, NULL},
    {"setup_dense", py_setup_dense, METH_VARARGS, NULL},
    {"linear", (PyCFunction)(void (*)(void))py_linear, METH_FASTCALL, NULL},
    {"linear_back", (PyCFunction)(void (*)(void))py_linear_back, METH_FASTCALL, NULL},
    {"layer_norm", (PyCFunction)(void (*)(void))py_layer_norm, METH_FASTCALL, NULL},
    {"layer_norm_back", (PyCFunction)(void (*)(void))py_layer_norm_back, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__layer_binding(void) {
  s_shape = PyUnicode_InternFromString("shape");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_ptr = PyUnicode_InternFromString("_ptr_value");
  s_index = PyUnicode_InternFromString("_device_index");
  s_fail = PyUnicode_InternFromString("_layer_fail");
  k_dtype = PyTuple_Pack(1, s_dtype);
  s_device = PyUnicode_InternFromString("device");
  k_new = PyTuple_Pack(2, s_dtype, s_device);
  s_requires = PyUnicode_InternFromString("requires_grad");
  return PyModule_Create(&module);
}
