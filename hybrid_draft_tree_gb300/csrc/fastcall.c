/* The per-layer calls of the binding without its Python-level work: a CPython
 * extension that reads what it needs of each tensor, checks it, and calls the
 * library's entry point (whose address it is given; it links nothing).  A call
 * whose arguments do not pass returns NotImplemented, and the binding's own
 * checks then say what is wrong.  They also take the call when this extension
 * is not built.  What it saves is host time: on the GPU's host the Python form
 * of the checks takes about as long as the launch.  The interpreter lock is
 * free during the call, as it is under ctypes: a call may wait for room in the
 * launch queue. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "graft.h"

static PyObject *s_dtype, *s_is_cuda, *s_numel, *s_contiguous, *s_data_ptr, *s_shape, *s_stride;

/* A whole number that an argument-less method returns; -1: it did not. */
static long long number(PyObject* t, PyObject* name) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) { PyErr_Clear(); return -1; }
  const long long v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (v == -1 && PyErr_Occurred()) PyErr_Clear();
  return v;
}
static int attribute_is(PyObject* t, PyObject* name, PyObject* want) {
  PyObject* r = PyObject_GetAttr(t, name);
  if (!r) { PyErr_Clear(); return 0; }
  Py_DECREF(r); /* dtypes and truth values live on */
  return r == want;
}

/* Contiguous device buffer of at least `numel` elements of `dtype`; None is a null pointer. */
static int buffer(PyObject* t, PyObject* dtype, long long numel, void** out) {
  *out = NULL;
  if (t == Py_None) return 1;
  if (!attribute_is(t, s_dtype, dtype) || !attribute_is(t, s_is_cuda, Py_True)) return 0;
  if (number(t, s_numel) < numel || number(t, s_contiguous) != 1) return 0;
  const long long p = number(t, s_data_ptr);
  *out = (void*)(uintptr_t)p;
  return p != -1;
}
/* The two sizes of a 2-d tensor (or its two strides). */
static int pair_of(PyObject* tuple, long long* x, long long* y) {
  if (!tuple) { PyErr_Clear(); return 0; }
  int ok = PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == 2;
  if (ok) {
    *x = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, 0));
    *y = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, 1));
    if (PyErr_Occurred()) { PyErr_Clear(); ok = 0; }
  }
  Py_DECREF(tuple);
  return ok;
}
/* A contiguous 2-d one of at least `rows` rows: its rows and their length. */
static int table(PyObject* t, PyObject* dtype, long long rows, void** out, long long* height, long long* width) {
  *out = NULL;
  *height = *width = 0;
  if (t == Py_None) return 1;
  if (!attribute_is(t, s_dtype, dtype) || !attribute_is(t, s_is_cuda, Py_True)) return 0;
  if (!pair_of(PyObject_GetAttr(t, s_shape), height, width) || *height < rows || number(t, s_contiguous) != 1) return 0;
  const long long p = number(t, s_data_ptr);
  *out = (void*)(uintptr_t)p;
  return p != -1;
}
/* Rows of at least `width` unit-stride elements at one stride. */
static int rows_of(PyObject* t, PyObject* dtype, long long rows, long long width, void** out, int64_t* stride) {
  *out = NULL;
  *stride = width;
  if (t == Py_None) return 1;
  long long h, w, step, unit;
  if (!attribute_is(t, s_dtype, dtype) || !attribute_is(t, s_is_cuda, Py_True)) return 0;
  if (!pair_of(PyObject_GetAttr(t, s_shape), &h, &w) || !pair_of(PyObject_CallMethodNoArgs(t, s_stride), &step, &unit)) return 0;
  if (w < width || unit != 1 || h < rows || step < w) return 0;
  const long long p = number(t, s_data_ptr);
  *out = (void*)(uintptr_t)p;
  *stride = step;
  return p != -1;
}

static int whole(PyObject* o, long long* v) {
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) { PyErr_Clear(); return 0; }
  return 1;
}
static int small(long long v) { return v >= INT32_MIN && v <= INT32_MAX; }

typedef int (*append_fn)(void*, int32_t, int32_t, const void*, int64_t, const void*, int64_t, const void*, int64_t,
                         const int32_t*, const int32_t*, const float*, int32_t, int32_t, const int32_t*, int32_t,
                         const int32_t*, void*, int64_t, void*, void*, void*);
typedef int (*attend_fn)(void*, int32_t, int32_t, const void*, int64_t, const void*, const void*, const int32_t*, int32_t,
                         const int32_t*, int32_t, const int32_t*, int32_t, const uint64_t*, float, void*, int64_t, float*,
                         void*);
typedef int (*logits_fn)(void*, int32_t, int32_t, const int32_t*, const uint64_t*, const void*, int64_t,
                         const graft_logit_rules*, void*, int64_t, void*);

#define GIVE_UP Py_RETURN_NOTIMPLEMENTED

/* append(entry, handle, stream, dtype, float32, int32, q_width, kv_width, rot_dim, span,
 *        batch, slots, prefix_len, q, k, v, rope, page_table, ctx_len, k_cache, v_cache, q_out, pos, rows) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[13];
  if (n != 24) GIVE_UP;
  for (int i = 0; i < 13; ++i)
    if (i != 3 && i != 4 && i != 5 && !whole(a[i], &v[i])) GIVE_UP;
  PyObject *dt = a[3], *f32 = a[4], *i32 = a[5];
  const long long qw = v[6], kw = v[7], rot = v[8], span = v[9], batch = v[10], slots = v[11], prefix = v[12];
  if (!small(batch) || !small(slots) || !small(prefix) || batch < 0 || slots < 1) GIVE_UP;
  const long long rows = batch * slots;
  void *q, *k, *w, *rope, *pt, *ctx, *kc, *vc, *qo, *pos, *src;
  int64_t qs, ks, ws, qos;
  long long width, pages, positions, unused;
  if (!rows_of(a[13], dt, rows, qw, &q, &qs) || !rows_of(a[14], dt, rows, kw, &k, &ks) ||
      !rows_of(a[15], dt, rows, kw, &w, &ws) || !table(a[16], f32, 0, &rope, &positions, &width) ||
      !table(a[17], i32, batch, &pt, &unused, &pages) || !buffer(a[18], i32, batch, &ctx) || !buffer(a[19], dt, span, &kc) ||
      !buffer(a[20], dt, span, &vc) || !rows_of(a[21], dt, rows, qw, &qo, &qos) || !buffer(a[22], i32, rows, &pos) ||
      !buffer(a[23], i32, rows, &src))
    GIVE_UP;
  if (rope && (width != rot || !small(positions))) GIVE_UP;
  if (!small(pages)) GIVE_UP;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((append_fn)(uintptr_t)v[0])((void*)(uintptr_t)v[1], (int32_t)batch, (int32_t)slots, q, qs, k, ks, w, ws, pos,
                                    src, rope, (int32_t)positions, (int32_t)prefix, pt, (int32_t)pages, ctx, qo, qos,
                                    kc, vc, (void*)(uintptr_t)v[2]);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

/* attend(entry, handle, stream, dtype, float32, int32, int64, q_width, q_heads, page_size, span,
 *        batch, slots, prefix_len, max_ctx, scale, q, k_cache, v_cache, page_table, ctx_len, out, prefix_pages, tree_mask, lse) */
static PyObject* attend(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[15];
  if (n != 25) GIVE_UP;
  for (int i = 0; i < 15; ++i)
    if (!(i >= 3 && i <= 6) && !whole(a[i], &v[i])) GIVE_UP;
  PyObject *dt = a[3], *f32 = a[4], *i32 = a[5], *i64 = a[6];
  const long long qw = v[7], heads = v[8], page = v[9], span = v[10], batch = v[11], slots = v[12], prefix = v[13], max_ctx = v[14];
  const double scale = PyFloat_AsDouble(a[15]);
  if (PyErr_Occurred()) { PyErr_Clear(); GIVE_UP; }
  if (!small(batch) || !small(slots) || !small(prefix) || !small(max_ctx) || batch < 0 || slots < 1 || prefix < 0) GIVE_UP;
  const long long rows = batch * slots;
  void *q, *kc, *vc, *pt, *ctx, *out, *pre, *mask, *lse;
  int64_t qs, os;
  long long pages, unused;
  if (!rows_of(a[16], dt, rows, qw, &q, &qs) || !buffer(a[17], dt, span, &kc) || !buffer(a[18], dt, span, &vc) ||
      !table(a[19], i32, batch, &pt, &unused, &pages) || !buffer(a[20], i32, batch, &ctx) || !rows_of(a[21], dt, rows, qw, &out, &os) ||
      !buffer(a[22], i32, (prefix + page - 1) / page, &pre) || !buffer(a[23], i64, rows, &mask) ||
      !buffer(a[24], f32, rows * heads, &lse) || !small(pages))
    GIVE_UP;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((attend_fn)(uintptr_t)v[0])((void*)(uintptr_t)v[1], (int32_t)batch, (int32_t)slots, q, qs, kc, vc, pre,
                                    (int32_t)prefix, pt, (int32_t)pages, ctx, (int32_t)max_ctx, mask, (float)scale,
                                    out, os, lse, (void*)(uintptr_t)v[2]);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

/* logits(entry, handle, stream, dtype, float32, int32, int64, vocab, batch, slots, logits, out, tree_tok, tree_mask,
 *        hist, hist_len, prompt_len, penalty, bias_tok, bias_val, grammar, grammar_row) */
static PyObject* logits(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[10];
  if (n != 22) GIVE_UP;
  for (int i = 0; i < 10; ++i)
    if (!(i >= 3 && i <= 6) && !whole(a[i], &v[i])) GIVE_UP;
  PyObject *dt = a[3], *f32 = a[4], *i32 = a[5], *i64 = a[6];
  const long long vocab = v[7], batch = v[8], slots = v[9];
  if (!small(batch) || !small(slots) || batch < 0 || slots < 1) GIVE_UP;
  const long long rows = batch * slots;
  graft_logit_rules r = {0};
  void *x, *out, *tok, *mask, *hist, *hist_len = NULL, *prompt = NULL, *pen, *btok, *bval = NULL, *gram, *grow = NULL;
  int64_t xs, os;
  long long hs, bs, gs, gr, unused;
  if (!rows_of(a[10], dt, rows, vocab, &x, &xs) || !rows_of(a[11], dt, rows, vocab, &out, &os) || !buffer(a[12], i32, rows, &tok) ||
      !buffer(a[13], i64, rows, &mask) || !table(a[14], i32, batch, &hist, &unused, &hs) || !buffer(a[17], f32, 3 * batch, &pen) ||
      !table(a[18], i32, batch, &btok, &unused, &bs) || !table(a[20], i32, 0, &gram, &gr, &gs))
    GIVE_UP;
  if (hist && (!buffer(a[15], i32, batch, &hist_len) || !buffer(a[16], i32, batch, &prompt))) GIVE_UP;
  if (a[18] != Py_None && !buffer(a[19], f32, batch * bs, &bval)) GIVE_UP;
  if (a[20] != Py_None && !buffer(a[21], i32, rows, &grow)) GIVE_UP;
  if (!small(bs) || !small(gr)) GIVE_UP;
  r.d_hist = hist; r.hist_stride = hs; r.d_hist_len = hist_len; r.d_prompt_len = prompt; r.d_penalty = pen;
  r.d_bias_tok = btok; r.d_bias_val = bval; r.n_bias = (int32_t)bs;
  r.n_grammar = (int32_t)gr; r.d_grammar = gram; r.grammar_stride = gs; r.d_grammar_row = grow;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((logits_fn)(uintptr_t)v[0])((void*)(uintptr_t)v[1], (int32_t)batch, (int32_t)slots, tok, mask, x, xs, &r,
                                    out, os, (void*)(uintptr_t)v[2]);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {{"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
                                {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, NULL},
                                {"logits", (PyCFunction)(void (*)(void))logits, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_numel = PyUnicode_InternFromString("numel");
  s_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  if (!s_dtype || !s_is_cuda || !s_numel || !s_contiguous || !s_data_ptr || !s_shape || !s_stride) return NULL;
  return PyModule_Create(&module);
}
