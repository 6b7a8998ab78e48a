/* binding.c -- the calls for candidate continuations and of a step over a cache in 8 bits from Python, without the cost of ctypes.
 *
 * These calls take a few microseconds on the GPU, less than what a Python function spends on
 * checking ten tensors and converting twenty arguments.  This module does the same in C: it
 * reads a tensor's type, shape, device and pointer through its Python attributes (no libtorch),
 * checks them, makes results and scratch and calls libpkv.
 *
 * torch.empty takes as long as such a call (5 us beside a launch on a Grace core), so small
 * results are made many at a time, away from the launches (1.4 us each), and handed out once each;
 * and scratch is kept per device, stream and call.  Work on one stream runs in order, and the GIL
 * is held while libpkv enqueues a call's kernels, so two calls never use one scratch at the same
 * time.  Where neither is safe -- while the stream is captured into a graph, whose
 * replays need memory of their own, or on a stream that the caller names -- both come from
 * torch.empty for that call alone, and for a named stream from that stream's memory: a block that
 * the allocator makes for the current stream may have a last user that still runs there.
 *
 * setup(path, torch, PkvError, ...) opens libpkv and keeps what is needed of torch.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>
#include <stdint.h>

#include "pkv.h"

typedef int64_t i64;

static struct {
  PyObject *empty, *error, *raw_stream, *current_device, *capturing, *ready, *empty_on;
  PyObject *results, *scratch; /* see take_result, take_scratch */
  PyObject *i32, *i64, *f32, *bf16, *u8, *e4m3, *boolean;
  PyObject *s_dtype, *s_shape, *s_data_ptr, *s_is_contiguous, *s_get_device, *s_stride, *s_cuda_stream,
      *s_view, *kw_empty;
  __typeof__(&paged_attention_tree) tree;
  __typeof__(&pkv_tree_workspace) tree_ws;
  __typeof__(&pkv_compact_path) compact;
  __typeof__(&pkv_beam_select) beam;
  __typeof__(&pkv_beam_workspace) beam_ws;
  __typeof__(&pkv_fork_tables) fork_;
  __typeof__(&pkv_fork_workspace) fork_ws;
  __typeof__(&pkv_rope_append) append;
  __typeof__(&paged_attention_q8) q8;
  __typeof__(&pkv_q8_workspace) q8_ws;
  __typeof__(&pkv_sample) sample;
} T;

/* A tensor argument: its shape, and (after check) its pointer. */
typedef struct {
  PyObject* t;
  const char* name;
  int dim;
  i64 n[5];
  void* ptr;
} Arg;

static int shape_of(Arg* a, PyObject* t, const char* name) {
  a->t = t;
  a->name = name;
  a->ptr = NULL;
  PyObject* s = PyObject_GetAttr(t, T.s_shape);
  if (!s) return 0;
  if (!PyTuple_Check(s)) {
    Py_DECREF(s);
    PyErr_Format(PyExc_ValueError, "%s must be a tensor", name);
    return 0;
  }
  const Py_ssize_t d = PyTuple_GET_SIZE(s);
  a->dim = d > 5 ? 6 : (int)d;
  for (Py_ssize_t i = 0; i < d && i < 5; ++i) a->n[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
  Py_DECREF(s);
  return !PyErr_Occurred();
}

static int is_dtype(PyObject* t, PyObject* dtype) {
  PyObject* d = PyObject_GetAttr(t, T.s_dtype);
  if (!d) return -1;
  const int same = d == dtype;
  Py_DECREF(d);
  return same;
}

/* A call's long result, or -2 with an exception set. */
static i64 call_long(PyObject* t, PyObject* name) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return -2;
  const i64 v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return v;
}

static int pointer(Arg* a) {
  PyObject* p = PyObject_CallMethodNoArgs(a->t, T.s_data_ptr);
  if (!p) return 0;
  a->ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}

/* The pointer of a contiguous tensor of this type on device dev. */
static int check(Arg* a, PyObject* dtype, i64 dev) {
  if (call_long(a->t, T.s_get_device) != dev) {
    if (!PyErr_Occurred())
      PyErr_Format(PyExc_ValueError, "%s must be a tensor on the current CUDA device (cuda:%lld)", a->name, (long long)dev);
    return 0;
  }
  const int same = is_dtype(a->t, dtype);
  if (same < 0) return 0;
  if (!same) {
    PyErr_Format(PyExc_ValueError, "%s must be %S", a->name, dtype);
    return 0;
  }
  PyObject* c = PyObject_CallMethodNoArgs(a->t, T.s_is_contiguous);
  if (!c) return 0;
  const int contiguous = c == Py_True;
  Py_DECREF(c);
  if (!contiguous) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", a->name);
    return 0;
  }
  return pointer(a);
}

static int refuse(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  return 0;
}

static int shaped(const Arg* a, int dim, i64 n0, i64 n1) {
  if (a->dim == dim && a->n[0] == n0 && (dim < 2 || a->n[1] == n1)) return 1;
  if (dim == 1) PyErr_Format(PyExc_ValueError, "%s must be [%lld]", a->name, (long long)n0);
  else PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld]", a->name, (long long)n0, (long long)n1);
  return 0;
}

/* Where a call runs: its device, its stream, and whether results and scratch may be kept ready. */
typedef struct {
  i64 dev;
  void* stream;
  PyObject* given; /* the caller's stream, or None */
  int keep;
} Place;

static int place(PyObject* stream, Place* w) {
  PyObject* d = PyObject_CallNoArgs(T.current_device);
  if (!d) return 0;
  w->dev = PyLong_AsLongLong(d);
  w->given = stream;
  PyObject* h = stream == Py_None ? PyObject_CallOneArg(T.raw_stream, d) : PyObject_GetAttr(stream, T.s_cuda_stream);
  Py_DECREF(d);
  if (!h) return 0;
  w->stream = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  PyObject* c = PyObject_CallNoArgs(T.capturing);
  if (!c) return 0;
  w->keep = stream == Py_None && c == Py_False;
  Py_DECREF(c);
  return !PyErr_Occurred();
}

/* torch.empty(shape, dtype=dtype, device=dev), for a given stream in that stream's memory; `shared`:
 * the current stream uses it too. */
static PyObject* made(int dim, const i64* n, PyObject* dtype, const Place* w, int shared) {
  PyObject* shape = PyTuple_New(dim);
  PyObject* d = PyLong_FromLongLong(w->dev);
  PyObject* r = NULL;
  if (shape && d) {
    for (int i = 0; i < dim; ++i) PyTuple_SET_ITEM(shape, i, PyLong_FromLongLong(n[i]));
    PyObject* args[5] = {shape, dtype, d, w->given, shared ? Py_True : Py_False};
    r = w->given == Py_None ? PyObject_Vectorcall(T.empty, args, 1, T.kw_empty) : PyObject_Vectorcall(T.empty_on, args, 5, NULL);
  }
  Py_XDECREF(shape);
  Py_XDECREF(d);
  return r;
}

/* A new tensor, those of up to 64 KB from a store of ready ones: per type, shape and stream a list of
 * how many to make next and those that are left.  The first call of a shape makes one, later ones
 * 8 and then 32, up to 256 KB: shapes that come once cost no more than torch.empty. */
static PyObject* take_result(int dim, const i64* n, PyObject* dtype, const Place* w) {
  enum { kMostReady = 32, kMostBytes = 65536, kMostKept = 262144 };
  i64 bytes = dtype == T.bf16 ? 2 : 4;
  for (int i = 0; i < dim; ++i) bytes = n[i] > kMostBytes ? kMostBytes + 1 : bytes * n[i];
  if (!w->keep || dim > 3 || bytes > kMostBytes || bytes <= 0) return made(dim, n, dtype, w, 1);
  struct {
    PyObject* dtype;
    void* stream;
    i64 dev, n[3];
  } key = {dtype, w->stream, w->dev, {n[0], dim > 1 ? n[1] : -1, dim > 2 ? n[2] : -1}};
  PyObject* k = PyBytes_FromStringAndSize((const char*)&key, sizeof key);
  if (!k) return NULL;
  PyObject* r = NULL;
  PyObject* ready = Py_XNewRef(PyDict_GetItemWithError(T.results, k)); /* (torch may let other threads run) */
  if (!ready && !PyErr_Occurred()) {
    if (PyDict_GET_SIZE(T.results) >= 512) PyDict_Clear(T.results);
    ready = Py_BuildValue("[i]", 1);
    if (ready && PyDict_SetItem(T.results, k, ready)) Py_CLEAR(ready);
  }
  Py_DECREF(k);
  if (!ready) return NULL;
  if (PyList_GET_SIZE(ready) == 1) {
    const long count = PyLong_AsLong(PyList_GET_ITEM(ready, 0));
    long next = count * 8 < kMostReady ? count * 8 : kMostReady;
    if (next * bytes > kMostKept) next = kMostKept / bytes;
    if (count == 1) {
      r = made(dim, n, dtype, w, 1);
    } else {
      PyObject* shape = dim == 1   ? Py_BuildValue("(L)", (long long)n[0])
                        : dim == 2 ? Py_BuildValue("(LL)", (long long)n[0], (long long)n[1])
                                   : Py_BuildValue("(LLL)", (long long)n[0], (long long)n[1], (long long)n[2]);
      PyObject* more = shape ? PyObject_CallFunction(T.ready, "lOOL", count, shape, dtype, (long long)w->dev) : NULL;
      if (more && PyList_GET_SIZE(more) > 0 && !PyList_SetSlice(ready, 1, 1, more)) {
        const Py_ssize_t last = PyList_GET_SIZE(ready) - 1;
        r = Py_NewRef(PyList_GET_ITEM(ready, last));
        if (PyList_SetSlice(ready, last, last + 1, NULL)) Py_CLEAR(r);
      }
      Py_XDECREF(more);
      Py_XDECREF(shape);
    }
    PyObject* number = PyLong_FromLong(next);
    if (!number || PyList_SetItem(ready, 0, number)) Py_CLEAR(r);
  } else {
    const Py_ssize_t last = PyList_GET_SIZE(ready) - 1;
    r = Py_NewRef(PyList_GET_ITEM(ready, last));
    if (PyList_SetSlice(ready, last, last + 1, NULL)) Py_CLEAR(r);
  }
  Py_DECREF(ready);
  return r;
}

/* Scratch of at least `bytes` for call number `call`. */
static PyObject* take_scratch(i64 bytes, int call, const Place* w) {
  if (bytes < 256) bytes = 256; /* (none is empty) */
  if (!w->keep) return made(1, &bytes, T.u8, w, 0);
  struct {
    void* stream;
    i64 dev, call;
  } key = {w->stream, w->dev, call};
  PyObject* k = PyBytes_FromStringAndSize((const char*)&key, sizeof key);
  if (!k) return NULL;
  PyObject* r = PyDict_GetItemWithError(T.scratch, k); /* (bytes, tensor), borrowed */
  if (r && PyLong_AsLongLong(PyTuple_GET_ITEM(r, 0)) >= bytes) {
    r = Py_NewRef(PyTuple_GET_ITEM(r, 1));
  } else if (PyErr_Occurred()) {
    r = NULL;
  } else {
    if (PyDict_GET_SIZE(T.scratch) >= 256) PyDict_Clear(T.scratch);
    r = made(1, &bytes, T.u8, w, 0);
    PyObject* entry = r ? Py_BuildValue("(LO)", (long long)bytes, r) : NULL;
    if (!entry || PyDict_SetItem(T.scratch, k, entry)) Py_CLEAR(r);
    Py_XDECREF(entry);
  }
  Py_DECREF(k);
  return r;
}

/* A result with its pointer: a given tensor of the right shape, checked, or a new one (a new
 * reference, also where the check fails; NULL: none could be made). */
static PyObject* result(Arg* a, PyObject* given, const char* name, int dim, const i64* n, PyObject* dtype, const Place* w, int* ok) {
  a->name = name;
  a->t = given == Py_None ? take_result(dim, n, dtype, w) : Py_NewRef(given);
  *ok = a->t && (given == Py_None ? pointer(a) : check(a, dtype, w->dev));
  return a->t;
}
/* The same for scratch, whose bytes a->n[0] tells afterwards. */
static PyObject* scratch(Arg* a, PyObject* given, i64 bytes, int call, const Place* w, int* ok) {
  if (given != Py_None) {
    *ok = shape_of(a, given, "workspace") && (a->dim < 1 || a->dim > 5 ? refuse("workspace must be a vector") : check(a, T.u8, w->dev));
    for (int i = 1; *ok && i < a->dim; ++i) a->n[0] *= a->n[i];
    return Py_NewRef(given);
  }
  a->t = take_scratch(bytes, call, w);
  a->n[0] = bytes;
  *ok = a->t && pointer(a);
  return a->t;
}

static PyObject* failed(int status, const char* what) {
  PyObject* e = PyObject_CallFunction(T.error, "is", status, what);
  if (e) {
    PyErr_SetObject(T.error, e);
    Py_DECREF(e);
  }
  return NULL;
}

/* Whether sizes fit the C entries' 32 bits. */
static int fit(i64 a, i64 b, i64 c) {
  return a <= INT32_MAX && b <= INT32_MAX && c <= INT32_MAX ? 1 : refuse("a size does not fit 32 bits");
}

/* The descriptor of one cache [blocks, Hkv, 16, d], or of a model's, [layers, ...]; `eight`: one in 8 bits will do. */
static int any_caches(Arg* k, Arg* v, int models, int eight, pkv_cache_desc* desc, i64* layers, PyObject** dtype) {
  int same = k->dim == v->dim;
  for (int i = 0; same && i < k->dim; ++i) same = k->n[i] == v->n[i];
  const int at = k->dim - 4;
  if (!same || at < 0 || at > models || (at == 1 && k->n[0] < 1))
    return refuse("k_cache and v_cache must both be [num_blocks, num_kv_heads, 16, head_dim]");
  const int f32 = is_dtype(k->t, T.f32), bf16 = f32 ? 0 : is_dtype(k->t, T.bf16);
  if (f32 < 0 || bf16 < 0) return 0;
  const int u8 = f32 || bf16 || !eight ? 0 : is_dtype(k->t, T.u8), e4m3 = f32 || bf16 || u8 || !eight ? 0 : is_dtype(k->t, T.e4m3);
  if (u8 < 0 || e4m3 < 0) return 0;
  if (!f32 && !bf16 && !u8 && !e4m3) return refuse("unsupported cache dtype");
  *dtype = f32 ? T.f32 : bf16 ? T.bf16 : u8 ? T.u8 : T.e4m3;
  if (!fit(k->n[at + 1], k->n[at + 2], k->n[at + 3])) return 0;
  *layers = at == 1 ? k->n[0] : 1;
  desc->num_blocks = k->n[at];
  desc->num_kv_heads = (int32_t)k->n[at + 1];
  desc->block_size = (int32_t)k->n[at + 2];
  desc->head_dim = (int32_t)k->n[at + 3];
  desc->dtype = f32 ? PKV_F32 : bf16 ? PKV_BF16 : PKV_E4M3;
  return 1;
}
static int caches(Arg* k, Arg* v, int models, pkv_cache_desc* desc, i64* layers, PyObject** dtype) {
  return any_caches(k, v, models, 0, desc, layers, dtype);
}

static int requests(const Arg* bt, const Arg* lens, const Arg* qsl) {
  if (lens->dim != 1 || bt->dim != 2 || bt->n[0] != lens->n[0] || qsl->dim != 1 || qsl->n[0] != lens->n[0] + 1)
    return refuse("block_tables, seq_lens and query_start_loc disagree on the number of requests");
  return 1;
}

static int want(Py_ssize_t n, Py_ssize_t should) {
  if (n == should) return 1;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", should, n);
  return 0;
}

/* Numbers of a call; -1 with an exception where one is none. */
static int as_int32(PyObject* o, int32_t* v) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) return 0;
  if (x != (int32_t)x) return refuse("a size does not fit 32 bits");
  *v = (int32_t)x;
  return 1;
}

/* (q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, tree_mask, scale, max_query_len, max_seq_len, out,
 *  workspace, stream) */
static PyObject* py_tree(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Arg q, k, v, bt, lens, qsl, mask, o, w;
  pkv_cache_desc desc;
  PyObject *dt, *out = NULL, *ws = NULL, *res = NULL;
  i64 layers, bytes = 0;
  Place at;
  int32_t max_q, max_len;
  int ok;
  if (!want(n, 13)) return NULL;
  if (!shape_of(&k, a[1], "k_cache") || !shape_of(&v, a[2], "v_cache") || !caches(&k, &v, 0, &desc, &layers, &dt)) return NULL;
  if (!shape_of(&q, a[0], "q")) return NULL;
  if (q.dim != 3 || q.n[2] != desc.head_dim) return refuse("q must be [num_tokens, num_q_heads, head_dim]"), NULL;
  if (!shape_of(&mask, a[6], "tree_mask")) return NULL;
  if (mask.dim != 2 || mask.n[0] != q.n[0]) return refuse("tree_mask must be int64 [num_tokens, words]"), NULL;
  if (!shape_of(&bt, a[3], "block_tables") || !shape_of(&lens, a[4], "seq_lens") || !shape_of(&qsl, a[5], "query_start_loc") ||
      !requests(&bt, &lens, &qsl))
    return NULL;
  if (a[10] != Py_None) {
    if (!shape_of(&o, a[10], "out")) return NULL;
    if (o.dim != 3 || o.n[0] != q.n[0] || o.n[1] != q.n[1] || o.n[2] != q.n[2]) return refuse("out must have the shape of q"), NULL;
  }
  if (!fit(q.n[1], bt.n[1], mask.n[1]) || !fit(lens.n[0], 0, 0)) return NULL;
  const double scale = PyFloat_AsDouble(a[7]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  if (!as_int32(a[8], &max_q) || !as_int32(a[9], &max_len)) return NULL;
  if (!place(a[12], &at)) return NULL;
  if (!check(&q, dt, at.dev) || !check(&k, dt, at.dev) || !check(&v, dt, at.dev) || !check(&bt, T.i32, at.dev) || !check(&lens, T.i32, at.dev) ||
      !check(&qsl, T.i32, at.dev) || !check(&mask, T.i64, at.dev))
    return NULL;
  out = result(&o, a[10], "out", 3, q.n, dt, &at, &ok);
  if (!ok) goto end;
  if (q.n[0] == 0) {
    res = Py_NewRef(out);
    goto end;
  }
  if (a[11] == Py_None) {
    const int st = T.tree_ws(&desc, (int32_t)q.n[1], max_q, &bytes);
    if (st) {
      failed(st, "paged_attention_tree");
      goto end;
    }
  }
  ws = scratch(&w, a[11], bytes, 0, &at, &ok);
  if (!ok) goto end;
  const int st = T.tree(q.ptr, k.ptr, v.ptr, &desc, bt.ptr, (int32_t)bt.n[1], lens.ptr, qsl.ptr, mask.ptr, (int32_t)mask.n[1],
                        (int32_t)lens.n[0], (int32_t)q.n[1], q.n[0], max_q, max_len, (float)scale, o.ptr, w.ptr, w.n[0], at.stream);
  res = st ? failed(st, "paged_attention_tree") : Py_NewRef(out);
end:
  Py_XDECREF(out);
  Py_XDECREF(ws);
  return res;
}

/* (path, path_lens, block_tables, seq_lens, query_start_loc, k_cache, v_cache, new_seq_lens, stream) */
static PyObject* py_compact(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Arg path, plens, bt, lens, qsl, k, v, o;
  pkv_cache_desc desc;
  PyObject *dt, *out = NULL, *res = NULL;
  i64 layers;
  Place at;
  int ok;
  if (!want(n, 9)) return NULL;
  if (!shape_of(&k, a[5], "k_cache") || !shape_of(&v, a[6], "v_cache") || !caches(&k, &v, 1, &desc, &layers, &dt)) return NULL;
  if (!shape_of(&bt, a[2], "block_tables") || !shape_of(&lens, a[3], "seq_lens") || !shape_of(&qsl, a[4], "query_start_loc") ||
      !requests(&bt, &lens, &qsl))
    return NULL;
  if (!shape_of(&path, a[0], "path") || !shape_of(&plens, a[1], "path_lens")) return NULL;
  if (path.dim != 2 || path.n[0] != lens.n[0] || plens.dim != 1 || plens.n[0] != lens.n[0])
    return refuse("path must be [num_seqs, max_path], path_lens [num_seqs]"), NULL;
  if (!fit(path.n[1], bt.n[1], lens.n[0]) || !fit(layers, 0, 0)) return NULL;
  if (a[7] != Py_None && (!shape_of(&o, a[7], "new_seq_lens") || !shaped(&o, 1, lens.n[0], 0))) return NULL;
  if (!place(a[8], &at)) return NULL;
  if (!check(&path, T.i32, at.dev) || !check(&plens, T.i32, at.dev) || !check(&bt, T.i32, at.dev) || !check(&lens, T.i32, at.dev) ||
      !check(&qsl, T.i32, at.dev) || !check(&k, dt, at.dev) || !check(&v, dt, at.dev))
    return NULL;
  out = result(&o, a[7], "new_seq_lens", 1, lens.n, T.i32, &at, &ok);
  if (!ok) goto end;
  const int st = T.compact(path.ptr, (int32_t)path.n[1], plens.ptr, bt.ptr, (int32_t)bt.n[1], lens.ptr, qsl.ptr,
                           (int32_t)lens.n[0], k.ptr, v.ptr, &desc, (int32_t)layers, o.ptr, at.stream);
  res = st ? failed(st, "pkv_compact_path") : Py_NewRef(out);
end:
  Py_XDECREF(out);
  return res;
}

/* (logits, cum_scores, num_select, finished, eos_token, out, workspace, stream) */
static PyObject* py_beam(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Arg x, cum, fin, r[3], w;
  PyObject *out[3] = {NULL, NULL, NULL}, *ws = NULL, *res = NULL, *done = NULL;
  PyObject* const types[3] = {T.f32, T.i32, T.i32};
  static const char* const names[3] = {"scores", "parents", "tokens"};
  i64 bytes = 0;
  Place at;
  int32_t K, eos;
  int ok;
  if (!want(n, 8)) return NULL;
  if (!shape_of(&x, a[0], "logits")) return NULL;
  if (x.dim != 3) return refuse("logits must be [num_seqs, num_beams, vocab]"), NULL;
  const i64 N = x.n[0], W = x.n[1], V = x.n[2];
  if (!fit(N, W, V)) return NULL;
  const int f32 = is_dtype(x.t, T.f32), bf16 = f32 ? 0 : is_dtype(x.t, T.bf16);
  if (f32 < 0 || bf16 < 0) return NULL;
  if (!f32 && !bf16) return refuse("logits must be float32 or bfloat16"), NULL;
  i64 step = V;
  PyObject* c = PyObject_CallMethodNoArgs(x.t, T.s_is_contiguous);
  if (!c) return NULL;
  const int contiguous = c == Py_True;
  Py_DECREF(c);
  if (!contiguous && N * W * V > 0) {
    PyObject* st = PyObject_CallMethodNoArgs(x.t, T.s_stride);
    if (!st) return NULL;
    i64 d[3] = {0, 0, 0};
    for (int i = 0; i < 3 && PyTuple_Check(st) && i < PyTuple_GET_SIZE(st); ++i) d[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    Py_DECREF(st);
    if (PyErr_Occurred()) return NULL;
    step = W > 1 ? d[1] : N > 1 ? d[0] : V;
    if ((V > 1 && d[2] != 1) || (N > 1 && d[0] != W * step) || step < V)
      return refuse("logits must have contiguous rows, evenly spaced"), NULL;
  }
  if (!shape_of(&cum, a[1], "cum_scores") || !shaped(&cum, 2, N, W)) return NULL;
  if (a[3] != Py_None && (!shape_of(&fin, a[3], "finished") || !shaped(&fin, 2, N, W))) return NULL;
  if (!as_int32(a[2], &K) || !as_int32(a[4], &eos)) return NULL;
  const i64 shape[2] = {N, K < 0 ? 0 : K};
  if (a[5] != Py_None) {
    if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 3) return refuse("out must be (scores, parents, tokens)"), NULL;
    for (int i = 0; i < 3; ++i)
      if (!shape_of(&r[i], PyTuple_GET_ITEM(a[5], i), names[i]) || !shaped(&r[i], 2, N, K)) return NULL;
  }
  if (!place(a[7], &at)) return NULL;
  if (call_long(x.t, T.s_get_device) != at.dev) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "logits must be a tensor on the current CUDA device (cuda:%lld)", (long long)at.dev);
    return NULL;
  }
  PyObject* p = PyObject_CallMethodNoArgs(x.t, T.s_data_ptr);
  if (!p) return NULL;
  x.ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  if (!check(&cum, T.f32, at.dev)) return NULL;
  fin.ptr = NULL;
  if (a[3] != Py_None) {
    const int b = is_dtype(a[3], T.boolean);
    if (b < 0) return NULL;
    done = b ? PyObject_CallMethodOneArg(a[3], T.s_view, T.u8) : Py_NewRef(a[3]);
    fin.t = done;
    if (!done || !check(&fin, T.u8, at.dev)) goto end;
  }
  if (a[6] == Py_None) {
    const int st = T.beam_ws((int32_t)N, (int32_t)W, (int32_t)V, K, &bytes);
    if (st) {
      failed(st, "pkv_beam_select");
      goto end;
    }
  }
  for (int i = 0; i < 3; ++i) {
    out[i] = result(&r[i], a[5] == Py_None ? Py_None : PyTuple_GET_ITEM(a[5], i), names[i], 2, shape, types[i], &at, &ok);
    if (!ok) goto end;
  }
  ws = scratch(&w, a[6], bytes, 1, &at, &ok);
  if (!ok) goto end;
  const int st = T.beam(x.ptr, f32 ? PKV_F32 : PKV_BF16, step, cum.ptr, fin.ptr, eos, (int32_t)N, (int32_t)W, (int32_t)V, K,
                        r[0].ptr, r[1].ptr, r[2].ptr, w.ptr, w.n[0], at.stream);
  res = st ? failed(st, "pkv_beam_select") : PyTuple_Pack(3, out[0], out[1], out[2]);
end:
  for (int i = 0; i < 3; ++i) Py_XDECREF(out[i]);
  Py_XDECREF(ws);
  Py_XDECREF(done);
  return res;
}

/* (block_tables, seq_lens, parents, ref_counts, k_cache, v_cache, new_tokens, out, workspace, stream) */
static PyObject* py_fork(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Arg bt, lens, par, refs, k, v, obt, olens, w;
  pkv_cache_desc desc = {0, PKV_BLOCK_SIZE, 1, 128, PKV_BF16};
  PyObject *dt = NULL, *tables = NULL, *nlens = NULL, *ws = NULL, *res = NULL;
  i64 layers = 1, bytes = 0;
  Place at;
  int32_t num_new;
  int ok;
  if (!want(n, 10)) return NULL;
  if (!shape_of(&bt, a[0], "block_tables")) return NULL;
  if (bt.dim != 2) return refuse("block_tables must be [num_rows, max_blocks_per_seq]"), NULL;
  if (!fit(bt.n[0], bt.n[1], 0)) return NULL;
  const int data = a[4] != Py_None;
  if (data != (a[5] != Py_None)) return refuse("k_cache and v_cache must be given together"), NULL;
  if (!shape_of(&refs, a[3], "ref_counts")) return NULL;
  if (data) {
    if (!shape_of(&k, a[4], "k_cache") || !shape_of(&v, a[5], "v_cache") || !caches(&k, &v, 1, &desc, &layers, &dt)) return NULL;
  } else if (refs.dim == 1) {
    desc.num_blocks = refs.n[0];
  }
  if (!fit(layers, 0, 0)) return NULL;
  if (refs.dim != 1 || refs.n[0] != desc.num_blocks) return refuse("ref_counts must be [num_blocks] of the cache"), NULL;
  if (!shape_of(&lens, a[1], "seq_lens") || !shaped(&lens, 1, bt.n[0], 0)) return NULL;
  if (!shape_of(&par, a[2], "parents") || !shaped(&par, 1, bt.n[0], 0)) return NULL;
  if (a[7] != Py_None) {
    if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 2) return refuse("out must be (block tables, lengths)"), NULL;
    if (!shape_of(&obt, PyTuple_GET_ITEM(a[7], 0), "new tables") || !shaped(&obt, 2, bt.n[0], bt.n[1]) ||
        !shape_of(&olens, PyTuple_GET_ITEM(a[7], 1), "new lengths") || !shaped(&olens, 1, bt.n[0], 0))
      return NULL;
  }
  if (!as_int32(a[6], &num_new)) return NULL;
  if (!place(a[9], &at)) return NULL;
  if (!check(&bt, T.i32, at.dev) || !check(&lens, T.i32, at.dev) || !check(&par, T.i32, at.dev) || !check(&refs, T.i32, at.dev)) return NULL;
  if (data && (!check(&k, dt, at.dev) || !check(&v, dt, at.dev))) return NULL;
  tables = result(&obt, a[7] == Py_None ? Py_None : PyTuple_GET_ITEM(a[7], 0), "new tables", 2, bt.n, T.i32, &at, &ok);
  if (!ok) goto end;
  nlens = result(&olens, a[7] == Py_None ? Py_None : PyTuple_GET_ITEM(a[7], 1), "new lengths", 1, bt.n, T.i32, &at, &ok);
  if (!ok) goto end;
  if (a[8] == Py_None) {
    const int st = T.fork_ws((int32_t)bt.n[0], &bytes);
    if (st) {
      failed(st, "pkv_fork_tables");
      goto end;
    }
  }
  ws = scratch(&w, a[8], bytes, 2, &at, &ok);
  if (!ok) goto end;
  const int st = T.fork_(bt.ptr, lens.ptr, (int32_t)bt.n[0], (int32_t)bt.n[1], par.ptr, num_new, refs.ptr, obt.ptr, olens.ptr,
                         data ? k.ptr : NULL, data ? v.ptr : NULL, &desc, (int32_t)layers, w.ptr, w.n[0], at.stream);
  res = st ? failed(st, "pkv_fork_tables") : PyTuple_Pack(2, tables, nlens);
end:
  Py_XDECREF(tables);
  Py_XDECREF(nlens);
  Py_XDECREF(ws);
  return res;
}

/* The strides of a tensor that is not contiguous (up to three). */
static int strides(PyObject* t, i64* d) {
  PyObject* st = PyObject_CallMethodNoArgs(t, T.s_stride);
  if (!st) return 0;
  d[0] = d[1] = d[2] = 0;
  for (int i = 0; i < 3 && PyTuple_Check(st) && i < PyTuple_GET_SIZE(st); ++i) d[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
  Py_DECREF(st);
  return !PyErr_Occurred();
}

static int on_device(const Arg* a, i64 dev) {
  if (call_long(a->t, T.s_get_device) == dev) return 1;
  if (!PyErr_Occurred())
    PyErr_Format(PyExc_ValueError, "%s must be a tensor on the current CUDA device (cuda:%lld)", a->name, (long long)dev);
  return 0;
}

/* The pointer of a [tokens, heads, d] tensor whose tokens may lie apart, and how far (elements). */
static int token_rows(Arg* a, PyObject* dtype, i64 dev, i64* step) {
  i64 s[3];
  if (!on_device(a, dev)) return 0;
  const int same = is_dtype(a->t, dtype);
  if (same < 0) return 0;
  if (!same) {
    PyErr_Format(PyExc_ValueError, "%s must be %S", a->name, dtype);
    return 0;
  }
  if (!strides(a->t, s)) return 0;
  const i64 width = a->n[1] * a->n[2];
  *step = a->n[0] > 1 ? s[0] : width;
  if ((a->n[2] > 1 && s[2] != 1) || (a->n[1] > 1 && s[1] != a->n[2]) || *step < width) {
    PyErr_Format(PyExc_ValueError, "%s must have tokens of contiguous heads", a->name);
    return 0;
  }
  return pointer(a);
}

/* (k, v, cos_sin, k_cache, v_cache, block_tables, seq_lens, query_start_loc, max_query_len, q, scales, positions, interleaved,
 *  q_out, stream) */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Arg k, v, angles, kc, vc, bt, lens, qsl, q, scales, pos, o;
  pkv_cache_desc desc;
  PyObject *dt, *out = NULL, *res = NULL;
  i64 layers, k_step, v_step, q_step = 0, o_step = 0;
  Place at;
  int32_t max_q;
  int ok;
  if (!want(n, 15)) return NULL;
  if (!shape_of(&kc, a[3], "k_cache") || !shape_of(&vc, a[4], "v_cache") || !any_caches(&kc, &vc, 0, 1, &desc, &layers, &dt)) return NULL;
  const int eight = desc.dtype == PKV_E4M3;
  PyObject* rows = eight ? T.bf16 : dt;
  if (!shape_of(&k, a[0], "k") || !shape_of(&v, a[1], "v")) return NULL;
  if (k.dim != 3 || k.n[1] != desc.num_kv_heads || k.n[2] != desc.head_dim || v.dim != 3 || v.n[0] != k.n[0] || v.n[1] != k.n[1] ||
      v.n[2] != k.n[2])
    return refuse("k and v must both be [num_tokens, num_kv_heads, head_dim]"), NULL;
  const int has_q = a[9] != Py_None, turns = a[2] != Py_None;
  if (has_q) {
    if (!shape_of(&q, a[9], "q")) return NULL;
    if (q.dim != 3 || q.n[0] != k.n[0] || q.n[2] != k.n[2]) return refuse("q must be [num_tokens, num_q_heads, head_dim]"), NULL;
    if (!fit(q.n[1], 0, 0)) return NULL;
  }
  if (a[13] != Py_None) {
    if (!has_q) return refuse("q_out without q"), NULL;
    if (!shape_of(&o, a[13], "q_out")) return NULL;
    if (o.dim != 3 || o.n[0] != q.n[0] || o.n[1] != q.n[1] || o.n[2] != q.n[2]) return refuse("q_out must have the shape of q"), NULL;
  }
  if (turns) {
    if (!shape_of(&angles, a[2], "cos_sin")) return NULL;
    if (angles.dim != 2) return refuse("cos_sin must be [num_angles, rot_dim]"), NULL;
    if (!fit(angles.n[1], 0, 0)) return NULL;
  }
  if (eight != (a[10] != Py_None)) return refuse("scales belong to a cache in 8 bits"), NULL;
  if (eight) {
    if (!shape_of(&scales, a[10], "scales")) return NULL;
    if (scales.dim != 3 || scales.n[0] != desc.num_blocks || scales.n[1] != desc.num_kv_heads || scales.n[2] != 2)
      return refuse("scales must be [num_blocks, num_kv_heads, 2]"), NULL;
  }
  if (a[11] != Py_None && (!shape_of(&pos, a[11], "positions") || !shaped(&pos, 1, k.n[0], 0))) return NULL;
  if (!shape_of(&bt, a[5], "block_tables") || !shape_of(&lens, a[6], "seq_lens") || !shape_of(&qsl, a[7], "query_start_loc") ||
      !requests(&bt, &lens, &qsl))
    return NULL;
  if (!fit(bt.n[1], lens.n[0], 0) || !as_int32(a[8], &max_q)) return NULL;
  const int interleaved = PyObject_IsTrue(a[12]);
  if (interleaved < 0 || !place(a[14], &at)) return NULL;
  if (!token_rows(&k, rows, at.dev, &k_step) || !token_rows(&v, rows, at.dev, &v_step) || !check(&kc, dt, at.dev) || !check(&vc, dt, at.dev) ||
      !check(&bt, T.i32, at.dev) || !check(&lens, T.i32, at.dev) || !check(&qsl, T.i32, at.dev))
    return NULL;
  if (has_q && !token_rows(&q, rows, at.dev, &q_step)) return NULL;
  if (turns && !check(&angles, T.f32, at.dev)) return NULL;
  if (eight && !check(&scales, T.f32, at.dev)) return NULL;
  if (a[11] != Py_None && !check(&pos, T.i32, at.dev)) return NULL;
  if (!has_q) {
    out = Py_NewRef(Py_None);
  } else if (a[13] == Py_None) {
    out = result(&o, Py_None, "q_out", 3, q.n, rows, &at, &ok);
    if (!ok) goto end;
    o_step = q.n[1] * q.n[2];
  } else {
    out = Py_NewRef(a[13]);
    if (!token_rows(&o, rows, at.dev, &o_step)) goto end;
  }
  const int st = T.append(has_q ? q.ptr : NULL, k.ptr, v.ptr, rows == T.f32 ? PKV_F32 : PKV_BF16, q_step, k_step, v_step,
                          has_q ? (int32_t)q.n[1] : 0, turns ? angles.ptr : NULL, turns ? (int32_t)angles.n[1] : 0, interleaved,
                          turns ? angles.n[0] : 0, a[11] != Py_None ? pos.ptr : NULL, kc.ptr, vc.ptr, eight ? scales.ptr : NULL, &desc,
                          bt.ptr, (int32_t)bt.n[1], lens.ptr, qsl.ptr, (int32_t)lens.n[0], k.n[0], max_q, has_q ? o.ptr : NULL, o_step,
                          at.stream);
  res = st ? failed(st, "pkv_rope_append") : Py_NewRef(out);
end:
  Py_XDECREF(out);
  return res;
}

/* (q, k_cache, v_cache, scales, block_tables, seq_lens, query_start_loc, scale, max_query_len, max_seq_len, out, workspace, stream) */
static PyObject* py_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Arg q, k, v, scales, bt, lens, qsl, o, w;
  pkv_cache_desc desc;
  PyObject *dt, *out = NULL, *ws = NULL, *res = NULL;
  i64 layers, bytes = 0;
  Place at;
  int32_t max_q, max_len;
  int ok;
  if (!want(n, 13)) return NULL;
  if (!shape_of(&k, a[1], "k_cache") || !shape_of(&v, a[2], "v_cache") || !any_caches(&k, &v, 0, 1, &desc, &layers, &dt)) return NULL;
  if (desc.dtype != PKV_E4M3) return refuse("the cache must be in 8 bits (uint8 or float8_e4m3fn)"), NULL;
  if (!shape_of(&q, a[0], "q")) return NULL;
  if (q.dim != 3 || q.n[2] != desc.head_dim) return refuse("q must be [num_tokens, num_q_heads, head_dim]"), NULL;
  if (!shape_of(&scales, a[3], "scales")) return NULL;
  if (scales.dim != 3 || scales.n[0] != desc.num_blocks || scales.n[1] != desc.num_kv_heads || scales.n[2] != 2)
    return refuse("scales must be [num_blocks, num_kv_heads, 2]"), NULL;
  if (!shape_of(&bt, a[4], "block_tables") || !shape_of(&lens, a[5], "seq_lens") || !shape_of(&qsl, a[6], "query_start_loc") ||
      !requests(&bt, &lens, &qsl))
    return NULL;
  if (a[10] != Py_None) {
    if (!shape_of(&o, a[10], "out")) return NULL;
    if (o.dim != 3 || o.n[0] != q.n[0] || o.n[1] != q.n[1] || o.n[2] != q.n[2]) return refuse("out must have the shape of q"), NULL;
  }
  if (!fit(q.n[1], bt.n[1], lens.n[0])) return NULL;
  const double scale = PyFloat_AsDouble(a[7]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  if (!as_int32(a[8], &max_q) || !as_int32(a[9], &max_len)) return NULL;
  if (!place(a[12], &at)) return NULL;
  if (!check(&q, T.bf16, at.dev) || !check(&k, dt, at.dev) || !check(&v, dt, at.dev) || !check(&scales, T.f32, at.dev) ||
      !check(&bt, T.i32, at.dev) || !check(&lens, T.i32, at.dev) || !check(&qsl, T.i32, at.dev))
    return NULL;
  out = result(&o, a[10], "out", 3, q.n, T.bf16, &at, &ok);
  if (!ok) goto end;
  if (q.n[0] == 0) {
    res = Py_NewRef(out);
    goto end;
  }
  if (a[11] == Py_None) {
    const int st = T.q8_ws(&desc, (int32_t)q.n[1], max_q, &bytes);
    if (st) {
      failed(st, "paged_attention_q8");
      goto end;
    }
  }
  ws = scratch(&w, a[11], bytes, 3, &at, &ok);
  if (!ok) goto end;
  const int st = T.q8(q.ptr, k.ptr, v.ptr, scales.ptr, &desc, bt.ptr, (int32_t)bt.n[1], lens.ptr, qsl.ptr, (int32_t)lens.n[0],
                      (int32_t)q.n[1], q.n[0], max_q, max_len, (float)scale, o.ptr, w.ptr, w.n[0], at.stream);
  res = st ? failed(st, "paged_attention_q8") : Py_NewRef(out);
end:
  Py_XDECREF(out);
  Py_XDECREF(ws);
  return res;
}

/* (logits, uniform, temperature, top_k, top_p, min_p, out, stream) */
static PyObject* py_sample(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Arg x, s[5], r[2]; /* s: uniform, temperature, top_k, top_p, min_p */
  static const char* const settings[5] = {"uniform", "temperature", "top_k", "top_p", "min_p"};
  static const char* const names[2] = {"tokens", "logprobs"};
  PyObject* const types[2] = {T.i32, T.f32};
  PyObject *out[2] = {NULL, NULL}, *res = NULL;
  Place at;
  int ok;
  if (!want(n, 8)) return NULL;
  if (!shape_of(&x, a[0], "logits")) return NULL;
  if (x.dim != 2) return refuse("logits must be [num_seqs, vocab]"), NULL;
  const i64 N = x.n[0], V = x.n[1];
  if (!fit(N, V, 0)) return NULL;
  const int f32 = is_dtype(x.t, T.f32), bf16 = f32 ? 0 : is_dtype(x.t, T.bf16);
  if (f32 < 0 || bf16 < 0) return NULL;
  if (!f32 && !bf16) return refuse("logits must be float32 or bfloat16"), NULL;
  i64 d[3];
  if (!strides(x.t, d)) return NULL;
  const i64 step = N > 1 ? d[0] : V;
  if ((V > 1 && d[1] != 1) || (N > 1 && step < V)) return refuse("logits must have contiguous rows, evenly spaced"), NULL;
  for (int i = 0; i < 5; ++i) {
    s[i].ptr = NULL;
    if ((i == 0 || a[i + 1] != Py_None) && (!shape_of(&s[i], a[i + 1], settings[i]) || !shaped(&s[i], 1, N, 0))) return NULL;
  }
  if (a[6] != Py_None) {
    if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 2) return refuse("out must be (tokens, logprobs)"), NULL;
    for (int i = 0; i < 2; ++i)
      if (!shape_of(&r[i], PyTuple_GET_ITEM(a[6], i), names[i]) || !shaped(&r[i], 1, N, 0)) return NULL;
  }
  if (!place(a[7], &at)) return NULL;
  if (!on_device(&x, at.dev) || !pointer(&x)) return NULL;
  for (int i = 0; i < 5; ++i)
    if ((i == 0 || a[i + 1] != Py_None) && !check(&s[i], i == 2 ? T.i32 : T.f32, at.dev)) return NULL;
  for (int i = 0; i < 2; ++i) {
    out[i] = result(&r[i], a[6] == Py_None ? Py_None : PyTuple_GET_ITEM(a[6], i), names[i], 1, &N, types[i], &at, &ok);
    if (!ok) goto end;
  }
  const int st = T.sample(x.ptr, f32 ? PKV_F32 : PKV_BF16, step, s[1].ptr, s[2].ptr, s[3].ptr, s[4].ptr, s[0].ptr, (int32_t)N,
                          (int32_t)V, r[0].ptr, r[1].ptr, at.stream);
  res = st ? failed(st, "pkv_sample") : PyTuple_Pack(2, out[0], out[1]);
end:
  for (int i = 0; i < 2; ++i) Py_XDECREF(out[i]);
  return res;
}

/* (path of libpkv, torch, PkvError, torch.cuda.current_device, a function from a device to its raw stream, one that tells
 * whether the current stream is captured, one that makes results: (number, shape, type, device) -> list, one that makes a
 * tensor for a named stream: (shape, type, device, stream, shared)) */
static PyObject* py_setup(PyObject* self, PyObject* args) {
  const char* path;
  PyObject* torch;
  if (!PyArg_ParseTuple(args, "sOOOOOOO", &path, &torch, &T.error, &T.current_device, &T.raw_stream, &T.capturing, &T.ready, &T.empty_on))
    return NULL;
  void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return NULL;
  }
#define SYMBOL(field, name)                                                   \
  if (!(T.field = (__typeof__(T.field))dlsym(h, #name))) {                    \
    PyErr_SetString(PyExc_ImportError, "libpkv does not export " #name);      \
    return NULL;                                                              \
  }
  SYMBOL(tree, paged_attention_tree)
  SYMBOL(tree_ws, pkv_tree_workspace)
  SYMBOL(compact, pkv_compact_path)
  SYMBOL(beam, pkv_beam_select)
  SYMBOL(beam_ws, pkv_beam_workspace)
  SYMBOL(fork_, pkv_fork_tables)
  SYMBOL(fork_ws, pkv_fork_workspace)
  SYMBOL(append, pkv_rope_append)
  SYMBOL(q8, paged_attention_q8)
  SYMBOL(q8_ws, pkv_q8_workspace)
  SYMBOL(sample, pkv_sample)
#undef SYMBOL
  Py_INCREF(T.error);
  Py_INCREF(T.current_device);
  Py_INCREF(T.raw_stream);
  Py_INCREF(T.capturing);
  Py_INCREF(T.ready);
  Py_INCREF(T.empty_on);
  if (!(T.results = PyDict_New()) || !(T.scratch = PyDict_New())) return NULL;
  if (!(T.empty = PyObject_GetAttrString(torch, "empty")) || !(T.i32 = PyObject_GetAttrString(torch, "int32")) ||
      !(T.i64 = PyObject_GetAttrString(torch, "int64")) || !(T.f32 = PyObject_GetAttrString(torch, "float32")) ||
      !(T.bf16 = PyObject_GetAttrString(torch, "bfloat16")) || !(T.u8 = PyObject_GetAttrString(torch, "uint8")) ||
      !(T.e4m3 = PyObject_GetAttrString(torch, "float8_e4m3fn")) ||
      !(T.boolean = PyObject_GetAttrString(torch, "bool")))
    return NULL;
  T.s_dtype = PyUnicode_InternFromString("dtype");
  T.s_shape = PyUnicode_InternFromString("shape");
  T.s_data_ptr = PyUnicode_InternFromString("data_ptr");
  T.s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  T.s_get_device = PyUnicode_InternFromString("get_device");
  T.s_stride = PyUnicode_InternFromString("stride");
  T.s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  T.s_view = PyUnicode_InternFromString("view");
  T.kw_empty = Py_BuildValue("(ss)", "dtype", "device");
  Py_RETURN_NONE;
}

/* Lets go of the ready results and of the scratch.  (Torch hands their memory out again in the order of the streams
 * that use it, so calls that still run keep theirs.) */
static PyObject* py_release(PyObject* self, PyObject* none) {
  if (T.results) PyDict_Clear(T.results);
  if (T.scratch) PyDict_Clear(T.scratch);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, NULL},
                                {"release", py_release, METH_NOARGS, NULL},
                                {"tree", (PyCFunction)(void*)py_tree, METH_FASTCALL, NULL},
                                {"compact", (PyCFunction)(void*)py_compact, METH_FASTCALL, NULL},
                                {"beam", (PyCFunction)(void*)py_beam, METH_FASTCALL, NULL},
                                {"fork", (PyCFunction)(void*)py_fork, METH_FASTCALL, NULL},
                                {"append", (PyCFunction)(void*)py_append, METH_FASTCALL, NULL},
                                {"q8", (PyCFunction)(void*)py_q8, METH_FASTCALL, NULL},
                                {"sample", (PyCFunction)(void*)py_sample, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
