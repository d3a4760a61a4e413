// The way from Python to the calls of the target's side of a step.  A kernel for a single token runs
// for 3 us, and checking 15 tensors in Python and converting 35 arguments took 10: here a
// well-formed call's tensors are asked for what the C ABI needs (type, device, shape, strides,
// address) and passed on.  Whatever is not as it should be, or is to be allocated, is left to the
// Python form of the same checks, which says what is wrong: a function returns the call's status, or
// None for "not checked here".
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include "../../include/dspark.h"

namespace {

decltype(&dspark_cache_append) append_fn;
decltype(&dspark_tree_attention) attend_fn;
decltype(&dspark_tree_verify) verify_fn;
decltype(&dspark_cache_keep) keep_fn;
PyObject *f32, *bf16, *f16, *i32, *get_device_fn, *get_stream_fn;
PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_numel, *s_device, *s_contiguous, *s_ptr, *s_nbytes, *s_buf,
    *s_key, *s_k;

bool number(PyObject* owned, int64_t* out) {             // takes the reference
  if (!owned) return false;
  const bool is = PyLong_Check(owned);
  *out = is ? PyLong_AsLongLong(owned) : 0;
  Py_DECREF(owned);
  return is && !PyErr_Occurred();
}
bool method(PyObject* t, PyObject* name, int64_t* out) {
  PyObject* args[1] = {t};
  return number(PyObject_VectorcallMethod(name, args, 1, nullptr), out);
}
bool is_type(PyObject* t, PyObject* dtype) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  Py_XDECREF(d);                                         // (the types outlive it)
  return d == dtype;
}
bool is_contiguous(PyObject* t) {
  PyObject* args[1] = {t};
  PyObject* r = PyObject_VectorcallMethod(s_contiguous, args, 1, nullptr);
  Py_XDECREF(r);
  return r == Py_True;
}

struct Dims {
  int n = 0;
  int64_t v[6];
  bool take(PyObject* tuple) {                           // takes the reference
    bool ok = tuple && PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) <= 6;
    n = ok ? (int)PyTuple_GET_SIZE(tuple) : 0;
    for (int i = 0; ok && i < n; ++i) {
      PyObject* x = PyTuple_GET_ITEM(tuple, i);
      ok = PyLong_Check(x);
      if (ok) v[i] = PyLong_AsLongLong(x);
    }
    Py_XDECREF(tuple);
    return ok && !PyErr_Occurred();
  }
  bool shape(PyObject* t) { return take(PyObject_GetAttr(t, s_shape)); }
  bool strides(PyObject* t) {
    PyObject* args[1] = {t};
    return take(PyObject_VectorcallMethod(s_stride, args, 1, nullptr));
  }
};

template <typename P>
bool pointer(PyObject* t, P** out) {
  int64_t a;
  if (!method(t, s_data_ptr, &a)) return false;
  *out = reinterpret_cast<P*>((uintptr_t)a);
  return true;
}

// A contiguous tensor of n entries; None: null.
template <typename P>
bool flat(PyObject* t, int64_t n, PyObject* dtype, int64_t dev, P** out) {
  *out = nullptr;
  if (t == Py_None) return true;
  int64_t count, on;
  return is_type(t, dtype) && method(t, s_numel, &count) && count == n && method(t, s_device, &on) && on == dev &&
         is_contiguous(t) && pointer(t, out);
}

bool whole(PyObject* x, int64_t* out) {                  // an int (borrowed)
  if (!PyLong_Check(x)) return false;
  *out = PyLong_AsLongLong(x);
  return !PyErr_Occurred() && *out >= INT_MIN && *out <= INT_MAX;
}
bool real(PyObject* x, float* out) {
  if (!PyFloat_Check(x)) return false;
  *out = (float)PyFloat_AS_DOUBLE(x);
  return true;
}

struct Where {                                           // the current device's stream and a workspace on it
  int64_t dev, stream, ws, nbytes;
  bool take(PyObject* like, PyObject* workspace) {
    int64_t now, on;
    if (!method(like, s_device, &dev) || dev < 0 || !number(PyObject_CallNoArgs(get_device_fn), &now) || now != dev)
      return false;
    if (!number(PyObject_GetAttr(workspace, s_ptr), &ws) || !number(PyObject_GetAttr(workspace, s_nbytes), &nbytes) ||
        nbytes < 0)
      return false;
    PyObject* buf = PyObject_GetAttr(workspace, s_buf);
    const bool ok = buf && method(buf, s_device, &on) && on == dev;
    Py_XDECREF(buf);
    if (!ok) return false;
    PyObject* index = PyLong_FromLongLong(dev);
    const bool got = index && number(PyObject_CallOneArg(get_stream_fn, index), &stream);
    Py_XDECREF(index);
    return got;
  }
  void* workspace() const { return reinterpret_cast<void*>((uintptr_t)ws); }
  cudaStream_t on() const { return reinterpret_cast<cudaStream_t>((uintptr_t)stream); }
};

struct Cache {                                           // PagedCache._key
  const dspark_paged_cache* ptr;
  PyObject* dtype;
  int64_t index, heads, head_dim;
  bool take(PyObject* cache) {
    PyObject* key = PyObject_GetAttr(cache, s_key);
    bool ok = key && PyTuple_Check(key) && PyTuple_GET_SIZE(key) == 5;
    int64_t at = 0;
    for (int i = 0; ok && i < 5; ++i) ok = i == 1 || PyLong_Check(PyTuple_GET_ITEM(key, i));
    if (ok) {
      at = PyLong_AsLongLong(PyTuple_GET_ITEM(key, 0));
      dtype = PyTuple_GET_ITEM(key, 1);                  // (a type, which outlives the tuple)
      index = PyLong_AsLongLong(PyTuple_GET_ITEM(key, 2));
      heads = PyLong_AsLongLong(PyTuple_GET_ITEM(key, 3));
      head_dim = PyLong_AsLongLong(PyTuple_GET_ITEM(key, 4));
      ptr = reinterpret_cast<const dspark_paged_cache*>((uintptr_t)at);
    }
    Py_XDECREF(key);
    return ok && !PyErr_Occurred();
  }
};

struct Tokens {                                          // rows of tokens with the leading dimensions `lead`
  int64_t B, N, rows;
  const int32_t *starts, *counts;
  bool take(const int64_t* lead, int n, PyObject* starts_o, PyObject* counts_o, PyObject* nodes, int64_t dev) {
    starts = counts = nullptr;
    if (starts_o == Py_None) {
      if (n != 2) return false;
      B = lead[0];
      N = lead[1];
      rows = B * N;
      return rows <= INT_MAX && flat(counts_o, B, i32, dev, &counts);
    }
    if (n != 1 || counts_o != Py_None || !whole(nodes, &N) || !method(starts_o, s_numel, &B)) return false;
    rows = lead[0];
    return --B >= 0 && rows <= INT_MAX && flat(starts_o, B + 1, i32, dev, &starts);
  }
};

struct Slots {
  const int32_t *pages, *lengths;
  int64_t most;
  bool take(PyObject* pages_o, PyObject* lengths_o, int64_t B, int64_t dev) {
    Dims d;
    if (pages_o == Py_None || lengths_o == Py_None || !d.shape(pages_o) || d.n != 2) return false;
    most = d.v[1];
    return most <= INT_MAX && flat(pages_o, B * most, i32, dev, &pages) && flat(lengths_o, B, i32, dev, &lengths);
  }
};

struct Heads {                                           // rows of heads
  void* p = nullptr;
  int64_t row = 0, head = 0, heads = 0;
  Dims shape;
  bool take(PyObject* t, const Cache& c) {
    int64_t on;
    Dims s;
    if (!is_type(t, c.dtype) || !method(t, s_device, &on) || on != c.index || !shape.shape(t) || !s.strides(t))
      return false;
    const int n = shape.n;
    if ((n != 3 && n != 4) || s.n != n || shape.v[n - 1] != c.head_dim || s.v[n - 1] != 1) return false;
    heads = shape.v[n - 2];
    int64_t rows = shape.v[0];
    row = s.v[0];
    if (n == 4) {
      const int64_t N = shape.v[1];
      if (N != 1) {
        row = s.v[1];
        if (rows > 1 && s.v[0] != N * row) return false;
      }
      rows *= N;
    }
    if (rows <= 1) row = 0;
    head = heads > 1 ? s.v[n - 2] : 0;
    return heads <= INT_MAX && pointer(t, &p);
  }
  bool like(const Heads& o) const {                      // the same leading dimensions
    if (shape.n != o.shape.n) return false;
    for (int i = 0; i < shape.n - 2; ++i)
      if (shape.v[i] != o.shape.v[i]) return false;
    return true;
  }
};

struct Matrix {                                          // rows of V entries, contiguous
  const void* p = nullptr;
  int dtype = -1;
  Dims shape;
  bool take(PyObject* t, int64_t dev) {
    int64_t on;
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d);
    dtype = d == f32 ? DSPARK_F32 : d == bf16 ? DSPARK_BF16 : d == f16 ? DSPARK_F16 : -1;
    return d && dtype >= 0 && method(t, s_device, &on) && on == dev && shape.shape(t) && shape.n >= 2 &&
           shape.v[shape.n - 1] > 0 && shape.v[shape.n - 1] <= INT_MAX && is_contiguous(t) && pointer(t, &p);
  }
};

PyObject* unchecked() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// (cache, k, v, pages, lengths, ws, q, q_out, starts, counts, nodes, parents, inv_freq, interleaved, q_weight,
//  k_weight, eps, layer)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Cache c;
  Where w;
  Heads k, v, q, o;
  Tokens t;
  Slots s;
  const int32_t* parents;
  const float *inv = nullptr, *qw, *kw;
  int64_t layer, half = 0;
  float eps;
  if (n != 18 || !c.take(a[0]) || !w.take(a[1], a[5]) || !k.take(a[1], c) || !v.take(a[2], c) || !v.like(k) ||
      k.heads != c.heads || v.heads != c.heads || !t.take(k.shape.v, k.shape.n - 2, a[8], a[9], a[10], w.dev) ||
      !s.take(a[3], a[4], t.B, w.dev) || !whole(a[17], &layer) || !real(a[16], &eps))
    return unchecked();
  if (a[6] == Py_None ? a[7] != Py_None
                      : a[7] == Py_None || !q.take(a[6], c) || !o.take(a[7], c) || !q.like(k) || !o.like(k) || o.heads != q.heads)
    return unchecked();
  if ((a[12] != Py_None && (!method(a[12], s_numel, &half) || half > 1024)) || !flat(a[12], half, f32, w.dev, &inv) ||
      !flat(a[11], t.rows, i32, w.dev, &parents) || !flat(a[14], c.head_dim, f32, w.dev, &qw) ||
      !flat(a[15], c.head_dim, f32, w.dev, &kw))
    return unchecked();
  const int interleaved = PyObject_IsTrue(a[13]);
  if (interleaved < 0) return unchecked();
  dspark_status st;
  Py_BEGIN_ALLOW_THREADS
  st = append_fn(c.ptr, (int)layer, t.starts, t.counts, parents, (int)t.B, (int)t.N, (int)t.rows, s.pages, (int)s.most,
                 s.lengths, k.p, k.row, k.head, v.p, v.row, v.head, q.p, q.row, q.head, (int)q.heads, o.p, o.row, o.head,
                 inv, (int)(2 * half), interleaved, qw, kw, eps, w.workspace(), (size_t)w.nbytes, w.on());
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// (q, cache, pages, lengths, ws, starts, counts, nodes, parents, scale, out, lse, layer)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Cache c;
  Where w;
  Heads q, o;
  Tokens t;
  Slots s;
  const int32_t* parents;
  float *lse, scale;
  int64_t layer;
  if (n != 13 || !c.take(a[1]) || !w.take(a[0], a[4]) || a[10] == Py_None || !q.take(a[0], c) || !o.take(a[10], c) ||
      !o.like(q) || o.heads != q.heads || !t.take(q.shape.v, q.shape.n - 2, a[5], a[6], a[7], w.dev) ||
      !s.take(a[2], a[3], t.B, w.dev) || !flat(a[8], t.rows, i32, w.dev, &parents) || !real(a[9], &scale) ||
      !flat(a[11], t.rows * q.heads, f32, w.dev, &lse) || !whole(a[12], &layer))
    return unchecked();
  dspark_status st;
  Py_BEGIN_ALLOW_THREADS
  st = attend_fn(c.ptr, (int)layer, t.starts, t.counts, parents, (int)t.B, (int)t.N, (int)t.rows, s.pages, (int)s.most,
                 s.lengths, q.p, q.row, q.head, (int)q.heads, scale, o.p, o.row, o.head, lse, w.workspace(),
                 (size_t)w.nbytes, w.on());
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// (p, tokens, uniforms, ws, q, starts, counts, nodes, parents, accept_len, path, out_tokens, n_out)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Where w;
  Matrix p, q;
  Tokens t;
  const int32_t *tokens, *parents;
  const float* uniforms;
  int32_t *accept_len, *path, *out_tokens, *n_out;
  for (int i = 9; i < n; ++i)
    if (a[i] == Py_None) return unchecked();             // an output that is to be made
  if (n != 13 || !w.take(a[0], a[3]) || !p.take(a[0], w.dev) ||
      !t.take(p.shape.v, p.shape.n - 1, a[5], a[6], a[7], w.dev))
    return unchecked();
  const int64_t V = p.shape.v[p.shape.n - 1];
  if (a[4] != Py_None) {
    if (!q.take(a[4], w.dev) || q.dtype != p.dtype || q.shape.n != p.shape.n) return unchecked();
    for (int i = 0; i < p.shape.n; ++i)
      if (q.shape.v[i] != p.shape.v[i]) return unchecked();
  }
  if (!flat(a[1], t.rows, i32, w.dev, &tokens) || !flat(a[2], t.rows, f32, w.dev, &uniforms) ||
      !flat(a[8], t.rows, i32, w.dev, &parents) || !flat(a[9], t.B, i32, w.dev, &accept_len) ||
      !flat(a[10], t.B * t.N, i32, w.dev, &path) || !flat(a[11], t.B * t.N, i32, w.dev, &out_tokens) ||
      !flat(a[12], t.B, i32, w.dev, &n_out))
    return unchecked();
  dspark_status st;
  Py_BEGIN_ALLOW_THREADS
  st = verify_fn(p.p, V, q.p, V, p.dtype, (int)V, tokens, uniforms, t.starts, t.counts, parents, (int)t.B, (int)t.N,
                 (int)t.rows, accept_len, path, out_tokens, n_out, w.workspace(), (size_t)w.nbytes, w.on());
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// (cache, pages, lengths, path, accept_len, ws)
PyObject* keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Cache c;
  Where w;
  Slots s;
  Dims d;
  const int32_t *path, *accept_len;
  if (n != 6 || !c.take(a[0])) return unchecked();
  PyObject* k = PyObject_GetAttr(a[0], s_k);
  const bool on = k && w.take(k, a[5]);
  Py_XDECREF(k);
  if (!on || !d.shape(a[3]) || d.n != 2 || d.v[0] > INT_MAX || d.v[1] > INT_MAX || a[4] == Py_None ||
      !s.take(a[1], a[2], d.v[0], w.dev) || !flat(a[3], d.v[0] * d.v[1], i32, w.dev, &path) ||
      !flat(a[4], d.v[0], i32, w.dev, &accept_len))
    return unchecked();
  dspark_status st;
  Py_BEGIN_ALLOW_THREADS
  st = keep_fn(c.ptr, (int)d.v[0], (int)d.v[1], s.pages, (int)s.most, s.lengths, path, accept_len, w.workspace(),
               (size_t)w.nbytes, w.on());
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// (addresses of the four calls, float32, bfloat16, float16, int32, current device, its raw stream)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) {
    PyErr_SetString(PyExc_TypeError, "setup: 10 arguments are needed");
    return nullptr;
  }
  void* fn[4];
  for (int i = 0; i < 4; ++i)
    if (!(fn[i] = PyLong_AsVoidPtr(a[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup: a call has no address");
      return nullptr;
    }
  append_fn = reinterpret_cast<decltype(append_fn)>(fn[0]);
  attend_fn = reinterpret_cast<decltype(attend_fn)>(fn[1]);
  verify_fn = reinterpret_cast<decltype(verify_fn)>(fn[2]);
  keep_fn = reinterpret_cast<decltype(keep_fn)>(fn[3]);
  PyObject** to[6] = {&f32, &bf16, &f16, &i32, &get_device_fn, &get_stream_fn};
  for (int i = 0; i < 6; ++i) *to[i] = Py_NewRef(a[4 + i]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(setup)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"verify", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(verify)), METH_FASTCALL, nullptr},
    {"keep", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(keep)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dspark_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dspark_calls() {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"}, {&s_data_ptr, "data_ptr"},
               {&s_numel, "numel"}, {&s_device, "get_device"}, {&s_contiguous, "is_contiguous"}, {&s_ptr, "ptr"},
               {&s_nbytes, "nbytes"}, {&s_buf, "buf"}, {&s_key, "_key"}, {&s_k, "k"}};
  for (auto& x : names)
    if (!(*x.to = PyUnicode_InternFromString(x.name))) return nullptr;
  return PyModule_Create(&module);
}
