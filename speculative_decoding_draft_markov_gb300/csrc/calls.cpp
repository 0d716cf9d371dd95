// The Python calls of the target model's side, which are made per layer and per token: arguments are checked
// (tensors' types, shapes, strides and devices, which the C ABI cannot see behind bare pointers), handed to the C ABI, and a
// status other than DSPARK_OK is raised.  GB300's host: 5.8 us for an append, 7.6 for an attention (its two launches and
// three tensor maps), 6.1 for the logit rules; through ctypes, with the checks in Python, 10.0, 11.7 and 9.2, more
// than the GPU spends on one token.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>
#include <cstdint>

#include "dspark.h"

namespace {

// set by init
PyObject *t_f32, *t_bf16, *t_i32, *t_i16;          // torch's types
PyObject *current_stream, *current_device, *error, *device_error;  // raw stream of a device; DSparkError, DSparkDeviceError
PyObject *m_data_ptr, *m_get_device, *m_is_contiguous;             // a tensor's methods, found once
PyObject *s_dtype, *s_shape, *s_stride, *s_cuda_stream, *s_numel;

bool bad(const char* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%s %s", name, what);
  return false;
}

bool to_int(PyObject* o, int* v, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) return false;
  if (x < INT_MIN || x > INT_MAX) return bad(name, "is beyond 32 bits");
  *v = int(x);
  return true;
}

// nd entries of a tuple of ints (a shape, strides)
bool ints_of(PyObject* t, PyObject* attr, bool method, int nd, int64_t* d, const char* name) {
  PyObject* s = method ? PyObject_CallMethodNoArgs(t, attr) : PyObject_GetAttr(t, attr);
  if (!s) return false;
  bool ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == nd;
  if (!ok) PyErr_Format(PyExc_ValueError, "%s must have %d dimensions", name, nd);
  for (int i = 0; ok && i < nd; ++i) {
    d[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
    ok = !(d[i] == -1 && PyErr_Occurred());
  }
  Py_DECREF(s);
  return ok;
}
bool shape_of(PyObject* t, int nd, int64_t* d, const char* name) {
  if (!ints_of(t, s_shape, false, nd, d, name)) return false;
  for (int i = 0; i < nd; ++i)
    if (d[i] > INT_MAX) return bad(name, "has a dimension beyond 32 bits");
  return true;
}

bool has_type(PyObject* t, PyObject* dtype, const char* name) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return false;
  const bool ok = d == dtype;
  if (!ok) PyErr_Format(PyExc_ValueError, "%s must be %R, not %R", name, dtype, d);
  Py_DECREF(d);
  return ok;
}

// Where a call's tensors lie: the first one's device, and the name of one that lies elsewhere or in host memory.
struct Place {
  long device = -1;
  const char* other = nullptr;
};

bool pointer(PyObject* t, const char* name, void** p, Place& at) {
  PyObject* o = PyObject_CallOneArg(m_data_ptr, t);
  if (!o) return false;
  *p = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  if (!*p) return !PyErr_Occurred();  // an empty tensor lies nowhere
  o = PyObject_CallOneArg(m_get_device, t);
  if (!o) return false;
  const long d = PyLong_AsLong(o);  // -1: host memory
  Py_DECREF(o);
  if (d == -1 && PyErr_Occurred()) return false;
  if (at.device < 0) at.device = d;
  if ((d < 0 || d != at.device) && !at.other) at.other = name;
  return true;
}

bool contiguous(PyObject* t, const char* name) {
  PyObject* c = PyObject_CallOneArg(m_is_contiguous, t);
  if (!c) return false;
  Py_DECREF(c);  // a singleton
  return c == Py_True || bad(name, "must be contiguous");
}

// The pointer of a dense tensor of that type and shape (nd = 0: any shape); None: NULL.
bool dense(PyObject* t, PyObject* dtype, int nd, const int64_t* want, const char* name, void** p, Place& at) {
  *p = nullptr;
  if (t == Py_None) return true;
  if (!has_type(t, dtype, name)) return false;
  if (nd) {
    int64_t d[4];
    if (!ints_of(t, s_shape, false, nd, d, name)) return false;
    for (int i = 0; i < nd; ++i)
      if (d[i] != want[i]) {
        PyErr_Format(PyExc_ValueError, "%s must have %lld entries in dimension %d, not %lld", name,
                     static_cast<long long>(want[i]), i, static_cast<long long>(d[i]));
        return false;
      }
  }
  return contiguous(t, name) && pointer(t, name, p, at);
}
bool dense1(PyObject* t, PyObject* dtype, int64_t n, const char* name, void** p, Place& at) {
  return dense(t, dtype, 1, &n, name, p, at);
}
bool dense2(PyObject* t, PyObject* dtype, int64_t n, int64_t m, const char* name, void** p, Place& at) {
  const int64_t d[2] = {n, m};
  return dense(t, dtype, 2, d, name, p, at);
}

bool table_of(PyObject* t, const int64_t* d, int64_t bs, void** p, Place& at) {  // a page table of shape d
  if (d[0] != bs) return bad("page_table", "must have one row per request");
  return dense(t, t_i32, 0, nullptr, "page_table", p, at);
}

// Pointer and elements from row to row of a [rows, H, D] tensor of shape d whose heads and lanes are dense.
bool rows_of(PyObject* t, PyObject* dtype, const int64_t* d, int64_t rows, int64_t H, int64_t D, const char* name, void** p,
             int64_t* stride, Place& at) {
  int64_t st[3];
  if (!has_type(t, dtype, name)) return false;
  if (d[0] != rows || d[1] != H || d[2] != D) {
    PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld)", name, static_cast<long long>(rows),
                 static_cast<long long>(H), static_cast<long long>(D));
    return false;
  }
  if (!ints_of(t, s_stride, true, 3, st, name)) return false;
  if (st[2] != 1 || (st[1] != D && H > 1)) return bad(name, "must be [rows, heads, lanes] with dense heads and lanes");
  *stride = rows > 1 ? st[0] : H * D;
  return pointer(t, name, p, at);
}

// Entries of a 1-D tensor, of any tensor.
bool length(PyObject* t, int64_t* n, const char* name) { return shape_of(t, 1, n, name); }
bool numel(PyObject* t, int64_t* n) {
  PyObject* o = PyObject_CallMethodNoArgs(t, s_numel);
  if (!o) return false;
  *n = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return !PyErr_Occurred();
}

bool workspace(PyObject* t, void** p, size_t* bytes, Place& at) {
  int64_t n;
  if (!numel(t, &n) || !contiguous(t, "ws") || !pointer(t, "ws", p, at)) return false;
  *bytes = size_t(n);
  return true;
}

// A torch stream, an integer, or None: torch's current one.  The kernels run on the current device, so that is where the
// tensors have to lie.
bool stream_of(PyObject* s, const char* call, const Place& at, dspark_stream_t* out) {
  PyObject* dev = nullptr;
  if (!at.other && at.device >= 0 && !(dev = PyObject_CallNoArgs(current_device))) return false;
  if (!dev || PyLong_AsLong(dev) != at.device) {
    Py_XDECREF(dev);
    PyObject* e = PyObject_CallFunction(device_error, "ss", call, at.other ? at.other : "every tensor");
    if (e) PyErr_SetObject(device_error, e), Py_DECREF(e);
    return false;
  }
  PyObject* o;
  if (s == Py_None)
    o = PyObject_CallOneArg(current_stream, dev);
  else
    o = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttr(s, s_cuda_stream);
  Py_DECREF(dev);
  if (!o) return false;
  *out = reinterpret_cast<dspark_stream_t>(PyLong_AsVoidPtr(o));
  Py_DECREF(o);
  return !PyErr_Occurred();
}

int dtype_code(PyObject* t, PyObject** dtype) {
  *dtype = PyObject_GetAttr(t, s_dtype);
  if (!*dtype) return -1;
  Py_DECREF(*dtype);  // torch keeps its types
  return *dtype == t_bf16 ? DSPARK_BF16 : *dtype == t_f32 ? DSPARK_F32 : -1;
}

PyObject* result(int rc, const char* name) {
  if (rc == DSPARK_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(error, "is", rc, name);
  if (e) PyErr_SetObject(error, e), Py_DECREF(e);
  return nullptr;
}

bool expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  return n == want;
}

template <typename T> T* as(void* p) { return static_cast<T*>(p); }

// q, k, v, cu_seqlens, ctx_len, cos_sin, page_table, q_out, k_cache, v_cache, ws, interleaved, stream
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 13)) return nullptr;
  PyObject* dt;
  int64_t c[4], k3[3], v3[3], cu_n, table[2], cs[2], q3[3], qs = 0, ks, vs;
  void *q = nullptr, *k, *v, *cu, *ctx, *cos, *pt, *qo = nullptr, *kc, *vc, *ws;
  size_t ws_bytes;
  Place at;
  dspark_stream_t s;
  const int code = dtype_code(a[8], &dt), turn = PyObject_IsTrue(a[11]);
  if (!dt || turn < 0 || !shape_of(a[8], 4, c, "k_cache") || !shape_of(a[1], 3, k3, "k") || !shape_of(a[2], 3, v3, "v") ||
      !length(a[3], &cu_n, "cu_seqlens") ||
      !shape_of(a[6], 2, table, "page_table") || !shape_of(a[5], 2, cs, "cos_sin"))
    return nullptr;
  const int64_t rows = k3[0], bs = cu_n - 1, Hkv = c[1], D = c[3];
  int64_t Hq = Hkv;
  if (a[0] != Py_None) {
    if (!shape_of(a[0], 3, q3, "q")) return nullptr;
    Hq = q3[1];
    const int64_t o[3] = {rows, Hq, D};
    if (!rows_of(a[0], dt, q3, rows, Hq, D, "q", &q, &qs, at) || !dense(a[7], dt, 3, o, "q_out", &qo, at)) return nullptr;
  }
  if (!rows_of(a[1], dt, k3, rows, Hkv, D, "k", &k, &ks, at) || !rows_of(a[2], dt, v3, rows, Hkv, D, "v", &v, &vs, at) ||
      !dense(a[3], t_i32, 0, nullptr, "cu_seqlens", &cu, at) || !dense1(a[4], t_i32, bs, "ctx_len", &ctx, at) ||
      !dense(a[5], t_f32, 0, nullptr, "cos_sin", &cos, at) || !table_of(a[6], table, bs, &pt, at) ||
      !dense(a[8], dt, 0, nullptr, "k_cache", &kc, at) || !dense(a[9], dt, 4, c, "v_cache", &vc, at) ||
      !workspace(a[10], &ws, &ws_bytes, at) || !stream_of(a[12], "dspark_append_kv", at, &s))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = dspark_append_kv(q, qs, k, ks, v, vs, code, as<int32_t>(cu), as<int32_t>(ctx), int(bs), int(rows), as<float>(cos),
                        int(cs[0]), int(cs[1]), turn, as<int32_t>(pt), int(table[1]), int(c[0]), int(c[2]), int(Hq), int(Hkv),
                        int(D), qo, kc, vc, ws, ws_bytes, s);
  Py_END_ALLOW_THREADS
  return result(rc, "dspark_append_kv");
}

// q, k_cache, v_cache, page_table, cu_seqlens, ctx_len, max_rows, scale, window, n_sink, out, lse, ws, stream
PyObject* window_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 14)) return nullptr;
  PyObject* dt;
  int64_t c[4], q3[3], cu_n, table[2], qs;
  void *q, *kc, *vc, *pt, *cu, *ctx, *out, *lse, *ws;
  size_t ws_bytes;
  Place at;
  dspark_stream_t s;
  int max_rows, window, n_sink;
  const int code = dtype_code(a[1], &dt);
  const double scale = PyFloat_AsDouble(a[7]);
  if (!dt || (scale == -1. && PyErr_Occurred()) || !to_int(a[6], &max_rows, "max_rows") || !to_int(a[8], &window, "window") ||
      !to_int(a[9], &n_sink, "n_sink") || !shape_of(a[1], 4, c, "k_cache") || !shape_of(a[0], 3, q3, "q") ||
      !length(a[4], &cu_n, "cu_seqlens") || !shape_of(a[3], 2, table, "page_table"))
    return nullptr;
  const int64_t rows = q3[0], Hq = q3[1], bs = cu_n - 1, Hkv = c[1], D = c[3];
  const int64_t o[3] = {rows, Hq, D};
  if (!rows_of(a[0], dt, q3, rows, Hq, D, "q", &q, &qs, at) || !dense(a[1], dt, 0, nullptr, "k_cache", &kc, at) ||
      !dense(a[2], dt, 4, c, "v_cache", &vc, at) || !table_of(a[3], table, bs, &pt, at) ||
      !dense(a[4], t_i32, 0, nullptr, "cu_seqlens", &cu, at) || !dense1(a[5], t_i32, bs, "ctx_len", &ctx, at) ||
      !dense(a[10], dt, 3, o, "out", &out, at) || !dense2(a[11], t_f32, rows, Hq, "lse", &lse, at) ||
      !workspace(a[12], &ws, &ws_bytes, at) || !stream_of(a[13], "dspark_window_attention", at, &s))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = dspark_window_attention(q, qs, code, kc, vc, as<int32_t>(pt), int(table[1]), int(c[0]), int(c[2]), as<int32_t>(cu),
                               as<int32_t>(ctx), int(bs), int(rows), max_rows, int(Hq), int(Hkv), int(D), float(scale), window,
                               n_sink, out, as<float>(lse), ws, ws_bytes, s);
  Py_END_ALLOW_THREADS
  return result(rc, "dspark_window_attention");
}

// logits, cu_seqlens, ids, hist, repetition, frequency, presence, bias_start, bias_ids, bias_vals, mask, out, ws, stream
PyObject* process_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 14)) return nullptr;
  PyObject* dt;
  int64_t x[2], cu_n, ids_n, n_bias = 0;
  void *in, *cu, *ids, *hist, *rep, *freq, *pres, *bst, *bid, *bval, *mask, *out, *ws;
  size_t ws_bytes;
  Place at;
  dspark_stream_t s;
  const int code = dtype_code(a[0], &dt);
  if (!dt || !shape_of(a[0], 2, x, "logits") || !length(a[1], &cu_n, "cu_seqlens") || !length(a[2], &ids_n, "ids") ||
      (a[8] != Py_None && !length(a[8], &n_bias, "bias_ids")))
    return nullptr;
  const int64_t rows = x[0], V = x[1], bs = cu_n - 1;
  if (ids_n < rows) return bad("ids", "must hold one entry per row"), nullptr;
  if (!dense(a[0], dt, 0, nullptr, "logits", &in, at) || !dense(a[1], t_i32, 0, nullptr, "cu_seqlens", &cu, at) ||
      !dense(a[2], t_i32, 0, nullptr, "ids", &ids, at) || !dense2(a[3], t_i16, bs, V, "hist", &hist, at) ||
      !dense1(a[4], t_f32, bs, "repetition", &rep, at) || !dense1(a[5], t_f32, bs, "frequency", &freq, at) ||
      !dense1(a[6], t_f32, bs, "presence", &pres, at) || !dense1(a[7], t_i32, bs + 1, "bias_start", &bst, at) ||
      !dense(a[8], t_i32, 0, nullptr, "bias_ids", &bid, at) || !dense1(a[9], t_f32, n_bias, "bias_vals", &bval, at) ||
      !dense2(a[10], t_i32, rows, (V + 31) / 32, "mask", &mask, at) || !dense(a[11], dt, 2, x, "out", &out, at) ||
      !workspace(a[12], &ws, &ws_bytes, at) || !stream_of(a[13], "dspark_process_logits", at, &s))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = dspark_process_logits(in, code, int(rows), int(V), as<int32_t>(cu), as<int32_t>(ids), int(bs), as<int16_t>(hist),
                             as<float>(rep), as<float>(freq), as<float>(pres), as<int32_t>(bst), as<int32_t>(bid),
                             as<float>(bval), int(n_bias), as<uint32_t>(mask), out, ws, ws_bytes, s);
  Py_END_ALLOW_THREADS
  return result(rc, "dspark_process_logits");
}

// tokens, start, n_prompt, hist, ws, stream
PyObject* history_build(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 6)) return nullptr;
  int64_t h[2], n_tokens;
  void *tokens, *start, *asked, *hist, *ws;
  size_t ws_bytes;
  Place at;
  dspark_stream_t s;
  if (!shape_of(a[3], 2, h, "hist") || !length(a[0], &n_tokens, "tokens") ||
      !dense(a[0], t_i32, 0, nullptr, "tokens", &tokens, at) ||
      !dense1(a[1], t_i32, h[0] + 1, "start", &start, at) || !dense1(a[2], t_i32, h[0], "n_prompt", &asked, at) ||
      !dense(a[3], t_i16, 0, nullptr, "hist", &hist, at) || !workspace(a[4], &ws, &ws_bytes, at) ||
      !stream_of(a[5], "dspark_history_build", at, &s))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = dspark_history_build(as<int32_t>(tokens), int(n_tokens), as<int32_t>(start), as<int32_t>(asked), int(h[0]), int(h[1]),
                            as<int16_t>(hist), ws, ws_bytes, s);
  Py_END_ALLOW_THREADS
  return result(rc, "dspark_history_build");
}

// out_tokens, hist, ws, stream
PyObject* history_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 4)) return nullptr;
  int64_t h[2], o[2];
  void *tokens, *hist, *ws;
  size_t ws_bytes;
  Place at;
  dspark_stream_t s;
  if (!shape_of(a[1], 2, h, "hist") || !shape_of(a[0], 2, o, "out_tokens")) return nullptr;
  if (o[0] != h[0]) return bad("out_tokens", "must have one row per request"), nullptr;
  if (!dense(a[0], t_i32, 0, nullptr, "out_tokens", &tokens, at) || !dense(a[1], t_i16, 0, nullptr, "hist", &hist, at) ||
      !workspace(a[2], &ws, &ws_bytes, at) || !stream_of(a[3], "dspark_history_commit", at, &s))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = dspark_history_commit(as<int32_t>(tokens), int(h[0]), int(o[1]) - 1, int(h[1]), as<int16_t>(hist), ws, ws_bytes, s);
  Py_END_ALLOW_THREADS
  return result(rc, "dspark_history_commit");
}

// float32, bfloat16, int32, int16, current raw stream of a device, current device, DSparkError, DSparkDeviceError, and the
// tensors' data_ptr, get_device and is_contiguous
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 11)) return nullptr;
  PyObject** const to[11] = {&t_f32, &t_bf16, &t_i32, &t_i16, &current_stream, &current_device, &error, &device_error,
                             &m_data_ptr, &m_get_device, &m_is_contiguous};
  for (int i = 0; i < 11; ++i) *to[i] = Py_NewRef(a[i]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init), FAST(append_kv), FAST(window_attention), FAST(process_logits), FAST(history_build),
                         FAST(history_commit), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  s_dtype = PyUnicode_InternFromString("dtype"), s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride"), s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  s_numel = PyUnicode_InternFromString("numel");
  if (!s_dtype || !s_shape || !s_stride || !s_cuda_stream || !s_numel) return nullptr;
  return PyModule_Create(&module);
}
