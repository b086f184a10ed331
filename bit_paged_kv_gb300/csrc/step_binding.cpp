// step_binding.cpp -- the Python binding of the serving step's calls
// (saw_build_tables, saw_rope_table, saw_rope_append, saw_prefix_decode_int4) and
// of a sparse decode step (saw_norm_rope_append, saw_page_summary,
// saw_select_pages, saw_sparse_decode_int4): a CPython extension without torch headers, which reads tensors through their
// own methods and calls the C ABI by address.
//
// These calls run once or more per layer on small batches, where the host's
// share of a call is what a user of eager steps waits for.  A rotary append of
// one token takes 6.0 us of a Grace core here, 2 of them the launch and 0.7 the
// checks that every tensor is on the call's device and the caches are as large
// as its counts say; through ctypes, with fewer checks, in Python, 9.7 us (2
// for the conversion of its 28 arguments).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "saw_int4.h"

namespace {

struct Entry {
  decltype(&saw_build_tables) build_tables;
  decltype(&saw_rope_table) rope_table;
  decltype(&saw_rope_append) rope_append;
  decltype(&saw_prefix_decode_int4) prefix_decode;
  decltype(&saw_cache_bytes) cache_bytes;
} g_entry;
struct SparseEntry {
  decltype(&saw_norm_rope_append) norm_rope_append;
  decltype(&saw_page_summary) page_summary;
  decltype(&saw_select_pages) select_pages;
  decltype(&saw_sparse_decode_int4) sparse_decode;
  decltype(&saw_summary_bytes) summary_bytes;
} g_sparse;
PyObject *g_int32, *g_f32, *g_bf16, *g_f16;     // dtypes
PyObject *g_device, *g_raw_stream;              // current device; its current stream
PyObject *n_dtype, *n_data_ptr, *n_contiguous, *n_numel, *n_shape, *n_stride, *n_get_device,
    *n_cuda_stream, *n_nbytes;

// Every helper returns false with a Python exception set.

bool call_i64(PyObject* t, PyObject* name, int64_t* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return false;
  *out = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return *out != -1 || !PyErr_Occurred();
}
// A tensor's address (addresses use all 64 bits), or null for None.
bool address(PyObject* t, void** out) {
  *out = nullptr;
  if (t == Py_None) return true;
  PyObject* r = PyObject_CallMethodNoArgs(t, n_data_ptr);
  if (!r) return false;
  *out = reinterpret_cast<void*>(uintptr_t(PyLong_AsUnsignedLongLong(r)));
  Py_DECREF(r);
  return !PyErr_Occurred();
}
template <typename T>
T* as(void* p) {
  return static_cast<T*>(p);
}
bool has_dtype(PyObject* t, PyObject* want, bool* yes) {
  PyObject* d = PyObject_GetAttr(t, n_dtype);
  if (!d) return false;
  *yes = d == want;
  Py_DECREF(d);
  return true;
}
bool contiguous(PyObject* t, bool* yes) {
  PyObject* r = PyObject_CallMethodNoArgs(t, n_contiguous);
  if (!r) return false;
  *yes = r == Py_True;
  Py_DECREF(r);
  return true;
}
// The entries of a shape or stride tuple of the given length.
bool entries(PyObject* tuple, const char* what, int n, int64_t* out) {
  if (!tuple) return false;
  bool ok = PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == n;
  if (!ok) PyErr_Format(PyExc_ValueError, "%s must have %d dimensions", what, n);
  for (int i = 0; ok && i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    ok = out[i] != -1 || !PyErr_Occurred();
  }
  Py_DECREF(tuple);
  return ok;
}
bool shape(PyObject* t, const char* what, int n, int64_t* out) {
  return entries(PyObject_GetAttr(t, n_shape), what, n, out);
}
// Every tensor has to be on the call's device: the kernels take it by address.
bool on_device(PyObject* t, const char* what, int64_t dev) {
  int64_t at;
  if (!call_i64(t, n_get_device, &at)) return false;
  if (at != dev) PyErr_Format(PyExc_ValueError, "%s must be on cuda:%lld", what, (long long)dev);
  return at == dev;
}
// Contiguous int32 on the device, of n entries (any number for n < 0; `size` may take it).
bool words(PyObject* t, const char* what, int64_t dev, int64_t n, int32_t** out, int64_t* size = nullptr) {
  *out = nullptr;
  if (size) *size = 0;
  if (t == Py_None) return true;
  bool type, cont;
  if (!on_device(t, what, dev) || !has_dtype(t, g_int32, &type) || !contiguous(t, &cont)) return false;
  if (!type || !cont) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous int32", what);
    return false;
  }
  if (n >= 0 || size) {
    int64_t have;
    if (!call_i64(t, n_numel, &have)) return false;
    if (n >= 0 && have != n) {
      PyErr_Format(PyExc_ValueError, "%s must have %lld entries, not %lld", what, (long long)n, (long long)have);
      return false;
    }
    if (size) *size = have;
  }
  void* p;
  if (!address(t, &p)) return false;
  *out = as<int32_t>(p);
  return true;
}
// The status word (one entry or more), or None.
bool status_word(PyObject* t, int64_t dev, int32_t** out) {
  int64_t n;
  if (!words(t, "dev_status", dev, -1, out, &n)) return false;
  if (t != Py_None && n < 1) PyErr_SetString(PyExc_ValueError, "dev_status must have an entry");
  return t == Py_None || n >= 1;
}
// Contiguous memory of any type on the device, of `need` bytes or more (None:
// null, for the library to refuse or take).
bool memory(PyObject* t, const char* what, int64_t dev, size_t need, void** out, int64_t* size = nullptr) {
  bool cont;
  *out = nullptr;
  if (t == Py_None) return true;
  if (!on_device(t, what, dev) || !contiguous(t, &cont) || !address(t, out)) return false;
  if (!cont) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", what);
    return false;
  }
  PyObject* r = PyObject_GetAttr(t, n_nbytes);
  if (!r) return false;
  const int64_t have = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (have == -1 && PyErr_Occurred()) return false;
  if (size) *size = have;
  if (uint64_t(have) < need)
    PyErr_Format(PyExc_ValueError, "%s must have %llu bytes, not %lld", what, (unsigned long long)need,
                 (long long)have);
  return uint64_t(have) >= need;
}
bool int32_of(PyObject* o, int32_t* out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument beyond 32 bits");
    return false;
  }
  *out = int32_t(v);
  return true;
}
bool size32(int64_t v, int32_t* out) {
  if (v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "more than 2^31 - 1 entries");
    return false;
  }
  *out = int32_t(v);
  return true;
}
bool flag_of(PyObject* o, int32_t* out) {
  *out = PyObject_IsTrue(o);
  return *out >= 0;
}
bool real_of(PyObject* o, double* out) {
  *out = PyFloat_AsDouble(o);
  return *out != -1.0 || !PyErr_Occurred();
}
// The library launches on the current device: it has to be the tensors'.
bool on_current(PyObject* t, int64_t* dev) {
  if (!call_i64(t, n_get_device, dev)) return false;
  if (*dev < 0) {
    PyErr_SetString(PyExc_ValueError, "tensors have to be on a CUDA device");
    return false;
  }
  PyObject* r = PyObject_CallNoArgs(g_device);
  if (!r) return false;
  const int64_t now = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (now == -1 && PyErr_Occurred()) return false;
  if (now != *dev)
    PyErr_Format(PyExc_ValueError, "tensors are on cuda:%lld, the current device is cuda:%lld", (long long)*dev,
                 (long long)now);
  return now == *dev;
}
// None: the device's current stream; else a Stream object or a handle.
bool stream_of(PyObject* s, int64_t dev, void** out) {
  PyObject* r;
  if (s == Py_None) {
    PyObject* d = PyLong_FromLongLong(dev);
    if (!d) return false;
    r = PyObject_CallOneArg(g_raw_stream, d);
    Py_DECREF(d);
  } else if (PyLong_Check(s)) {
    r = Py_NewRef(s);
  } else {
    r = PyObject_GetAttr(s, n_cuda_stream);
  }
  if (!r) return false;
  *out = reinterpret_cast<void*>(uintptr_t(PyLong_AsUnsignedLongLong(r)));
  Py_DECREF(r);
  return !PyErr_Occurred();
}
bool formats_of(PyObject* t, PyObject* meta_bf16, int32_t* out) {
  PyObject* d = PyObject_GetAttr(t, n_dtype);
  if (!d) return false;
  const bool f16 = d == g_f16, bf16 = d == g_bf16;
  if (!f16 && !bf16) PyErr_Format(PyExc_ValueError, "inputs must be bfloat16 or float16, not %S", d);
  Py_DECREF(d);
  int32_t meta;
  if ((!f16 && !bf16) || !flag_of(meta_bf16, &meta)) return false;
  *out = (f16 ? SAW_FMT_F16_INPUT : 0) | (meta ? SAW_FMT_BF16_META : 0);
  return true;
}
// Rows [T, heads, D] of a type, only the token dimension strided.
struct Rows {
  void* p = nullptr;
  int64_t heads = 0, stride = 0;
};
bool rows_of(PyObject* t, PyObject* dtype, int64_t dev, int64_t T, int64_t D, const char* what, Rows* out) {
  int64_t n[3], s[3];
  bool type;
  if (!on_device(t, what, dev) || !shape(t, what, 3, n) ||
      !entries(PyObject_CallMethodNoArgs(t, n_stride), what, 3, s) || !has_dtype(t, dtype, &type) || !address(t, &out->p))
    return false;
  if (!type || n[0] != T || n[2] != D || s[2] != 1 || (s[1] != D && n[1] != 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, heads, %lld] rows of k's type, each token's contiguous", what,
                 (long long)T, (long long)D);
    return false;
  }
  out->heads = n[1];
  // (a single token's stride is whatever the view says; it is never used)
  out->stride = T > 1 ? s[0] : n[1] * D;
  return true;
}
bool f32_table(PyObject* t, const char* what, int64_t dev, int64_t* dims, void** out) {
  bool type, cont;
  if (!on_device(t, what, dev) || !has_dtype(t, g_f32, &type) || !contiguous(t, &cont)) return false;
  if (!type || !cont) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous float32 [max_pos, rope_dim]", what);
    return false;
  }
  return shape(t, what, 2, dims) && address(t, out);
}
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  return n == want;
}
template <typename F>
PyObject* status_of(F&& f) {
  int32_t rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// The arguments are those of the functions of bit_paged_kv_gb300/_binding.py, in order.

PyObject* build_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 16)) return nullptr;
  int64_t dev, B, tokens, frees = 0, src[2] = {0, 0}, dst[2];
  int32_t *cached, *fresh, *free_pages, *num_free, *tables, *seq_lens, *cu, *slots, *positions, *taken, *from, *from_rows,
      *status;
  int32_t page_size, num_pages, nb, nt, nf, nr, ns, width;
  void* stream;
  if (!on_current(a[1], &dev) || !words(a[1], "new_lens", dev, -1, &fresh, &B) ||
      !words(a[9], "slot_mapping", dev, -1, &slots, &tokens) || !shape(a[6], "block_tables", 2, dst))
    return nullptr;
  if (dst[0] != B) {
    PyErr_Format(PyExc_ValueError, "block_tables must have %lld rows, not %lld", (long long)B, (long long)dst[0]);
    return nullptr;
  }
  if (a[12] != Py_None && !shape(a[12], "src_tables", 2, src)) return nullptr;
  if (!words(a[0], "cached_lens", dev, B, &cached) || !words(a[2], "free_pages", dev, -1, &free_pages, &frees) ||
      !words(a[3], "num_free", dev, 1, &num_free) || !int32_of(a[4], &page_size) || !int32_of(a[5], &num_pages) ||
      !words(a[6], "block_tables", dev, -1, &tables) || !words(a[7], "seq_lens", dev, B, &seq_lens) ||
      !words(a[8], "cu_q_lens", dev, B + 1, &cu) || !words(a[10], "positions", dev, tokens, &positions) ||
      !words(a[11], "pages_taken", dev, 1, &taken) || !words(a[12], "src_tables", dev, -1, &from) ||
      !words(a[13], "src_rows", dev, B, &from_rows) || !status_word(a[14], dev, &status) ||
      !stream_of(a[15], dev, &stream) || !size32(B, &nb) || !size32(tokens, &nt) || !size32(frees, &nf) ||
      !size32(src[0], &nr) || !size32(src[1], &ns) || !size32(dst[1], &width))
    return nullptr;
  return status_of([&] {
    return g_entry.build_tables(from, nr, ns, from_rows, cached, fresh, free_pages, nf, num_free, nb, nt, num_pages,
                                page_size, tables, width, seq_lens, cu, slots, positions, taken, status, stream);
  });
}

PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  int64_t dev, dims[2];
  int32_t max_pos, rope_dim, scaling, orig;
  double base, factor, low, high, att;
  void *p, *stream;
  if (!on_current(a[0], &dev) || !f32_table(a[0], "cos_sin", dev, dims, &p) || !size32(dims[0], &max_pos) ||
      !size32(dims[1], &rope_dim) || !real_of(a[1], &base) || !int32_of(a[2], &scaling) || !real_of(a[3], &factor) ||
      !int32_of(a[4], &orig) || !real_of(a[5], &low) || !real_of(a[6], &high) || !real_of(a[7], &att) ||
      !stream_of(a[8], dev, &stream))
    return nullptr;
  return status_of([&] {
    return g_entry.rope_table(as<float>(p), max_pos, rope_dim, base, scaling, factor, orig, low, high, float(att),
                              stream);
  });
}

// What the rotary appends have in common.
struct RopeArgs {
  Rows q, k, v, out;
  int32_t *positions, *slots, *status;
  int32_t num_pages, page_size, rot_k, rot_v, h, inter, formats, T, D, hq, hkv, max_pos, rope_dim;
  void *cos_sin, *kc, *vc = nullptr, *stream;
  int64_t dev;
  PyObject* dtype;
};
// Places of a call's arguments (q, k and v come first).
struct RopePlaces {
  int positions, cos_sin, slots, q_out, k_cache, v_cache, num_pages, page_size, rot_k, rot_v, h, inter, status, stream,
      meta;
};
bool rope_args(PyObject* const* a, const RopePlaces& at, RopeArgs* r) {
  PyObject *q = a[0], *k = a[1], *v = a[2];
  int64_t dims[3], table[2];
  if (!on_current(k, &r->dev) || !shape(k, "k", 3, dims) || !formats_of(k, a[at.meta], &r->formats)) return false;
  const int64_t dev = r->dev;
  r->dtype = (r->formats & SAW_FMT_F16_INPUT) ? g_f16 : g_bf16;
  if (!rows_of(k, r->dtype, dev, dims[0], dims[2], "k", &r->k) ||
      !f32_table(a[at.cos_sin], "cos_sin", dev, table, &r->cos_sin))
    return false;
  if (q != Py_None) {
    if (!rows_of(q, r->dtype, dev, dims[0], dims[2], "q", &r->q) ||
        !rows_of(a[at.q_out], r->dtype, dev, dims[0], dims[2], "q_out", &r->out))
      return false;
    if (r->q.heads != r->out.heads) {
      PyErr_SetString(PyExc_ValueError, "q_out must have q's heads");
      return false;
    }
  }
  if (v != Py_None) {
    if (!rows_of(v, r->dtype, dev, dims[0], dims[2], "v", &r->v)) return false;
    if (r->v.heads != r->k.heads) {
      PyErr_SetString(PyExc_ValueError, "v must have k's heads");
      return false;
    }
  }
  if (!words(a[at.positions], "positions", dev, dims[0], &r->positions) ||
      !words(a[at.slots], "slot_mapping", dev, dims[0], &r->slots) || !int32_of(a[at.num_pages], &r->num_pages) ||
      !int32_of(a[at.page_size], &r->page_size) || !flag_of(a[at.rot_k], &r->rot_k) ||
      !flag_of(a[at.rot_v], &r->rot_v) || !int32_of(a[at.h], &r->h) || !flag_of(a[at.inter], &r->inter) ||
      !status_word(a[at.status], dev, &r->status) || !stream_of(a[at.stream], dev, &r->stream) ||
      !size32(dims[0], &r->T) || !size32(dims[2], &r->D) || !size32(r->q.heads, &r->hq) ||
      !size32(r->k.heads, &r->hkv) || !size32(table[0], &r->max_pos) || !size32(table[1], &r->rope_dim))
    return false;
  const size_t need = g_entry.cache_bytes(r->num_pages, r->page_size, r->hkv, r->D);
  return memory(a[at.k_cache], "k_cache", dev, need, &r->kc) &&
         (v == Py_None || memory(a[at.v_cache], "v_cache", dev, need, &r->vc));
}

PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 18)) return nullptr;
  RopeArgs r;
  if (!rope_args(a, {3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17}, &r)) return nullptr;
  return status_of([&] {
    return g_entry.rope_append(r.q.p, r.q.stride, r.k.p, r.k.stride, r.v.p, r.v.stride, r.positions,
                               as<float>(r.cos_sin), r.max_pos, r.rope_dim, r.inter, r.slots, r.T, r.hq, r.hkv, r.D,
                               r.out.p, r.out.stride, r.kc, r.vc, r.num_pages, r.page_size, r.rot_k, r.rot_v, r.h,
                               r.formats, r.status, r.stream);
  });
}

// A norm's gains [D] of the rows' type or float32 (*f32), or None.
bool gains_of(PyObject* t, PyObject* dtype, int64_t dev, int32_t D, const char* what, void** out, int* f32) {
  *out = nullptr;
  *f32 = -1;
  if (t == Py_None) return true;
  bool same, wide, cont;
  int64_t have;
  if (!on_device(t, what, dev) || !has_dtype(t, dtype, &same) || !has_dtype(t, g_f32, &wide) ||
      !contiguous(t, &cont) || !call_i64(t, n_numel, &have) || !address(t, out))
    return false;
  *f32 = wide;
  if ((same || wide) && cont && have == D) return true;
  PyErr_Format(PyExc_ValueError, "%s must be %d contiguous entries of k's type or float32", what, int(D));
  return false;
}

PyObject* norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 22)) return nullptr;
  RopeArgs r;
  void *wq, *wk;
  int fq, fk;
  double eps, offset;
  if (!rope_args(a, {5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 18, 19, 20, 21}, &r) ||
      !gains_of(a[3], r.dtype, r.dev, r.D, "q_weight", &wq, &fq) ||
      !gains_of(a[4], r.dtype, r.dev, r.D, "k_weight", &wk, &fk) || !real_of(a[16], &eps) || !real_of(a[17], &offset))
    return nullptr;
  if (fq >= 0 && fk >= 0 && fq != fk) {
    PyErr_SetString(PyExc_ValueError, "q_weight and k_weight must be of one type");
    return nullptr;
  }
  if (fq == 1 || fk == 1) r.formats |= SAW_FMT_F32_WEIGHT;
  return status_of([&] {
    return g_sparse.norm_rope_append(r.q.p, r.q.stride, r.k.p, r.k.stride, r.v.p, r.v.stride, wq, wk, float(offset),
                                     float(eps), r.positions, as<float>(r.cos_sin), r.max_pos, r.rope_dim, r.inter,
                                     r.slots, r.T, r.hq, r.hkv, r.D, r.out.p, r.out.stride, r.kc, r.vc, r.num_pages,
                                     r.page_size, r.rot_k, r.rot_v, r.h, r.formats, r.status, r.stream);
  });
}

// A table [rows, width] of int32 on the device with this many rows.
bool table_of(PyObject* t, const char* what, int64_t dev, int64_t rows, int32_t** out, int32_t* width) {
  int64_t td[2];
  if (!shape(t, what, 2, td)) return false;
  if (td[0] != rows) {
    PyErr_Format(PyExc_ValueError, "%s must have %lld rows, not %lld", what, (long long)rows, (long long)td[0]);
    return false;
  }
  return words(t, what, dev, -1, out) && size32(td[1], width);
}
// Lists [seqs, kv-heads, width] of int32.
bool lists_of(PyObject* t, const char* what, int64_t dev, int64_t seqs, int32_t hkv, int32_t** out, int32_t* width) {
  int64_t td[3];
  if (!shape(t, what, 3, td)) return false;
  if (td[0] != seqs || td[1] != hkv) {
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, %d, pages]", what, (long long)seqs, int(hkv));
    return false;
  }
  return words(t, what, dev, -1, out) && size32(td[2], width);
}

PyObject* page_summary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 13)) return nullptr;
  int64_t dev, seqs;
  int32_t *tables, *seq_lens, *new_lens, *status;
  int32_t max_new, hkv, D, num_pages, page_size, formats, B, width;
  void *kc, *summary, *stream;
  if (!on_current(a[0], &dev) || !words(a[2], "seq_lens", dev, -1, &seq_lens, &seqs) ||
      !table_of(a[1], "block_tables", dev, seqs, &tables, &width) || !words(a[3], "new_lens", dev, seqs, &new_lens) ||
      !int32_of(a[4], &max_new) || !int32_of(a[5], &hkv) || !int32_of(a[6], &D) || !int32_of(a[7], &num_pages) ||
      !int32_of(a[8], &page_size) || !status_word(a[10], dev, &status) || !stream_of(a[11], dev, &stream) ||
      !flag_of(a[12], &formats) || !size32(seqs, &B) ||
      !memory(a[0], "k_cache", dev, g_entry.cache_bytes(num_pages, page_size, hkv, D), &kc) ||
      !memory(a[9], "summary", dev, g_sparse.summary_bytes(num_pages, hkv, D), &summary))
    return nullptr;
  return status_of([&] {
    return g_sparse.page_summary(kc, tables, width, seq_lens, new_lens, B, max_new, hkv, D, num_pages, page_size,
                                 summary, formats ? SAW_FMT_BF16_META : 0, status, stream);
  });
}

PyObject* select_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 18)) return nullptr;
  PyObject* q = a[0];
  int64_t dev, dims[3];
  int32_t *tables, *seq_lens, *sel_tables, *sel_lens, *sel_pages = nullptr, *status;
  int32_t max_len, hkv, num_pages, page_size, rot_k, h, first, last, formats, B, hq, D, width, take, take2;
  void *pq, *summary, *stream;
  bool cq;
  if (!on_current(q, &dev) || !shape(q, "q", 3, dims) || !formats_of(q, a[17], &formats) || !contiguous(q, &cq) ||
      !address(q, &pq) || !size32(dims[0], &B) || !size32(dims[1], &hq) || !size32(dims[2], &D))
    return nullptr;
  if (!cq) {
    PyErr_SetString(PyExc_ValueError, "q must be contiguous");
    return nullptr;
  }
  if (!table_of(a[2], "block_tables", dev, dims[0], &tables, &width) ||
      !words(a[3], "seq_lens", dev, dims[0], &seq_lens) || !int32_of(a[4], &max_len) || !int32_of(a[5], &hkv) ||
      !int32_of(a[6], &num_pages) || !int32_of(a[7], &page_size) || !flag_of(a[8], &rot_k) || !int32_of(a[9], &h) ||
      !int32_of(a[10], &first) || !int32_of(a[11], &last) ||
      !lists_of(a[12], "sel_tables", dev, dims[0], hkv, &sel_tables, &take) ||
      !words(a[13], "sel_lens", dev, dims[0] * hkv, &sel_lens) || !status_word(a[15], dev, &status) ||
      !stream_of(a[16], dev, &stream) ||
      !memory(a[1], "summary", dev, g_sparse.summary_bytes(num_pages, hkv, D), &summary))
    return nullptr;
  if (a[14] != Py_None) {
    if (!lists_of(a[14], "sel_pages", dev, dims[0], hkv, &sel_pages, &take2)) return nullptr;
    if (take2 != take) {
      PyErr_SetString(PyExc_ValueError, "sel_pages must be of sel_tables' shape");
      return nullptr;
    }
  }
  return status_of([&] {
    return g_sparse.select_pages(pq, summary, tables, width, seq_lens, B, max_len, hq, hkv, D, num_pages, page_size,
                                 rot_k, h, take, first, last, sel_tables, sel_pages, sel_lens, formats, status, stream);
  });
}

PyObject* sparse_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 18)) return nullptr;
  PyObject *q = a[0], *out = a[12], *ws = a[13];
  int64_t dev, dims[3], od[3], bytes = 0;
  int32_t *tables, *lens, *status;
  int32_t max_len, hkv, num_pages, page_size, rot_k, rot_v, h, formats, B, hq, D, take;
  double scale;
  void *pq, *kc, *vc, *po, *pw, *stream;
  bool cq, co, same, f32;
  if (!on_current(q, &dev) || !shape(q, "q", 3, dims) || !formats_of(q, a[17], &formats) ||
      !on_device(out, "out", dev) || !shape(out, "out", 3, od) || !contiguous(q, &cq) || !contiguous(out, &co) ||
      !has_dtype(out, (formats & SAW_FMT_F16_INPUT) ? g_f16 : g_bf16, &same) || !has_dtype(out, g_f32, &f32))
    return nullptr;
  if (!same && !f32) {
    PyErr_SetString(PyExc_ValueError, "out must be float32 or q's type");
    return nullptr;
  }
  if (same) formats |= SAW_FMT_OUT_INPUT;
  if (!cq || !co || dims[0] != od[0] || dims[1] != od[1] || dims[2] != od[2]) {
    PyErr_SetString(PyExc_ValueError, "q and out must be contiguous and of one shape");
    return nullptr;
  }
  if (!int32_of(a[5], &max_len) || !int32_of(a[6], &hkv) ||
      !lists_of(a[3], "sel_tables", dev, dims[0], hkv, &tables, &take) ||
      !words(a[4], "sel_lens", dev, dims[0] * hkv, &lens) || !int32_of(a[7], &num_pages) ||
      !int32_of(a[8], &page_size) || !flag_of(a[9], &rot_k) || !flag_of(a[10], &rot_v) || !int32_of(a[11], &h) ||
      !memory(ws, "workspace", dev, 0, &pw, &bytes) || !real_of(a[14], &scale) || !status_word(a[15], dev, &status) ||
      !stream_of(a[16], dev, &stream) || !address(q, &pq) || !address(out, &po) || !size32(dims[0], &B) ||
      !size32(dims[1], &hq) || !size32(dims[2], &D))
    return nullptr;
  const size_t need = g_entry.cache_bytes(num_pages, page_size, hkv, D);
  if (!memory(a[1], "k_cache", dev, need, &kc) || !memory(a[2], "v_cache", dev, need, &vc)) return nullptr;
  return status_of([&] {
    return g_sparse.sparse_decode(pq, kc, vc, tables, take, lens, B, max_len, hq, hkv, D, num_pages, page_size, rot_k,
                                  rot_v, h, float(scale), po, pw, size_t(bytes), formats, status, stream);
  });
}

PyObject* prefix_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 22)) return nullptr;
  PyObject *q = a[0], *out = a[15], *ws = a[16];
  int64_t dev, dims[3], od[3], td[2], groups, bytes = 0;
  int32_t *tables, *seq_lens, *cu, *prefix, *status;
  int32_t max_prefix, max_own, hkv, num_pages, page_size, rot_k, rot_v, h, mode, formats, B, hq, D, G, width;
  double scale;
  void *pq, *kc, *vc, *po, *pw, *stream;
  bool cq, co, same, f32;
  if (!on_current(q, &dev) || !shape(q, "q", 3, dims) || !formats_of(q, a[20], &formats) ||
      !on_device(out, "out", dev) || !shape(out, "out", 3, od) || !contiguous(q, &cq) || !contiguous(out, &co) ||
      !has_dtype(out, (formats & SAW_FMT_F16_INPUT) ? g_f16 : g_bf16, &same) || !has_dtype(out, g_f32, &f32))
    return nullptr;
  if (!same && !f32) {
    PyErr_SetString(PyExc_ValueError, "out must be float32 or q's type");
    return nullptr;
  }
  if (same) formats |= SAW_FMT_OUT_INPUT;
  if (!cq || !co || dims[0] != od[0] || dims[1] != od[1] || dims[2] != od[2]) {
    PyErr_SetString(PyExc_ValueError, "q and out must be contiguous and of one shape");
    return nullptr;
  }
  if (!shape(a[3], "block_tables", 2, td)) return nullptr;
  if (td[0] != dims[0]) {
    PyErr_Format(PyExc_ValueError, "block_tables must have %lld rows, not %lld", (long long)dims[0], (long long)td[0]);
    return nullptr;
  }
  if (!memory(ws, "workspace", dev, 0, &pw, &bytes)) return nullptr;
  if (!words(a[3], "block_tables", dev, -1, &tables) || !words(a[4], "seq_lens", dev, dims[0], &seq_lens) ||
      !words(a[6], "prefix_lens", dev, -1, &prefix, &groups) || !words(a[5], "cu_group_seqs", dev, groups + 1, &cu) ||
      !int32_of(a[7], &max_prefix) || !int32_of(a[8], &max_own) || !int32_of(a[9], &hkv) ||
      !int32_of(a[10], &num_pages) || !int32_of(a[11], &page_size) || !flag_of(a[12], &rot_k) ||
      !flag_of(a[13], &rot_v) || !int32_of(a[14], &h) || !real_of(a[17], &scale) ||
      !status_word(a[18], dev, &status) || !stream_of(a[19], dev, &stream) || !int32_of(a[21], &mode) ||
      !address(q, &pq) || !address(out, &po) || !size32(dims[0], &B) || !size32(dims[1], &hq) ||
      !size32(dims[2], &D) || !size32(groups, &G) || !size32(td[1], &width))
    return nullptr;
  const size_t need = g_entry.cache_bytes(num_pages, page_size, hkv, D);
  if (!memory(a[1], "k_cache", dev, need, &kc) || !memory(a[2], "v_cache", dev, need, &vc)) return nullptr;
  return status_of([&] {
    return g_entry.prefix_decode(pq, kc, vc, tables, width, seq_lens, cu, prefix, G, B, max_prefix, max_own, hq, hkv, D,
                                 num_pages, page_size, rot_k, rot_v, h, float(scale), po, pw, size_t(bytes), mode,
                                 formats, status, stream);
  });
}

// (five entry points' addresses; dtypes int32, float32, bfloat16, float16;
// current device; current raw stream of a device)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  uint64_t at[5];
  for (int i = 0; i < 5; ++i) {
    at[i] = PyLong_AsUnsignedLongLong(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_entry = {reinterpret_cast<decltype(Entry::build_tables)>(at[0]), reinterpret_cast<decltype(Entry::rope_table)>(at[1]),
             reinterpret_cast<decltype(Entry::rope_append)>(at[2]),
             reinterpret_cast<decltype(Entry::prefix_decode)>(at[3]),
             reinterpret_cast<decltype(Entry::cache_bytes)>(at[4])};
  PyObject** const keep[6] = {&g_int32, &g_f32, &g_bf16, &g_f16, &g_device, &g_raw_stream};
  for (int i = 0; i < 6; ++i) Py_XSETREF(*keep[i], Py_NewRef(a[5 + i]));
  Py_RETURN_NONE;
}

// (five entry points' addresses; after init, whose other arguments hold here too)
PyObject* init_sparse(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 5)) return nullptr;
  uint64_t at[5];
  for (int i = 0; i < 5; ++i) {
    at[i] = PyLong_AsUnsignedLongLong(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_sparse = {reinterpret_cast<decltype(SparseEntry::norm_rope_append)>(at[0]),
              reinterpret_cast<decltype(SparseEntry::page_summary)>(at[1]),
              reinterpret_cast<decltype(SparseEntry::select_pages)>(at[2]),
              reinterpret_cast<decltype(SparseEntry::sparse_decode)>(at[3]),
              reinterpret_cast<decltype(SparseEntry::summary_bytes)>(at[4])};
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(init)), METH_FASTCALL, nullptr},
    {"build_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(build_tables)), METH_FASTCALL, nullptr},
    {"rope_table", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_table)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_append)), METH_FASTCALL, nullptr},
    {"prefix_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_decode)), METH_FASTCALL, nullptr},
    {"init_sparse", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(init_sparse)), METH_FASTCALL, nullptr},
    {"norm_rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rope_append)), METH_FASTCALL,
     nullptr},
    {"page_summary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(page_summary)), METH_FASTCALL, nullptr},
    {"select_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(select_pages)), METH_FASTCALL, nullptr},
    {"sparse_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sparse_decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_saw_step", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__saw_step(void) {
  struct {
    PyObject** at;
    const char* name;
  } const names[] = {{&n_dtype, "dtype"},   {&n_data_ptr, "data_ptr"},     {&n_contiguous, "is_contiguous"},
                     {&n_numel, "numel"},   {&n_shape, "shape"},           {&n_stride, "stride"},
                     {&n_get_device, "get_device"}, {&n_cuda_stream, "cuda_stream"}, {&n_nbytes, "nbytes"}};
  for (const auto& x : names)
    if (!(*x.at = PyUnicode_InternFromString(x.name))) return nullptr;
  return PyModule_Create(&g_module);
}
