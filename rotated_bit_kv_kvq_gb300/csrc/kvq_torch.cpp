// The step operators for torch tensors (kvq.py's functions of the same names): checks of types,
// shapes, strides and devices, then the C ABI.  Compiled rather than written in Python because a
// call has up to ten tensors and the GPU's part of a decode step's call takes four microseconds:
// the checks and argument conversions took six of them, here half a microsecond.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "kvq.h"

namespace {

using at::Tensor;
using Shape = std::initializer_list<int64_t>;

// the memory of a ctypes structure (its buffer) for the length of a call
template <class T>
struct Struct {
  Py_buffer view{};
  bool held = false;
  Struct(PyObject* o, const char* what, bool given = true) {
    if (!given) return;
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      throw std::invalid_argument(std::string(what) + ": not a descriptor");
    }
    held = true;
    if (view.len != Py_ssize_t(sizeof(T))) {
      PyBuffer_Release(&view);
      held = false;
      throw std::invalid_argument(std::string(what) + ": a descriptor of another kind");
    }
  }
  ~Struct() { if (held) PyBuffer_Release(&view); }
  const T* get() const { return static_cast<const T*>(view.buf); }
  const T* operator->() const { return get(); }
};

// a tensor argument; NULL for None where that is allowed
const Tensor* tensor(PyObject* o, const char* what, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(what) + ": a tensor is expected");
  return &THPVariable_Unpack(o);
}

int dtype_id(at::ScalarType t) {
  return t == at::kFloat ? KVQ_F32 : t == at::kBFloat16 ? KVQ_BF16 : t == at::kHalf ? KVQ_F16 : -1;
}

[[noreturn]] void refuse(const char* what, const Tensor& t, const std::string& want) {
  std::ostringstream s;
  s << what << ": expected " << want << "; got " << t.sizes() << " of " << t.scalar_type() << " on " << t.device();
  throw std::invalid_argument(s.str());
}

// contiguous, on CUDA device `dev` (torch's current one)
void* plain(const char* what, const Tensor& t, int dev) {
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    refuse(what, t, "a contiguous tensor on CUDA device " + std::to_string(dev));
  return t.data_ptr();
}
void* ints(const char* what, const Tensor* t, int dev, Shape shape) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->sizes() != at::IntArrayRef(shape)) {
    std::ostringstream s;
    s << at::IntArrayRef(shape) << " of Int";
    refuse(what, *t, s.str());
  }
  return plain(what, *t, dev);
}
int floats(const char* what, const Tensor& t, Shape shape) {
  const int id = dtype_id(t.scalar_type());
  if (id < 0 || t.sizes() != at::IntArrayRef(shape)) {
    std::ostringstream s;
    s << at::IntArrayRef(shape) << " of fp32, bf16 or fp16";
    refuse(what, t, s.str());
  }
  return id;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw std::invalid_argument("an integer is expected");
  }
  return v;
}
int32_t int32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw std::invalid_argument("an integer does not fit 32 bits");
  return int32_t(v);
}

// None: torch's current stream; an integer handle; or an object with cuda_stream
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  if (PyLong_Check(o)) return reinterpret_cast<void*>(uintptr_t(integer(o)));
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) {
    PyErr_Clear();
    throw std::invalid_argument("stream: None, a handle or a torch.cuda.Stream is expected");
  }
  const int64_t v = PyLong_AsLongLong(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw std::invalid_argument("stream: no handle");
  }
  return reinterpret_cast<void*>(uintptr_t(v));
}

// Runs f (which returns the call's status); the arguments' errors become ValueError.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  try {
    if (n != want) throw std::invalid_argument("wrong number of arguments");
    return PyLong_FromLong(f());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "kvq: unknown error");
  }
  return nullptr;
}
#define KVQ_LAUNCH(call)      \
  kvq_status status;          \
  Py_BEGIN_ALLOW_THREADS      \
  status = (call);            \
  Py_END_ALLOW_THREADS        \
  return status

// Row stride of projection rows [n][heads * d] or [n][heads][d] whose heads lie side by side.
int64_t row_stride(const char* what, const Tensor& t, int dev, at::ScalarType dt, int64_t n, int64_t heads, int64_t d) {
  bool ok = t.scalar_type() == dt && t.is_cuda() && t.get_device() == dev;
  if (ok && t.dim() == 2) {
    ok = t.size(0) == n && t.size(1) == heads * d && (n == 0 || t.stride(1) == 1);
  } else if (ok) {
    ok = t.dim() == 3 && t.size(0) == n && t.size(1) == heads && t.size(2) == d &&
         (n == 0 || (t.stride(2) == 1 && (heads == 1 || t.stride(1) == d)));
  }
  if (!ok) {
    std::ostringstream s;
    s << n << " rows of " << heads << " x " << d << " values of " << dt << ", heads side by side, on CUDA device " << dev;
    refuse(what, t, s.str());
  }
  return n > 1 ? t.stride(0) : heads * d;  // (a single row's stride is free: torch may report any number)
}

// (cache, plan, weight_dim, q, k, v, pos, q_out, k_out, v_out, dst_row, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> kvq_status {
    static const char* const me = "kvq_qk_norm_rope";
    const Struct<kvq_cache> c(a[0], me);
    const Struct<kvq_rope_norm> r(a[1], me);
    const int64_t wd = integer(a[2]), d = c->head_dim, hkv = c->n_kv_heads;
    const Tensor &q = *tensor(a[3], me), &k = *tensor(a[4], me), &pos = *tensor(a[6], me);
    const Tensor &qo = *tensor(a[7], me), &ko = *tensor(a[8], me);
    const Tensor *v = tensor(a[5], me, true), *vo = tensor(a[9], me, true), *dst = tensor(a[10], me, true);
    const int dev = c10::cuda::current_device();
    const at::ScalarType dt = q.scalar_type();
    if (wd && wd != d) throw std::invalid_argument("kvq_qk_norm_rope: the weights have not head_dim values");
    if (dtype_id(dt) < 0 || q.dim() < 1) refuse(me, q, "rows of fp32, bf16 or fp16");
    if (qo.dim() < 2 || qo.size(-1) != d || qo.size(-2) < 1) refuse(me, qo, "[..][heads][head_dim] outputs");
    const int64_t rows_in = q.size(0), hq = qo.size(-2), rows = qo.numel() / (hq * d);
    if (rows_in > INT32_MAX || rows > INT32_MAX || hq > INT32_MAX) throw std::invalid_argument("kvq_qk_norm_rope: too many rows");
    for (const Tensor* o : {&qo, &ko, vo})
      if (o && (o->scalar_type() != dt || (o != &qo && o->numel() != rows * hkv * d)))
        refuse(me, *o, "outputs of the inputs' type, of the same rows");
    const int64_t qs = row_stride("kvq_qk_norm_rope: q", q, dev, dt, rows_in, hq, d);
    const int64_t ks = row_stride("kvq_qk_norm_rope: k", k, dev, dt, rows_in, hkv, d);
    const int64_t vs = v ? row_stride("kvq_qk_norm_rope: v", *v, dev, dt, rows_in, hkv, d) : 0;
    const auto* p = static_cast<const int32_t*>(ints("kvq_qk_norm_rope: pos", &pos, dev, {rows_in}));
    const auto* ds = static_cast<const int32_t*>(ints("kvq_qk_norm_rope: dst_row", dst, dev, {rows_in}));
    void *qp = plain(me, qo, dev), *kp = plain(me, ko, dev), *vp = vo ? plain(me, *vo, dev) : nullptr;
    void* st = stream_of(a[11]);
    KVQ_LAUNCH(kvq_qk_norm_rope(c.get(), r.get(), dtype_id(dt), int32_t(hq), q.data_ptr(), qs, k.data_ptr(), ks,
                                v ? v->data_ptr() : nullptr, vs, p, ds, int32_t(rows_in), int32_t(rows), qp, kp, vp, st));
  });
}

// (cache, pool, pages of the pool, n_new, n_new_max, granted, row_pos, row_dst, row_slot, seq_len_out, stream)
PyObject* page_update(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> kvq_status {
    static const char* const me = "kvq_page_update";
    const Struct<kvq_cache> c(a[0], me);
    const Struct<kvq_page_pool> pool(a[1], me);
    if (integer(a[2]) < c->n_pages) throw std::invalid_argument("kvq_page_update: the pool was made for fewer pages");
    const Tensor &want = *tensor(a[3], me), &granted = *tensor(a[5], me);
    const int32_t widest = int32(a[4]);
    const Tensor *maps[3] = {tensor(a[6], me, true), tensor(a[7], me, true), tensor(a[8], me, true)};
    const Tensor* after = tensor(a[9], me, true);
    const int dev = c10::cuda::current_device();
    const int64_t batch = c->batch;
    int64_t rows = std::min<int64_t>(std::max<int64_t>(batch * widest, 0), INT32_MAX);  // without maps no limit of rows
    for (const Tensor* m : maps)
      if (m) rows = m->numel();
    if (rows > INT32_MAX) throw std::invalid_argument("kvq_page_update: too many rows");
    int32_t* out[3];
    for (int i = 0; i < 3; ++i) out[i] = static_cast<int32_t*>(ints("kvq_page_update: row maps", maps[i], dev, {rows}));
    const auto* w = static_cast<const int32_t*>(ints("kvq_page_update: n_new", &want, dev, {batch}));
    auto* g = static_cast<int32_t*>(ints("kvq_page_update: granted", &granted, dev, {batch}));
    auto* s = static_cast<int32_t*>(ints("kvq_page_update: seq_len_out", after, dev, {batch}));
    void* st = stream_of(a[10]);
    KVQ_LAUNCH(kvq_page_update(c.get(), pool.get(), w, widest, g, int32_t(rows), out[0], out[1], out[2], s, st));
  });
}

// (cache, index, n_last, stream)
PyObject* block_index_update(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> kvq_status {
    const Struct<kvq_cache> c(a[0], "kvq_block_index_update");
    const Struct<kvq_block_index> x(a[1], "kvq_block_index_update");
    const int32_t last = int32(a[2]);
    void* st = stream_of(a[3]);
    KVQ_LAUNCH(kvq_block_index_update(c.get(), x.get(), last, st));
  });
}

// (cache, index, q, sel, n_first, n_last, stream)
PyObject* select_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> kvq_status {
    const Struct<kvq_cache> c(a[0], "kvq_select_blocks");
    const Struct<kvq_block_index> x(a[1], "kvq_select_blocks");
    const Tensor &q = *tensor(a[2], "kvq_select_blocks: q"), &sel = *tensor(a[3], "kvq_select_blocks: sel");
    const int32_t first = int32(a[4]), last = int32(a[5]);
    const int dev = c10::cuda::current_device();
    const int64_t hq = q.dim() == 3 ? q.size(1) : 0, m = sel.dim() == 3 ? sel.size(2) : 0;
    const int id = floats("kvq_select_blocks: q", q, {c->batch, hq, c->head_dim});
    auto* sp = static_cast<int32_t*>(ints("kvq_select_blocks: sel", &sel, dev, {c->batch, c->n_kv_heads, m}));
    const void* qp = plain("kvq_select_blocks: q", q, dev);
    if (hq > INT32_MAX || m > INT32_MAX) throw std::invalid_argument("kvq_select_blocks: sizes do not fit 32 bits");
    void* st = stream_of(a[6]);
    KVQ_LAUNCH(kvq_select_blocks(c.get(), x.get(), qp, id, int32_t(hq), first, last, int32_t(m), sp, st));
  });
}

// (cache, q, sel, out, block_tokens, scale, stream)
PyObject* sparse_decode_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> kvq_status {
    static const char* const me = "kvq_sparse_decode_attention";
    const Struct<kvq_cache> c(a[0], me);
    const Tensor &q = *tensor(a[1], me), &sel = *tensor(a[2], me), &out = *tensor(a[3], me);
    const int32_t bt = int32(a[4]);
    const double scale = PyFloat_AsDouble(a[5]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw std::invalid_argument("kvq_sparse_decode_attention: scale is a number");
    }
    const int dev = c10::cuda::current_device();
    const int64_t hq = q.dim() == 3 ? q.size(1) : 0, m = sel.dim() == 3 ? sel.size(2) : 0;
    const int id = floats("kvq_sparse_decode_attention: q", q, {c->batch, hq, c->head_dim});
    const int od = floats("kvq_sparse_decode_attention: out", out, {c->batch, hq, c->head_dim});
    const auto* sp = static_cast<const int32_t*>(ints("kvq_sparse_decode_attention: sel", &sel, dev, {c->batch, c->n_kv_heads, m}));
    const void* qp = plain("kvq_sparse_decode_attention: q", q, dev);
    void* op = plain("kvq_sparse_decode_attention: out", out, dev);
    if (hq > INT32_MAX || m > INT32_MAX) throw std::invalid_argument("kvq_sparse_decode_attention: sizes do not fit 32 bits");
    void* st = stream_of(a[6]);
    KVQ_LAUNCH(kvq_sparse_decode_attention(c.get(), qp, id, int32_t(hq), float(scale), bt, sp, int32_t(m), op, od, st));
  });
}

int32_t* int_out(const char* what, const Tensor* t, int dev, Shape shape) {
  return static_cast<int32_t*>(ints(what, t, dev, shape));
}
// pages of a pool or of counts (what they were made for) against the cache's
void for_pages(const char* what, PyObject* pages, const kvq_cache* c) {
  if (integer(pages) < c->n_pages) throw std::invalid_argument(std::string(what) + ": the pool or the counts were made for fewer pages");
}

// (cache, pool, share, pages, src, dst, granted, n_tokens, seq_len_out, stream)
PyObject* page_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> kvq_status {
    static const char* const me = "kvq_page_fork";
    const Struct<kvq_cache> c(a[0], me);
    const Struct<kvq_page_pool> pool(a[1], me);
    const Struct<kvq_page_share> share(a[2], me);
    for_pages(me, a[3], c.get());
    const Tensor &src = *tensor(a[4], me), &dst = *tensor(a[5], me), &granted = *tensor(a[6], me);
    const Tensor *count = tensor(a[7], me, true), *after = tensor(a[8], me, true);
    const int dev = c10::cuda::current_device();
    const int64_t forks = src.numel();
    if (forks > INT32_MAX) throw std::invalid_argument("kvq_page_fork: too many forks");
    const int32_t* s = int_out("kvq_page_fork: src", &src, dev, {forks});
    const int32_t* d = int_out("kvq_page_fork: dst", &dst, dev, {forks});
    int32_t* g = int_out("kvq_page_fork: granted", &granted, dev, {forks});
    const int32_t* k = int_out("kvq_page_fork: n_tokens", count, dev, {forks});
    int32_t* l = after ? int_out("kvq_page_fork: seq_len_out", after, dev, {c->batch}) : c->seq_len;
    void* st = stream_of(a[9]);
    KVQ_LAUNCH(kvq_page_fork(c.get(), pool.get(), share.get(), s, d, k, int32_t(forks), g, l, st));
  });
}

// (cache, pool, share, pages, release, seq_len_out, stream)
PyObject* page_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> kvq_status {
    static const char* const me = "kvq_page_free";
    const Struct<kvq_cache> c(a[0], me);
    const Struct<kvq_page_pool> pool(a[1], me);
    const Struct<kvq_page_share> share(a[2], me);
    for_pages(me, a[3], c.get());
    const Tensor& release = *tensor(a[4], me);
    const Tensor* after = tensor(a[5], me, true);
    const int dev = c10::cuda::current_device();
    const int32_t* r = int_out("kvq_page_free: release", &release, dev, {c->batch});
    int32_t* l = after ? int_out("kvq_page_free: seq_len_out", after, dev, {c->batch}) : c->seq_len;
    void* st = stream_of(a[6]);
    KVQ_LAUNCH(kvq_page_free(c.get(), pool.get(), share.get(), r, l, st));
  });
}

// (cache, pool, share or None, pages, table_out or None, ring_out or None, workspace, page_map or None, stream)
PyObject* page_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> kvq_status {
    static const char* const me = "kvq_page_compact";
    const Struct<kvq_cache> c(a[0], me);
    const Struct<kvq_page_pool> pool(a[1], me);
    const bool counts = a[2] != Py_None;
    const Struct<kvq_page_share> share(counts ? a[2] : a[1], me, counts);
    for_pages(me, a[3], c.get());
    const Tensor *table = tensor(a[4], me, true), *ring = tensor(a[5], me, true), *map = tensor(a[7], me, true);
    const Tensor& ws = *tensor(a[6], me);
    const int dev = c10::cuda::current_device();
    const int64_t per = c->page_tokens > 0 ? c->max_ctx / c->page_tokens : 0;
    int32_t* t = table ? int_out("kvq_page_compact: table_out", table, dev, {c->batch, per}) : const_cast<int32_t*>(c->page_table);
    int32_t* r = ring ? int_out("kvq_page_compact: ring_out", ring, dev, {c->n_pages}) : pool->ring;
    int32_t* m = int_out("kvq_page_compact: page_map", map, dev, {c->n_pages});
    void* w = plain("kvq_page_compact: workspace", ws, dev);
    const size_t bytes = size_t(ws.numel()) * ws.element_size();
    void* st = stream_of(a[8]);
    KVQ_LAUNCH(kvq_page_compact(c.get(), pool.get(), counts ? share.get() : nullptr, t, r, m, w, bytes, st));
  });
}

// (cache, mod or None, slopes, first_key, prefix_len, q, row_start, out, workspace, scale, stream); the three tensors are mod's, or None
PyObject* chunk_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> kvq_status {
    static const char* const me = "kvq_chunk_attention";
    const Struct<kvq_cache> c(a[0], me);
    const bool mods = a[1] != Py_None;
    const Struct<kvq_score_mod> mod(mods ? a[1] : a[0], me, mods);
    const Tensor *slopes = tensor(a[2], me, true), *first = tensor(a[3], me, true), *prefix = tensor(a[4], me, true);
    const Tensor &q = *tensor(a[5], me), &start = *tensor(a[6], me), &out = *tensor(a[7], me), &ws = *tensor(a[8], me);
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw std::invalid_argument("kvq_chunk_attention: scale is a number");
    }
    const int dev = c10::cuda::current_device();
    const int64_t rows = q.dim() == 3 ? q.size(0) : 0, hq = q.dim() == 3 ? q.size(1) : 0;
    const int id = floats("kvq_chunk_attention: q", q, {rows, hq, c->head_dim});
    const int od = floats("kvq_chunk_attention: out", out, {rows, hq, c->head_dim});
    const int32_t* s = int_out("kvq_chunk_attention: row_start", &start, dev, {int64_t(c->batch) + 1});
    if (slopes && slopes->sizes() != at::IntArrayRef({hq})) refuse("kvq_chunk_attention: slopes", *slopes, "a value per query head");
    if (slopes) plain("kvq_chunk_attention: slopes", *slopes, dev);
    int_out("kvq_chunk_attention: first_key", first, dev, {rows});
    int_out("kvq_chunk_attention: prefix_len", prefix, dev, {c->batch});
    const void* qp = plain("kvq_chunk_attention: q", q, dev);
    void* op = plain("kvq_chunk_attention: out", out, dev);
    void* w = plain("kvq_chunk_attention: workspace", ws, dev);
    if (rows > INT32_MAX || hq > INT32_MAX) throw std::invalid_argument("kvq_chunk_attention: sizes do not fit 32 bits");
    const size_t bytes = size_t(ws.numel()) * ws.element_size();
    void* st = stream_of(a[10]);
    KVQ_LAUNCH(kvq_chunk_attention(c.get(), mods ? mod.get() : nullptr, qp, id, int32_t(hq), int32_t(rows), s, float(scale), op,
                                   od, w, bytes, st));
  });
}

#define KVQ_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KVQ_METHOD(qk_norm_rope), KVQ_METHOD(page_update), KVQ_METHOD(block_index_update),
                         KVQ_METHOD(select_blocks), KVQ_METHOD(sparse_decode_attention), KVQ_METHOD(page_fork),
                         KVQ_METHOD(page_free), KVQ_METHOD(page_compact), KVQ_METHOD(chunk_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvq_torch(void) { return PyModule_Create(&module); }
