// The serving operators' Python binding: checks torch tensors, allocates
// outputs and workspaces through torch, takes the current stream and calls the
// C ABI.  A decode step calls these operators once or more for every layer, so
// the call itself counts: in C++ it costs 3.5 to 7 us where the same checks in
// Python with ctypes cost 13 to 20 us, more than the kernels of a small step.
//
// The C functions are not linked: serving.py hands over their addresses in
// the library that it has loaded (bind).  Each function returns its result,
// or a non-zero ttq_status as an int, which serving.py raises.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <initializer_list>

#include "../../include/ttq.h"

namespace {

decltype(&ttq_cache_write) p_write;
decltype(&ttq_cache_copy_pages) p_copy;
decltype(&ttq_paged_attention_workspace_bytes) p_attention_ws;
decltype(&ttq_paged_attention) p_attention;
decltype(&ttq_token_logprobs_workspace_bytes) p_logprobs_ws;
decltype(&ttq_token_logprobs) p_logprobs;
decltype(&ttq_cache_append) p_append;
decltype(&ttq_packed_append) p_packed_append;
decltype(&ttq_packed_read) p_packed_read;
decltype(&ttq_packed_copy_pages) p_packed_copy;
decltype(&ttq_packed_attention_workspace_bytes) p_packed_attention_ws;
decltype(&ttq_packed_attention) p_packed_attention;
decltype(&ttq_beam_select_workspace_bytes) p_beams_ws;
decltype(&ttq_beam_select) p_beams;

using at::ScalarType;
using at::Tensor;

// A Python exception is set; the function returns NULL.
struct Raised {};

[[noreturn]] void raise(PyObject* kind, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(kind, fmt, ap);
  va_end(ap);
  throw Raised{};
}

const char* name_of(ScalarType t) { return c10::toString(t); }

const Tensor& gpu(PyObject* o, const char* name, int device = -1) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch tensor", name);
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be on the GPU (got %s)", name, t.device().str().c_str());
  if (device >= 0 && t.get_device() != device)
    raise(PyExc_ValueError, "%s must be on the GPU cuda:%d (got %s)", name, device, t.device().str().c_str());
  return t;
}

void want(const Tensor& t, const char* name, ScalarType type) {
  if (t.scalar_type() != type) raise(PyExc_TypeError, "%s must be %s (got %s)", name, name_of(type), name_of(t.scalar_type()));
}

void* vector(PyObject* o, const char* name, ScalarType type, int64_t n, int device) {
  const Tensor& t = gpu(o, name, device);
  want(t, name, type);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    raise(PyExc_ValueError, "%s must be a dense vector of %lld values", name, (long long)n);
  return t.data_ptr();
}

// a [rows][cols] tensor with unit column stride; its row stride in *ld
void* rows_of(const Tensor& t, const char* name, int64_t rows, int64_t cols, ScalarType type, int64_t* ld) {
  want(t, name, type);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || (cols > 1 && t.stride(1) != 1))
    raise(PyExc_ValueError, "%s must be [%lld][%lld] with unit column stride", name, (long long)rows, (long long)cols);
  *ld = rows > 1 ? t.stride(0) : (cols + 7) / 8 * 8;
  return t.data_ptr();
}

// One layer's cache, k and v [pages][kv heads][page size][head dim], after
// `skip` leading dimensions (layers).  `last` names the last dimension.
template <typename Cache>
void pages_of(Cache& c, const Tensor& k, const Tensor& v, int skip, const char* last) {
  if (k.dim() != 4 + skip || k.sizes() != v.sizes())
    raise(PyExc_ValueError, "kcache and vcache must be [pages][kv heads][page size][%s], of one shape", last);
  const int64_t n = k.size(skip), h = k.size(skip + 1), p = k.size(skip + 2), d = k.size(skip + 3);
  const int64_t stride = n > 1 ? k.stride(skip) : h * p * d;
  if (n > 1 && v.stride(skip) != stride) raise(PyExc_ValueError, "kcache and vcache must have one page stride");
  for (const Tensor* t : {&k, &v})
    if ((d > 1 && t->stride(skip + 3) != 1) || (p > 1 && t->stride(skip + 2) != d) ||
        (h > 1 && t->stride(skip + 1) != p * d))
      raise(PyExc_ValueError, "a page of the cache must be dense: [kv heads][page size][%s]", last);
  if (h > INT32_MAX || p > INT32_MAX || d > INT32_MAX) raise(PyExc_ValueError, "a page of the cache is too large");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.n_pages = n;
  c.page_stride = stride;
  c.n_kv_heads = (int32_t)h;
  c.page_size = (int32_t)p;
  c.head_dim = (int32_t)d;
}
ttq_paged_cache cache_of(const Tensor& k, const Tensor& v, int skip) {
  ttq_paged_cache c{};
  const ScalarType type = k.scalar_type();
  if (type != ScalarType::Half && type != ScalarType::BFloat16)
    raise(PyExc_TypeError, "kcache must be Half or BFloat16 (got %s)", name_of(type));
  want(v, "vcache", type);
  pages_of(c, k, v, skip, "head dim");
  c.dtype = type == ScalarType::Half ? TTQ_F16 : TTQ_BF16;
  return c;
}
// A layer's cache in 4 bits, bytes [pages][kv heads][page size][5/8 head dim];
// `type` is that of its queries, keys and values.
ttq_packed_cache packed_of(const Tensor& k, const Tensor& v, int skip, ScalarType type) {
  ttq_packed_cache c{};
  want(k, "kcache", ScalarType::Byte);
  want(v, "vcache", ScalarType::Byte);
  if (type != ScalarType::Half && type != ScalarType::BFloat16)
    raise(PyExc_TypeError, "a 4-bit cache takes Half or BFloat16 rows (got %s)", name_of(type));
  pages_of(c, k, v, skip, "5/8 head dim");
  if (c.head_dim % 5 != 0) raise(PyExc_ValueError, "rows of %d bytes are not 5/8 of a head dim", c.head_dim);
  c.head_dim = c.head_dim / 5 * 8;
  c.dtype = type == ScalarType::Half ? TTQ_F16 : TTQ_BF16;
  return c;
}

int32_t* table_of(PyObject* o, const char* name, int device, int64_t* rows, int64_t* cols, int64_t* stride) {
  const Tensor& t = gpu(o, name, device);
  want(t, name, ScalarType::Int);
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1) || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
    raise(PyExc_ValueError, "%s must be [rows][blocks] with unit column stride", name);
  *rows = t.size(0);
  *cols = t.size(1);
  *stride = *rows > 1 ? t.stride(0) : *cols;
  return static_cast<int32_t*>(t.data_ptr());
}

ttq_paged_batch batch_of(PyObject* table, PyObject* q_start, PyObject* kv_len, int64_t total, int max_q, int max_kv,
                         int device) {
  ttq_paged_batch b{};
  int64_t n, blocks;
  b.block_table = table_of(table, "block_table", device, &n, &blocks, &b.table_stride);
  b.q_start = static_cast<int32_t*>(vector(q_start, "q_start", ScalarType::Int, n + 1, device));
  b.kv_len = static_cast<int32_t*>(vector(kv_len, "kv_len", ScalarType::Int, n, device));
  b.n_blocks = (int32_t)blocks;
  b.n_seqs = (int32_t)n;
  b.total_q = total;
  b.max_q_len = max_q;
  b.max_kv_len = max_kv;
  return b;
}

double number(PyObject* o, const char* name) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}
int whole(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_ValueError, "%s=%lld is out of range", name, x);
  return (int)x;
}

void* stream_of(int device) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }

Tensor make(at::IntArrayRef sizes, ScalarType type, int device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
}

// the caller's workspace, or one of torch's when `need` bytes are needed
void* workspace(PyObject* given, size_t need, int device, Tensor* own, size_t* bytes) {
  if (given != Py_None) {
    const Tensor& t = gpu(given, "workspace", device);
    want(t, "workspace", ScalarType::Byte);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
    *bytes = (size_t)t.numel();
    return t.data_ptr();
  }
  *bytes = need;
  if (need == 0) return nullptr;
  *own = make({(int64_t)need}, ScalarType::Byte, device);
  return own->data_ptr();
}

void arguments(Py_ssize_t got, Py_ssize_t n, const char* f) {
  if (got != n) raise(PyExc_TypeError, "%s takes %d arguments", f, (int)n);
  if (p_write == nullptr) raise(PyExc_RuntimeError, "the library is not bound");
}

// Work is enqueued for the tensors' device whatever the current one is.
class OnDevice {
 public:
  explicit OnDevice(int device) {
    if (hipGetDevice(&was_) != hipSuccess || was_ == device) was_ = -1;
    else if (hipSetDevice(device) != hipSuccess) raise(PyExc_RuntimeError, "cannot use GPU %d", device);
  }
  ~OnDevice() {
    if (was_ >= 0) (void)hipSetDevice(was_);
  }

 private:
  int was_;
};

// The addresses of the functions, in this order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** const to[] = {
      reinterpret_cast<void**>(&p_write),         reinterpret_cast<void**>(&p_copy),
      reinterpret_cast<void**>(&p_attention_ws),  reinterpret_cast<void**>(&p_attention),
      reinterpret_cast<void**>(&p_logprobs_ws),   reinterpret_cast<void**>(&p_logprobs),
      reinterpret_cast<void**>(&p_append),        reinterpret_cast<void**>(&p_packed_append),
      reinterpret_cast<void**>(&p_packed_read),   reinterpret_cast<void**>(&p_packed_copy),
      reinterpret_cast<void**>(&p_packed_attention_ws), reinterpret_cast<void**>(&p_packed_attention),
      reinterpret_cast<void**>(&p_beams_ws),      reinterpret_cast<void**>(&p_beams),
  };
  constexpr int N = sizeof(to) / sizeof(to[0]);
  if (n != N) return PyErr_Format(PyExc_TypeError, "bind takes %d addresses", N);
  void* p[N];
  for (int i = 0; i < N; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "address %d is NULL", i);
  }
  for (int i = 0; i < N; ++i) *to[i] = p[i];
  Py_RETURN_NONE;
}

// K, V, kcache, vcache, block_table, q_start, kv_len
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 7, "cache_write");
    const Tensor &kc = gpu(a[2], "kcache"), &vc = gpu(a[3], "vcache", kc.get_device());
    const int dev = kc.get_device();
    const ttq_paged_cache c = cache_of(kc, vc, 0);
    const Tensor &K = gpu(a[0], "K", dev), &V = gpu(a[1], "V", dev);
    const int64_t rows = K.dim() > 0 ? K.size(0) : 0, cols = (int64_t)c.n_kv_heads * c.head_dim;
    int64_t ldk, ldv;
    void* k = rows_of(K, "K", rows, cols, kc.scalar_type(), &ldk);
    void* v = rows_of(V, "V", rows, cols, kc.scalar_type(), &ldv);
    const ttq_paged_batch b = batch_of(a[4], a[5], a[6], rows, 0, 0, dev);
    OnDevice on(dev);
    const ttq_status s = p_write(&c, &b, k, ldk, v, ldv, stream_of(dev));
    if (s != TTQ_OK) return PyLong_FromLong(s);
    Py_RETURN_NONE;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <typename Of, typename Copy>
PyObject* copy_pages(PyObject* const* a, Py_ssize_t n, const char* name, Of of, Copy* copy) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 5, name);
    const Tensor &kc = gpu(a[0], "kcache"), &vc = gpu(a[1], "vcache", kc.get_device());
    const int dev = kc.get_device();
    const int skip = kc.dim() == 5 ? 1 : 0;
    const auto c = of(kc, vc, skip);
    int64_t layers = 1, layer_stride = 0;
    if (skip) {
      layers = kc.size(0);
      layer_stride = kc.stride(0);
      if (layers < 1 || layers > INT32_MAX) raise(PyExc_ValueError, "kcache has %lld layers", (long long)layers);
      if (layers > 1 && vc.stride(0) != layer_stride)
        raise(PyExc_ValueError, "kcache and vcache must have one layer stride");
    }
    const Tensor& S = gpu(a[2], "src", dev);
    const int64_t pairs = S.dim() == 1 ? S.size(0) : -1;
    if (pairs > INT32_MAX) raise(PyExc_ValueError, "too many pairs");
    auto* src = static_cast<int32_t*>(vector(a[2], "src", ScalarType::Int, pairs, dev));
    auto* dst = static_cast<int32_t*>(vector(a[3], "dst", ScalarType::Int, pairs, dev));
    int64_t rows = 0, cols = 0, stride = 0;
    int32_t* table = a[4] == Py_None ? nullptr : table_of(a[4], "table", dev, &rows, &cols, &stride);
    OnDevice on(dev);
    const ttq_status s = (*copy)(&c, (int32_t)layers, layer_stride, src, dst, (int32_t)pairs, table, (int32_t)rows,
                                 (int32_t)cols, stride, stream_of(dev));
    if (s != TTQ_OK) return PyLong_FromLong(s);
    Py_RETURN_NONE;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
// kcache, vcache, src, dst, table
PyObject* cache_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return copy_pages(a, n, "cache_copy_pages", cache_of, &p_copy);
}
PyObject* packed_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // the rows' type does not matter to a copy
  auto of = [](const Tensor& k, const Tensor& v, int skip) { return packed_of(k, v, skip, ScalarType::Half); };
  return copy_pages(a, n, "packed_copy_pages", of, &p_packed_copy);
}

template <typename Of, typename Append>
PyObject* append(PyObject* const* a, Py_ssize_t n, const char* name, Of of, Append* call) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 12, name);
    const Tensor &kc = gpu(a[3], "kcache"), &vc = gpu(a[4], "vcache", kc.get_device());
    const int dev = kc.get_device();
    const Tensor &K = gpu(a[1], "K", dev), &V = gpu(a[2], "V", dev);
    const ScalarType type = K.scalar_type();
    const auto c = of(kc, vc, type);
    const int64_t rows = K.dim() > 0 ? K.size(0) : 0, cols = (int64_t)c.n_kv_heads * c.head_dim;
    int64_t ldk, ldv, ldq = 0, ldo = 0, heads = 0;
    void* k = rows_of(K, "K", rows, cols, type, &ldk);
    void* v = rows_of(V, "V", rows, cols, type, &ldv);
    const ttq_paged_batch b = batch_of(a[5], a[6], a[7], rows, 0, 0, dev);
    ttq_rotation r{};
    if (a[8] != Py_None) {
      const Tensor& T = gpu(a[8], "rotation", dev);
      want(T, "rotation", ScalarType::Float);
      if (T.dim() != 2 || !T.is_contiguous() || T.size(1) > INT32_MAX)
        raise(PyExc_ValueError, "rotation must be a dense [positions][channels]");
      r.table = static_cast<float*>(T.data_ptr());
      r.n_positions = T.size(0);
      r.dim = (int32_t)T.size(1);
    }
    if (a[9] != Py_None) r.positions = static_cast<int32_t*>(vector(a[9], "positions", ScalarType::Int, rows, dev));
    const int interleaved = PyObject_IsTrue(a[10]);
    if (interleaved < 0) return nullptr;
    r.interleaved = interleaved;
    Tensor made;
    const Tensor* out = &made;
    void *q = nullptr, *o = nullptr;
    if (a[0] != Py_None) {
      const Tensor& Q = gpu(a[0], "Q", dev);
      heads = Q.dim() == 2 && c.head_dim > 0 ? Q.size(1) / c.head_dim : 0;
      if (heads < 1 || heads > INT32_MAX) raise(PyExc_ValueError, "Q must be [tokens][heads * head dim]");
      q = rows_of(Q, "Q", rows, heads * c.head_dim, type, &ldq);
      if (a[11] == Py_None) made = make({rows, heads * c.head_dim}, type, dev);
      else out = &gpu(a[11], "out", dev);
      o = rows_of(*out, "out", rows, heads * c.head_dim, type, &ldo);
    } else if (a[11] != Py_None) {
      raise(PyExc_ValueError, "out without Q");
    }
    OnDevice on(dev);
    const ttq_status s = (*call)(&c, &b, a[8] != Py_None ? &r : nullptr, (int32_t)heads, q, ldq, o, ldo, k, ldk, v, ldv,
                                 stream_of(dev));
    if (s != TTQ_OK) return PyLong_FromLong(s);
    if (a[0] == Py_None) Py_RETURN_NONE;
    if (a[11] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[11]);
    return a[11];
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
// Q, K, V, kcache, vcache, block_table, q_start, kv_len, rotation, positions, interleaved, out
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  auto of = [](const Tensor& k, const Tensor& v, ScalarType type) {
    want(k, "kcache", type);
    return cache_of(k, v, 0);
  };
  return append(a, n, "cache_append", of, &p_append);
}
PyObject* packed_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  auto of = [](const Tensor& k, const Tensor& v, ScalarType type) { return packed_of(k, v, 0, type); };
  return append(a, n, "packed_append", of, &p_packed_append);
}

// kcache, vcache, block_table, q_start, kv_len, tokens, dtype
PyObject* packed_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 7, "packed_read");
    const Tensor &kc = gpu(a[0], "kcache"), &vc = gpu(a[1], "vcache", kc.get_device());
    const int dev = kc.get_device(), rows = whole(a[5], "tokens");
    if (rows < 0) raise(PyExc_ValueError, "tokens=%d is negative", rows);
    if (!THPDtype_Check(a[6])) raise(PyExc_TypeError, "dtype must be a torch dtype");
    const ScalarType type = reinterpret_cast<THPDtype*>(a[6])->scalar_type;
    const ttq_packed_cache c = packed_of(kc, vc, 0, type);
    const int64_t cols = (int64_t)c.n_kv_heads * c.head_dim;
    const ttq_paged_batch b = batch_of(a[2], a[3], a[4], rows, 0, 0, dev);
    Tensor k = make({rows, cols}, type, dev), v = make({rows, cols}, type, dev);
    OnDevice on(dev);
    const ttq_status s = p_packed_read(&c, &b, k.data_ptr(), cols, v.data_ptr(), cols, stream_of(dev));
    if (s != TTQ_OK) return PyLong_FromLong(s);
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(k)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(v)));
    return r;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// Q, kcache, vcache, block_table, q_start, kv_len, max_q_len, max_kv_len, scale, softcap, window, slopes, prefix_len,
// out, lse, workspace
template <typename Of, typename Workspace, typename Call>
PyObject* attention(PyObject* const* a, Py_ssize_t n, const char* name, Of of, Workspace* need, Call* call) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 16, name);
    const Tensor &kc = gpu(a[1], "kcache"), &vc = gpu(a[2], "vcache", kc.get_device());
    const int dev = kc.get_device();
    const Tensor& Q = gpu(a[0], "Q", dev);
    const auto c = of(kc, vc, Q.scalar_type());
    const ScalarType type = c.dtype == TTQ_F16 ? ScalarType::Half : ScalarType::BFloat16;
    const int64_t total = Q.dim() == 2 ? Q.size(0) : 0, cols = Q.dim() == 2 ? Q.size(1) : 0;
    const int64_t heads = c.head_dim > 0 ? cols / c.head_dim : 0;
    if (heads > INT32_MAX) raise(PyExc_ValueError, "Q has too many columns");
    int64_t ldq, ldo;
    void* q = rows_of(Q, "Q", total, heads * c.head_dim, type, &ldq);
    const ttq_paged_batch b = batch_of(a[3], a[4], a[5], total, whole(a[6], "max_q_len"), whole(a[7], "max_kv_len"), dev);
    ttq_attention t{};
    t.n_heads = (int32_t)heads;
    t.scale = a[8] == Py_None ? 1.0f / std::sqrt((float)c.head_dim) : (float)number(a[8], "scale");
    t.softcap = (float)number(a[9], "softcap");
    t.window = whole(a[10], "window");
    if (a[11] != Py_None) t.slopes = static_cast<float*>(vector(a[11], "slopes", ScalarType::Float, heads, dev));
    if (a[12] != Py_None) t.prefix_len = static_cast<int32_t*>(vector(a[12], "prefix_len", ScalarType::Int, b.n_seqs, dev));
    float* lse = nullptr;
    if (a[14] != Py_None) {
      const Tensor& L = gpu(a[14], "lse", dev);
      want(L, "lse", ScalarType::Float);
      if (L.dim() != 2 || L.size(0) != total || L.size(1) != heads || !L.is_contiguous())
        raise(PyExc_ValueError, "lse must be a dense [%lld][%lld]", (long long)total, (long long)heads);
      lse = static_cast<float*>(L.data_ptr());
    }
    Tensor own, made;
    const Tensor* out = &made;
    if (a[13] == Py_None) made = make({total, heads * c.head_dim}, type, dev);
    else out = &gpu(a[13], "out", dev);
    void* o = rows_of(*out, "out", total, heads * c.head_dim, type, &ldo);
    size_t bytes = 0;
    void* ws = workspace(a[15], (*need)(&c, &b, &t), dev, &own, &bytes);
    OnDevice on(dev);
    const ttq_status s = (*call)(&c, &b, &t, q, ldq, o, ldo, lse, ws, bytes, stream_of(dev));
    if (s != TTQ_OK) return PyLong_FromLong(s);
    if (a[13] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[13]);
    return a[13];
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  auto of = [](const Tensor& k, const Tensor& v, ScalarType) { return cache_of(k, v, 0); };
  return attention(a, n, "paged_attention", of, &p_attention_ws, &p_attention);
}
PyObject* packed_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  auto of = [](const Tensor& k, const Tensor& v, ScalarType type) { return packed_of(k, v, 0, type); };
  return attention(a, n, "packed_attention", of, &p_packed_attention_ws, &p_packed_attention);
}

ttq_dtype logits_of(const Tensor& x) {
  if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
    raise(PyExc_ValueError, "logits must be [T][V] with unit column stride");
  switch (x.scalar_type()) {
    case ScalarType::Float: return TTQ_F32;
    case ScalarType::Half: return TTQ_F16;
    case ScalarType::BFloat16: return TTQ_BF16;
    default: raise(PyExc_TypeError, "logits must be Float, Half or BFloat16 (got %s)", name_of(x.scalar_type()));
  }
}

// logits, scores, keep, history, workspace
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 5, "beam_select");
    const Tensor& x = gpu(a[0], "logits");
    const int dev = x.get_device(), keep = whole(a[2], "keep");
    const ttq_dtype dt = logits_of(x);
    const Tensor& S = gpu(a[1], "scores", dev);
    want(S, "scores", ScalarType::Float);
    if (S.dim() != 2 || !S.is_contiguous() || S.size(1) < 1 || S.size(1) > INT32_MAX || S.size(0) * S.size(1) != x.size(0))
      raise(PyExc_ValueError, "scores must be a dense [requests][beams], a value for each of the %lld rows", (long long)x.size(0));
    const int64_t requests = S.size(0), beams = S.size(1), V = x.size(1);
    if (keep < 1 || keep > 64) raise(PyExc_ValueError, "keep=%d, expected 1 to 64", keep);
    const int64_t* history = nullptr;
    int64_t ldh = 0, length = 0;
    if (a[3] != Py_None) {
      const Tensor& H = gpu(a[3], "history", dev);
      want(H, "history", ScalarType::Long);
      if (H.dim() != 2 || H.size(0) != x.size(0) || (H.size(1) > 1 && H.stride(1) != 1))
        raise(PyExc_ValueError, "history must be [%lld][tokens] with unit column stride", (long long)x.size(0));
      history = static_cast<int64_t*>(H.data_ptr());
      length = H.size(1);
      ldh = x.size(0) > 1 ? H.stride(0) : length;
    }
    Tensor os = make({requests, keep}, ScalarType::Float, dev), op = make({requests, keep}, ScalarType::Long, dev);
    Tensor ot = make({requests, keep}, ScalarType::Long, dev), oh, own;
    if (a[3] != Py_None) oh = make({requests * keep, length + 1}, ScalarType::Long, dev);
    size_t bytes = 0;
    void* ws = workspace(a[4], p_beams_ws(requests, (int32_t)beams, V, keep), dev, &own, &bytes);
    OnDevice on(dev);
    const ttq_status s = p_beams(x.data_ptr(), dt, requests, (int32_t)beams, V, x.size(0) > 1 ? x.stride(0) : V,
                                 static_cast<float*>(S.data_ptr()), keep, static_cast<float*>(os.data_ptr()),
                                 static_cast<int64_t*>(op.data_ptr()), static_cast<int64_t*>(ot.data_ptr()), history, ldh, length,
                                 a[3] != Py_None ? static_cast<int64_t*>(oh.data_ptr()) : nullptr, length + 1, ws, bytes,
                                 stream_of(dev));
    if (s != TTQ_OK) return PyLong_FromLong(s);
    PyObject* r = PyTuple_New(a[3] != Py_None ? 4 : 3);
    if (r == nullptr) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(os)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(op)));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(ot)));
    if (a[3] != Py_None) PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(std::move(oh)));
    return r;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// logits, tokens, top, workspace
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 4, "token_logprobs");
    const Tensor& x = gpu(a[0], "logits");
    const int dev = x.get_device();
    const ttq_dtype dt = logits_of(x);
    const int64_t T = x.size(0), V = x.size(1);
    auto* tokens = static_cast<int64_t*>(vector(a[1], "tokens", ScalarType::Long, T, dev));
    const int top = whole(a[2], "top");
    Tensor lp = make({T}, ScalarType::Float, dev), en = make({T}, ScalarType::Float, dev), ids, tl, own;
    if (top > 0) {
      ids = make({T, top}, ScalarType::Long, dev);
      tl = make({T, top}, ScalarType::Float, dev);
    }
    size_t bytes = 0;
    void* ws = workspace(a[3], p_logprobs_ws(T, V, top), dev, &own, &bytes);
    OnDevice on(dev);
    const ttq_status s = p_logprobs(x.data_ptr(), dt, T, V, T > 1 ? x.stride(0) : V, tokens,
                                    static_cast<float*>(lp.data_ptr()), static_cast<float*>(en.data_ptr()), top,
                                    top > 0 ? static_cast<int64_t*>(ids.data_ptr()) : nullptr,
                                    top > 0 ? static_cast<float*>(tl.data_ptr()) : nullptr, ws, bytes, stream_of(dev));
    if (s != TTQ_OK) return PyLong_FromLong(s);
    PyObject* r = PyTuple_New(top > 0 ? 4 : 2);
    if (r == nullptr) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(lp)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(en)));
    if (top > 0) {
      PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(ids)));
      PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(std::move(tl)));
    }
    return r;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define TTQ_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TTQ_METHOD(bind), TTQ_METHOD(cache_write), TTQ_METHOD(cache_copy_pages),
                         TTQ_METHOD(paged_attention), TTQ_METHOD(token_logprobs), TTQ_METHOD(cache_append),
                         TTQ_METHOD(packed_append), TTQ_METHOD(packed_read), TTQ_METHOD(packed_copy_pages),
                         TTQ_METHOD(packed_attention), TTQ_METHOD(beam_select),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
