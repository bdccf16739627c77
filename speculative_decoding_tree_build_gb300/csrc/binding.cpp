// Python entry points of the plain-decoding and 8-bit-cache calls, and of those
// around a serving step (pages, slots, filtered sampling).
//
// A decode step makes the first ones once a layer, and at one token a request
// the GPU needs 2 to 5 us for each: checking a dozen tensors attribute by
// attribute from Python and converting twenty arguments took 17 us a call.
// Here the same checks read the tensors directly. Each function returns the
// C entry point's code; a wrong tensor raises ValueError before any launch.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/treeverify.h"

namespace {

using at::ScalarType;
using at::Tensor;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

// The arguments of one call: what they share is that they lie on one device.
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : args_(args) {
    if (n != want) refuse("wrong number of arguments");
  }

  bool none(int i) const { return args_[i] == Py_None; }

  const Tensor& tensor(int i, const char* name) {
    if (!THPVariable_Check(args_[i])) refuse(std::string(name) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(args_[i]);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    const int device = t.device().index();
    if (device_ < 0) device_ = device;
    if (device != device_) refuse(std::string(name) + " is on another device than the tensors before it");
    return t;
  }

  const Tensor& typed(int i, ScalarType type, const char* name) {
    const Tensor& t = tensor(i, name);
    if (t.scalar_type() != type) refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    return t;
  }

  // a contiguous tensor of at least `least` elements
  void* flat(int i, ScalarType type, const char* name, int64_t least = 0) {
    const Tensor& t = typed(i, type, name);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    if (t.numel() < least) refuse(std::string(name) + " must hold at least " + std::to_string(least) + " elements");
    return t.data_ptr();
  }

  const int32_t* ints(int i, const char* name, int64_t least) {
    return static_cast<const int32_t*>(flat(i, ScalarType::Int, name, least));
  }

  int device() const { return device_; }

 private:
  PyObject* const* args_;
  int device_ = -1;
};

// A ctypes structure's memory.
template <typename T>
T structure(PyObject* o, const char* name) {
  Py_buffer view;
  if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    refuse(std::string(name) + " must be the structure that the call names");
  }
  const bool fits = view.len == static_cast<Py_ssize_t>(sizeof(T));
  T out{};
  if (fits) memcpy(&out, view.buf, sizeof(T));
  PyBuffer_Release(&view);
  if (!fits) refuse(std::string(name) + " must be the structure that the call names");
  return out;
}

// None: the current stream of the tensors' device; an int or an object with cuda_stream
void* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
  PyObject* n = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (n == nullptr) {
    PyErr_Clear();
    refuse("stream must be None, an int or a CUDA stream");
  }
  void* s = PyLong_AsVoidPtr(n);
  Py_DECREF(n);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse("stream must be None, an int or a CUDA stream");
  }
  return s;
}

struct Rows {
  void* ptr;
  int64_t rows, ld;
  ScalarType type;
};

// [rows][heads][d] with contiguous rows; the row stride may exceed heads * d
Rows heads_of(Call& c, int i, int64_t heads, int64_t d, const char* name) {
  const Tensor& t = c.tensor(i, name);
  const auto s = t.sizes();
  if (s.size() != 3 || s[1] != heads || s[2] != d ||
      (t.numel() != 0 && ((d > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != d) ||
                          (s[0] > 1 && t.stride(0) < heads * d))))
    refuse(std::string(name) + " must be a CUDA tensor [rows][" + std::to_string(heads) + "][" + std::to_string(d) +
           "] with contiguous rows");
  // the stride of a single row is free: any legal value does
  return {t.data_ptr(), s[0], s[0] > 1 ? t.stride(0) : heads * d, t.scalar_type()};
}

struct Pools {
  int32_t format, blocks;
  void *k, *v;
  float *ks, *vs;
};

int32_t format_of(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return TV_KV_BF16;
    case ScalarType::Float8_e4m3fn: return TV_KV_E4M3;
    case ScalarType::Char: return TV_KV_INT8;
    default: refuse(std::string("a KV pool must be BFloat16, Float8_e4m3fn or Char, got ") + c10::toString(t));
  }
}

// Two pools [num_blocks][Hkv][16][D] and their scales [num_blocks][Hkv][16]
Pools pools_of(Call& c, const tv_geom& g, int i, int scales) {
  Pools p{};
  const Tensor& k = c.tensor(i, "k_cache");
  p.format = format_of(k.scalar_type());
  const Tensor& v = c.typed(i + 1, k.scalar_type(), "v_cache");
  for (const Tensor* t : {&k, &v}) {
    const auto s = t->sizes();
    if (s.size() != 4 || s[0] != k.size(0) || s[1] != g.num_kv_heads || s[2] != TV_BLOCK_SIZE || s[3] != g.head_dim || !t->is_contiguous())
      refuse("a KV pool must be contiguous [num_blocks][" + std::to_string(g.num_kv_heads) + "][16][" + std::to_string(g.head_dim) + "]");
  }
  if (k.size(0) > INT32_MAX) refuse("a KV pool has at most 2^31 - 1 blocks");
  p.blocks = static_cast<int32_t>(k.size(0));
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  if (scales >= 0 && p.format != TV_KV_BF16) {
    float** out[2] = {&p.ks, &p.vs};
    for (int j = 0; j < 2; ++j) {
      const char* name = j ? "v_scale" : "k_scale";
      if (c.none(scales + j)) refuse(std::string(name) + " is needed for an 8-bit pool");
      const Tensor& t = c.typed(scales + j, ScalarType::Float, name);
      const auto s = t.sizes();
      if (s.size() != 3 || s[0] != k.size(0) || s[1] != g.num_kv_heads || s[2] != TV_BLOCK_SIZE || !t.is_contiguous())
        refuse(std::string(name) + " must be contiguous float32 [num_blocks][" + std::to_string(g.num_kv_heads) + "][16]");
      *out[j] = t.data_ptr<float>();
    }
  }
  return p;
}

struct Table {
  const int32_t* ptr;
  int32_t width;
};

Table table_of(Call& c, int i, int64_t batch, const char* name) {
  const Tensor& t = c.typed(i, ScalarType::Int, name);
  if (t.dim() != 2 || t.size(0) != batch || t.size(1) < 1 || t.size(1) > INT32_MAX || !t.is_contiguous())
    refuse(std::string(name) + " must be contiguous int32 [batch][max_blocks_per_req]");
  return {t.data_ptr<int32_t>(), static_cast<int32_t>(t.size(1))};
}

int32_t count(int64_t n, const char* name) {
  if (n < 0 || n > INT32_MAX) refuse(std::string(name) + " is out of range");
  return static_cast<int32_t>(n);
}

// The interpreter's lock, let go for a scope (an exception takes it back too).
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// Run the call with the tensors' device current and without the interpreter's
// lock. What can be refused is refused before: the call itself only returns codes.
template <typename F>
PyObject* launch(const Call& c, PyObject* stream, F f) {
  void* s = stream_of(stream, c.device());
  int rc;
  {
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device()));
    const Unlocked unlocked;
    rc = f(s);
  }
  return PyLong_FromLong(rc);
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// rope_axes(geom, q, k, positions, inv_freq, q_out, k_out, stream)
PyObject* rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 8);
    const auto g = structure<tv_rope_axes_geom>(a[0], "geom");
    const Rows q = heads_of(c, 1, g.num_q_heads, g.head_dim, "q");
    if (q.type != ScalarType::BFloat16 && q.type != ScalarType::Float) refuse("q must be bfloat16 or float32");
    const Rows qo = heads_of(c, 5, g.num_q_heads, g.head_dim, "q_out");
    Rows k{}, ko{};
    const bool keys = g.num_kv_heads > 0;
    if (keys) {
      k = heads_of(c, 2, g.num_kv_heads, g.head_dim, "k");
      ko = heads_of(c, 6, g.num_kv_heads, g.head_dim, "k_out");
      if (k.rows != q.rows || ko.rows != q.rows) refuse("k and k_out must have as many rows as q");
      if (k.type != q.type || ko.type != q.type) refuse("k and k_out must have q's type");
    }
    if (qo.rows != q.rows || qo.type != q.type) refuse("q_out must have q's rows and type");
    const Tensor& pos = c.typed(3, ScalarType::Int, "positions");
    if (pos.dim() != 2 || pos.size(0) != g.num_axes || pos.size(1) != q.rows || (q.rows > 1 && pos.stride(1) != 1))
      refuse("positions must be an int32 CUDA matrix [axes][rows] with contiguous rows");
    int64_t pairs = 0;
    for (int i = 0; i < g.num_axes && i < TV_MAX_ROPE_AXES; ++i) pairs += g.section[i];
    const Tensor& inv = c.typed(4, ScalarType::Float, "inv_freq");
    if (inv.numel() != pairs || !inv.is_contiguous()) refuse("inv_freq must hold one frequency per rotated pair");
    const int32_t rows = count(q.rows, "rows");
    return launch(c, a[7], [&](void* s) {
      return tv_rope_axes(&g, rows, q.type == ScalarType::Float ? TV_DTYPE_F32 : TV_DTYPE_BF16, q.ptr, q.ld,
                          k.ptr, k.ld, pos.data_ptr<int32_t>(), g.num_axes > 1 ? pos.stride(0) : q.rows,
                          inv.data_ptr<float>(), qo.ptr, qo.ld, ko.ptr, ko.ld, s);
    });
  });
}

// kv_quant_append(geom, k_new, v_new, cu_rows, start_len, block_table, n_blocks, k_cache, v_cache, k_scale, v_scale,
//                 status, stream)
PyObject* kv_quant_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 13);
    const auto g = structure<tv_geom>(a[0], "geom");
    const Rows k = heads_of(c, 1, g.num_kv_heads, g.head_dim, "k_new"), v = heads_of(c, 2, g.num_kv_heads, g.head_dim, "v_new");
    if (k.type != ScalarType::BFloat16 || v.type != ScalarType::BFloat16) refuse("k_new and v_new must be bfloat16");
    if (k.rows != v.rows || k.ld != v.ld) refuse("k_new and v_new must have the same rows and row stride");
    const int32_t* cu = c.ints(3, "cu_rows", 1);
    const int64_t batch = c.tensor(3, "cu_rows").numel() - 1;
    const int32_t* start = c.ints(4, "start_len", batch);
    const Table t = table_of(c, 5, batch, "block_table");
    const int32_t* held = c.ints(6, "n_blocks", batch);
    const Pools p = pools_of(c, g, 7, 9);
    int32_t* status = const_cast<int32_t*>(c.ints(11, "status", batch));
    const int32_t requests = count(batch, "batch"), rows = count(k.rows, "rows");
    return launch(c, a[12], [&](void* s) {
      return tv_kv_quant_append(&g, p.format, requests, rows, k.ptr, v.ptr, k.ld, cu, start, t.ptr, held,
                                t.width, p.k, p.v, p.ks, p.vs, p.blocks, status, s);
    });
  });
}

// kv_quant_read(geom, first, last, block_table, n_blocks, k_cache, v_cache, k_scale, v_scale, out_block_table,
//               out_n_blocks, k_out, v_out, status, stream)
PyObject* kv_quant_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 15);
    const auto g = structure<tv_geom>(a[0], "geom");
    const int32_t* last = c.ints(2, "last", 0);
    const int64_t batch = c.tensor(2, "last").numel();
    const int32_t* first = c.none(1) ? nullptr : c.ints(1, "first", batch);
    const Table t = table_of(c, 3, batch, "block_table");
    const int32_t* held = c.ints(4, "n_blocks", batch);
    const Pools p = pools_of(c, g, 5, 7);
    const Table to = table_of(c, 9, batch, "out_block_table");
    const int32_t* to_held = c.ints(10, "out_n_blocks", batch);
    const Pools out = pools_of(c, g, 11, -1);
    if (out.format != TV_KV_BF16) refuse("k_out and v_out must be bfloat16 pools");
    int32_t* status = const_cast<int32_t*>(c.ints(13, "status", batch));
    const int32_t requests = count(batch, "batch");
    return launch(c, a[14], [&](void* s) {
      return tv_kv_quant_read(&g, p.format, requests, first, last, t.ptr, held, t.width, p.k, p.v, p.ks, p.vs,
                              p.blocks, to.ptr, to_held, to.width, out.k, out.v, out.blocks, status, s);
    });
  });
}

// decode_attention(geom, q, seq_len, block_table, n_blocks, k_cache, v_cache, k_scale, v_scale, out, lse, workspace,
//                  status, stream)
PyObject* decode_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 14);
    const auto g = structure<tv_geom>(a[0], "geom");
    const Rows q = heads_of(c, 1, g.num_q_heads, g.head_dim, "q");
    if (q.type != ScalarType::BFloat16) refuse("q must be bfloat16");
    const int32_t* len = c.ints(2, "seq_len", 0);
    const int64_t batch = c.tensor(2, "seq_len").numel();
    if (q.rows != batch) refuse("q must have one row per request");
    const Table t = table_of(c, 3, batch, "block_table");
    const int32_t* held = c.ints(4, "n_blocks", batch);
    const Pools p = pools_of(c, g, 5, 7);
    const int64_t heads = batch * g.num_q_heads;
    void* out = c.flat(9, ScalarType::BFloat16, "out", heads * g.head_dim);
    float* lse = c.none(10) ? nullptr : static_cast<float*>(c.flat(10, ScalarType::Float, "lse", heads));
    const Tensor& ws = c.tensor(11, "workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
    int32_t* status = const_cast<int32_t*>(c.ints(12, "status", batch));
    const int32_t requests = count(batch, "batch");
    return launch(c, a[13], [&](void* s) {
      return tv_decode_attention(&g, p.format, requests, q.ptr, q.ld, len, t.ptr, held, t.width, p.k, p.v, p.ks,
                                 p.vs, p.blocks, out, lse, ws.data_ptr(), ws.nbytes(), status, s);
    });
  });
}

// [batch] of one type, None allowed where `optional`
template <typename T>
T* per_request(Call& c, int i, ScalarType type, const char* name, int64_t batch, bool optional = false) {
  if (optional && c.none(i)) return nullptr;
  return static_cast<T*>(c.flat(i, type, name, batch));
}

int32_t number(PyObject* o, const char* name) {
  const long long n = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an int");
  }
  return count(n, name);
}

// block_tables(want_len, block_table, n_blocks, free_blocks, free_count, released, released_count, status, stream)
PyObject* block_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 9);
    const int32_t* want = c.ints(0, "want_len", 0);
    const int64_t batch = c.tensor(0, "want_len").numel();
    const Table t = table_of(c, 1, batch, "block_table");
    auto* held = per_request<int32_t>(c, 2, ScalarType::Int, "n_blocks", batch);
    auto* list = static_cast<int32_t*>(c.flat(3, ScalarType::Int, "free_blocks"));
    const int32_t pool = count(c.tensor(3, "free_blocks").numel(), "free_blocks");
    auto* top = static_cast<int32_t*>(c.flat(4, ScalarType::Int, "free_count", 1));
    if (c.none(5) != c.none(6)) refuse("released and released_count come together");
    const int32_t* released = nullptr;
    if (!c.none(5)) {
      const Table r = table_of(c, 5, batch, "released");
      if (r.width != t.width) refuse("released must be as wide as block_table");
      released = r.ptr;
    }
    auto* released_count = per_request<int32_t>(c, 6, ScalarType::Int, "released_count", batch, true);
    auto* status = per_request<int32_t>(c, 7, ScalarType::Int, "status", batch);
    const int32_t requests = count(batch, "batch");
    return launch(c, a[8], [&](void* s) {
      return tv_block_tables(requests, want, const_cast<int32_t*>(t.ptr), held, t.width, pool, list, top, released,
                             released_count, status, s);
    });
  });
}

// slot_map(cu_rows, start_len, block_table, n_blocks, num_blocks, slots, status, stream)
PyObject* slot_map(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 8);
    const int32_t* cu = c.ints(0, "cu_rows", 1);
    const int64_t batch = c.tensor(0, "cu_rows").numel() - 1;
    const int32_t* start = c.ints(1, "start_len", batch);
    const Table t = table_of(c, 2, batch, "block_table");
    const int32_t* held = c.ints(3, "n_blocks", batch);
    const int32_t blocks = number(a[4], "num_blocks");
    auto* slots = static_cast<int64_t*>(c.flat(5, ScalarType::Long, "slots"));
    const int32_t rows = count(c.tensor(5, "slots").numel(), "rows"), requests = count(batch, "batch");
    auto* status = per_request<int32_t>(c, 6, ScalarType::Int, "status", batch);
    return launch(c, a[7], [&](void* s) {
      return tv_slot_map(requests, rows, cu, start, t.ptr, held, t.width, blocks, slots, status, s);
    });
  });
}

// kv_rows_write(geom, k_new, v_new, slots, k_cache, v_cache, stream)
// kv_rows_read(geom, slots, k_cache, v_cache, k_out, v_out, stream)
template <bool kWrite>
PyObject* kv_rows(PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 7);
    const auto g = structure<tv_geom>(a[0], "geom");
    const int at = kWrite ? 1 : 4, slot_at = kWrite ? 3 : 1, pool_at = kWrite ? 4 : 2;
    const Rows k = heads_of(c, at, g.num_kv_heads, g.head_dim, kWrite ? "k_new" : "k_out");
    const Rows v = heads_of(c, at + 1, g.num_kv_heads, g.head_dim, kWrite ? "v_new" : "v_out");
    if (k.type != ScalarType::BFloat16 || v.type != ScalarType::BFloat16) refuse("K and V rows must be bfloat16");
    if (k.rows != v.rows) refuse("K and V must have the same rows");
    const auto* slots = static_cast<const int64_t*>(c.flat(slot_at, ScalarType::Long, "slots"));
    if (c.tensor(slot_at, "slots").numel() != k.rows) refuse("slots must hold one slot per row");
    const Pools p = pools_of(c, g, pool_at, -1);
    if (p.format != TV_KV_BF16) refuse("k_cache and v_cache must be bfloat16 pools");
    const int32_t rows = count(k.rows, "rows");
    return launch(c, a[6], [&](void* s) {
      return kWrite ? tv_kv_rows_write(&g, rows, k.ptr, k.ld, v.ptr, v.ld, slots, p.k, p.v, p.blocks, s)
                    : tv_kv_rows_read(&g, rows, slots, p.k, p.v, p.blocks, k.ptr, k.ld, v.ptr, v.ld, s);
    });
  });
}
PyObject* kv_rows_write(PyObject*, PyObject* const* a, Py_ssize_t n) { return kv_rows<true>(a, n); }
PyObject* kv_rows_read(PyObject*, PyObject* const* a, Py_ssize_t n) { return kv_rows<false>(a, n); }

struct Matrix {
  void* ptr;
  int64_t rows, cols, ld;
  ScalarType type;
};

// [rows][cols] with contiguous rows; the stride of a single row is free: the next legal one
Matrix matrix_of(Call& c, int i, const char* name, int64_t step) {
  const Tensor& t = c.tensor(i, name);
  if (t.dim() != 2 || (t.numel() != 0 && ((t.size(1) > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) < t.size(1)))))
    refuse(std::string(name) + " must be a CUDA matrix with contiguous rows");
  return {t.data_ptr(), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : (t.size(1) + step - 1) / step * step, t.scalar_type()};
}

struct Filter {
  Matrix logits;
  int32_t dtype, batch, max_nodes, vocab;
  const int32_t* cu;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
};

// logits at 0; from `at` on cu_nodes, temperature, top_k, top_p, min_p, max_nodes
Filter filter_of(Call& c, PyObject* const* a, int at) {
  Filter f{};
  f.logits = matrix_of(c, 0, "logits", 8);
  if (f.logits.type != ScalarType::BFloat16 && f.logits.type != ScalarType::Float) refuse("logits must be bfloat16 or float32");
  f.dtype = f.logits.type == ScalarType::Float ? TV_DTYPE_F32 : TV_DTYPE_BF16;
  f.cu = c.ints(at, "cu_nodes", 1);
  const int64_t batch = c.tensor(at, "cu_nodes").numel() - 1;
  f.temperature = per_request<float>(c, at + 1, ScalarType::Float, "temperature", batch);
  f.top_k = per_request<int32_t>(c, at + 2, ScalarType::Int, "top_k", batch, true);
  f.top_p = per_request<float>(c, at + 3, ScalarType::Float, "top_p", batch, true);
  f.min_p = per_request<float>(c, at + 4, ScalarType::Float, "min_p", batch, true);
  f.max_nodes = number(a[at + 5], "max_nodes");
  f.batch = count(batch, "batch");
  f.vocab = count(f.logits.cols, "vocab");
  return f;
}

// sample_filtered(logits, gumbel, cu_nodes, temperature, top_k, top_p, min_p, max_nodes, tokens, logp, status, stream)
PyObject* sample_filtered(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 12);
    const Filter f = filter_of(c, a, 2);
    Matrix g{};
    if (!c.none(1)) {
      g = matrix_of(c, 1, "gumbel", 4);
      if (g.type != ScalarType::Float) refuse("gumbel must be float32");
      if (g.rows < f.logits.rows || g.cols < f.logits.cols) refuse("gumbel must have the logits' rows and columns");
    }
    auto* tokens = static_cast<int32_t*>(c.flat(8, ScalarType::Int, "tokens", f.logits.rows));
    auto* logp = c.none(9) ? nullptr : static_cast<float*>(c.flat(9, ScalarType::Float, "logp", f.logits.rows));
    auto* status = per_request<int32_t>(c, 10, ScalarType::Int, "status", f.batch);
    return launch(c, a[11], [&](void* s) {
      return tv_sample_filtered(f.dtype, f.logits.ptr, f.logits.ld, static_cast<const float*>(g.ptr), g.ld, f.cu,
                                f.temperature, f.top_k, f.top_p, f.min_p, f.batch, f.max_nodes, f.vocab, tokens, logp,
                                status, s);
    });
  });
}

// filter_logits(logits, cu_nodes, temperature, top_k, top_p, min_p, max_nodes, out, kept, status, stream)
PyObject* filter_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(a, n, 11);
    const Filter f = filter_of(c, a, 1);
    const Matrix out = matrix_of(c, 7, "out", 8);
    if (out.type != f.logits.type || out.rows != f.logits.rows || out.cols != f.logits.cols)
      refuse("out must have the logits' type, rows and columns");
    auto* kept = c.none(8) ? nullptr : static_cast<int32_t*>(c.flat(8, ScalarType::Int, "kept", f.logits.rows));
    auto* status = per_request<int32_t>(c, 9, ScalarType::Int, "status", f.batch);
    return launch(c, a[10], [&](void* s) {
      return tv_filter_logits(f.dtype, f.logits.ptr, f.logits.ld, f.cu, f.temperature, f.top_k, f.top_p, f.min_p,
                              f.batch, f.max_nodes, f.vocab, out.ptr, out.ld, kept, status, s);
    });
  });
}

#define TV_FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {TV_FN(rope_axes), TV_FN(kv_quant_append), TV_FN(kv_quant_read), TV_FN(decode_attention),
                          TV_FN(block_tables), TV_FN(slot_map), TV_FN(kv_rows_write), TV_FN(kv_rows_read),
                          TV_FN(sample_filtered), TV_FN(filter_logits), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_treeverify_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__treeverify_torch() {
  PyObject* m = PyModule_Create(&kModule);
  // the loader compares it with the torch that is running
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TV_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
