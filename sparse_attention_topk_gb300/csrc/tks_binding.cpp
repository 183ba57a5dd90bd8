// The Python side of the cache, attention, block and page calls: checks of the
// tensors, the outputs' allocation and the call of the C entry point
// (include/tks_attention.h, include/tks_blocks.h), in one C++ step.  A decode step makes these calls for every layer, and the
// same work in Python took longer than the kernels of a short context (33 us
// of host time a call, 6 so, where the kernels take 9).
//
// The module calls the entry points of the libtks that the package has loaded
// (set_library), so there is no second copy of the library.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <optional>
#include <string>

#include "tks_attention.h"
#include "tks_blocks.h"

namespace {

using at::Tensor;

decltype(&tks_cache_write) f_write = nullptr;
decltype(&tks_cache_read) f_read = nullptr;
decltype(&tks_tree_attention) f_tree = nullptr;
decltype(&tks_selected_attention) f_selected = nullptr;
decltype(&tks_cache_bounds) f_bounds = nullptr;
decltype(&tks_block_scores) f_scores = nullptr;
decltype(&tks_block_attention) f_block = nullptr;
decltype(&tks_cache_fork) f_fork = nullptr;
decltype(&tks_cache_compact) f_compact = nullptr;
decltype(&tks_cache_copy) f_copy = nullptr;
PyObject* tks_error = nullptr;  // the package's TksError

struct Refused : std::exception {
  std::string what_;
  explicit Refused(std::string s) : what_(std::move(s)) {}
  const char* what() const noexcept override { return what_.c_str(); }
};
struct Raised : std::exception {};  // a Python error is set

void want(bool ok, const char* what) {
  if (!ok) throw Refused(what);
}

Tensor tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}
std::optional<Tensor> maybe(PyObject* o, const char* what) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, what);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A paged cache and its device.
struct Paged {
  tks_cache c;
  at::Device device;
};

Paged cache_of(const Tensor& k, const Tensor& v, const std::optional<Tensor>& scales) {
  want(k.dim() == 4 && k.is_cuda(), "caches must be CUDA tensors [pages, page_size, kv_heads, head_dim]");
  want(v.dim() == 4 && v.sizes() == k.sizes() && v.strides() == k.strides() && v.scalar_type() == k.scalar_type() && v.device() == k.device(),
       "k_cache and v_cache must have one shape, strides, dtype and device");
  const int64_t pages = k.size(0), page = k.size(1), heads = k.size(2), dim = k.size(3);
  want((dim == 64 || dim == 128) && k.stride(3) == 1, "head_dim must be 64 or 128, and contiguous");
  want(page >= 1 && (page & (page - 1)) == 0, "page_size must be a power of two");
  want(pages >= 1 && heads >= 1 && pages <= INT32_MAX && page <= INT32_MAX && heads <= INT32_MAX, "a cache has at least one page and one head");
  Paged r{tks_cache{}, k.device()};
  r.c.k = k.data_ptr();
  r.c.v = v.data_ptr();
  if (k.scalar_type() == at::kChar) {
    want(scales && scales->dim() == 4 && scales->size(0) == pages && scales->size(1) == page && scales->size(2) == heads && scales->size(3) == 2 &&
             scales->scalar_type() == at::kFloat && scales->is_contiguous() && scales->device() == k.device(),
         "an int8 cache needs scales: a contiguous float32 CUDA tensor [pages, page_size, kv_heads, 2]");
    r.c.held = TKS_I8;
    r.c.scales = static_cast<float*>(scales->data_ptr());
  } else {
    want(k.scalar_type() == at::kBFloat16, "a cache is bfloat16 or int8");
    want(!scales, "a bfloat16 cache has no scales");
    r.c.held = TKS_BF16;
  }
  r.c.pages = (int32_t)pages;
  r.c.page_size = (int32_t)page;
  r.c.kv_heads = (int32_t)heads;
  r.c.head_dim = (int32_t)dim;
  r.c.page_stride = k.stride(0);
  r.c.token_stride = k.stride(1);
  r.c.head_stride = k.stride(2);
  return r;
}

// An int32 tensor of this shape, contiguous, on the cache's device.
const int32_t* ints(const Tensor& t, at::IntArrayRef shape, const at::Device& device, const char* what) {
  if (t.scalar_type() != at::kInt || t.sizes() != shape || t.device() != device || !t.is_contiguous()) {
    std::string s = std::string(what) + " must be a contiguous int32 CUDA tensor [";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    throw Refused(s + "] on the cache's device");
  }
  return static_cast<const int32_t*>(t.data_ptr());
}

// t where the kernels can read it as it is (a contiguous last dimension, 16-byte pieces
// everywhere else; an extent of one is never stepped over), else a copy.
Tensor readable(const Tensor& t) {
  const int64_t unit = 16 / t.element_size();
  const int64_t last = t.dim() - 1;
  bool ok = t.stride(last) == 1 || t.size(last) <= 1;
  for (int64_t i = 0; i < last && ok; ++i) ok = t.size(i) <= 1 || (t.stride(i) >= 0 && t.stride(i) % unit == 0);
  Tensor r = ok ? t : t.contiguous();
  return aligned16(r.data_ptr()) ? r : r.clone(at::MemoryFormat::Contiguous);
}
int64_t step(const Tensor& t, int64_t i) { return t.size(i) > 1 ? t.stride(i) : 0; }

// An output (without the dispatcher's way, which takes half a microsecond more).
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Device& device) {
  return Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

// The device and stream of a call: what is allocated here belongs to the stream that writes it.
struct Place {
  c10::cuda::OptionalCUDAStreamGuard stream_guard;
  c10::cuda::OptionalCUDAGuard device_guard;
  void* stream;
  Place(PyObject* given, const at::Device& device) {
    if (given == Py_None) {
      device_guard.set_device(device);
      stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    } else {
      stream = PyLong_AsVoidPtr(given);
      if (PyErr_Occurred()) throw Raised();
      const cudaStream_t s = static_cast<cudaStream_t>(stream);
      stream_guard.reset_stream(s ? c10::cuda::getStreamFromExternal(s, device.index()) : c10::cuda::getDefaultCUDAStream(device.index()));
    }
  }
};

void check(int status, const char* what) {
  if (status == TKS_OK) return;
  PyObject* e = PyObject_CallFunction(tks_error, "is", status, what);
  if (e) {
    PyErr_SetObject(tks_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// Runs f, turning what it throws into Python errors.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "an unknown C++ error");
  }
  return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t wanted, bool set) {
  if (n == wanted && set) return true;
  PyErr_SetString(PyExc_TypeError, set ? "wrong number of arguments" : "the library is not set");
  return false;
}
bool arity(Py_ssize_t n, Py_ssize_t wanted) { return arity(n, wanted, f_write != nullptr); }
bool arity_blocks(Py_ssize_t n, Py_ssize_t wanted) { return arity(n, wanted, f_bounds != nullptr); }

int dtype_of(at::ScalarType t, const char* what) {
  want(t == at::kBFloat16 || t == at::kFloat, what);
  return t == at::kFloat ? TKS_F32 : TKS_BF16;
}

// write(k, v, k_cache, v_cache, slots, scales, stream)
PyObject* py_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor k = tensor(a[0], "k"), v = tensor(a[1], "v"), slots = tensor(a[4], "slots");
    Paged c = cache_of(tensor(a[2], "k_cache"), tensor(a[3], "v_cache"), maybe(a[5], "scales"));
    const int64_t count = slots.numel();
    const int32_t* at_slots = ints(slots, {count}, c.device, "slots");
    want(k.dim() == 3 && k.size(0) == count && k.size(1) == c.c.kv_heads && k.size(2) == c.c.head_dim && v.sizes() == k.sizes() &&
             v.scalar_type() == k.scalar_type() && k.device() == c.device && v.device() == c.device,
         "k and v must be CUDA tensors [slots, kv_heads, head_dim] of one dtype on the cache's device");
    const int dt = dtype_of(k.scalar_type(), "k and v must be bfloat16 or float32");
    want(count <= INT32_MAX, "too many tokens");
    if (count) {
      Place place(a[6], c.device);
      const Tensor x = readable(k), y = readable(v);
      check(f_write(&c.c, x.data_ptr(), y.data_ptr(), (int32_t)count, dt, step(x, 0), step(x, 1), step(y, 0), step(y, 1), at_slots, place.stream),
            "tks_cache_write");
    }
    Py_RETURN_NONE;
  });
}

// read(k_cache, v_cache, slots, scales, float32, k_out, v_out, stream) -> (k, v)
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor slots = tensor(a[2], "slots");
    Paged c = cache_of(tensor(a[0], "k_cache"), tensor(a[1], "v_cache"), maybe(a[3], "scales"));
    const int64_t count = slots.numel();
    const int32_t* at_slots = ints(slots, {count}, c.device, "slots");
    want(count <= INT32_MAX, "too many slots");
    const at::ScalarType type = a[4] == Py_True ? at::kFloat : at::kBFloat16;
    const int64_t shape[3] = {count, c.c.kv_heads, c.c.head_dim};
    Place place(a[7], c.device);
    Tensor out[2];
    for (int i = 0; i < 2; ++i) {
      if (a[5 + i] == Py_None) {
        out[i] = fresh(shape, type, c.device);
      } else {
        out[i] = tensor(a[5 + i], "out");
        want(out[i].sizes() == at::IntArrayRef(shape) && out[i].scalar_type() == type && out[i].device() == c.device && out[i].is_contiguous() &&
                 aligned16(out[i].data_ptr()),
             "out must be two contiguous, 16-byte aligned CUDA tensors [slots, kv_heads, head_dim] of the dtype asked for");
      }
    }
    if (count)
      check(f_read(&c.c, at_slots, (int32_t)count, out[0].data_ptr(), out[1].data_ptr(), type == at::kFloat ? TKS_F32 : TKS_BF16, place.stream),
            "tks_cache_read");
    return Py_BuildValue("NN", THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]));
  });
}

// The queries and the page table, as the C entry points take them; x: q as the kernels can read it.
tks_queries queries_of(const Tensor& x, const Tensor& table) {
  tks_queries r{};
  r.q = x.data_ptr();
  r.q_batch_stride = step(x, 0);
  r.q_token_stride = step(x, 1);
  r.q_head_stride = step(x, 2);
  r.batch = (int32_t)x.size(0);
  r.tokens = (int32_t)x.size(1);
  r.q_heads = (int32_t)x.size(2);
  r.page_table = static_cast<const int32_t*>(table.data_ptr());
  r.table_stride = step(table, 0);
  r.table_pages = (int32_t)table.size(1);
  return r;
}
void check_table(const Tensor& table, int64_t rows, const at::Device& device, const char* what) {
  want(table.dim() == 2 && (rows < 0 || table.size(0) == rows) && table.scalar_type() == at::kInt && table.device() == device && table.is_cuda() &&
           (table.size(1) <= 1 || table.stride(1) == 1),
       what);
}

// What the attention calls share: the queries, the page table, the outputs.
template <typename F>
PyObject* attend(const Paged& c, const Tensor& q, const Tensor& table, PyObject* scale, PyObject* out_given, bool with_lse, PyObject* stream,
                 const char* what, F&& call) {
  const int64_t batch = q.size(0), tokens = q.size(1), heads = q.size(2), dim = q.size(3);
  want(heads >= 1 && heads % c.c.kv_heads == 0, "q_heads must be a multiple of kv_heads");
  check_table(table, batch, c.device, "page_table must be an int32 CUDA tensor [batch, pages of a sequence] with contiguous rows");
  want(batch <= INT32_MAX && tokens <= INT32_MAX && heads <= INT32_MAX && table.size(1) <= INT32_MAX, "too many queries");
  const double s = scale == Py_None ? 1.0 / std::sqrt((double)dim) : PyFloat_AsDouble(scale);
  if (PyErr_Occurred()) throw Raised();
  want(std::isfinite((float)((double)(float)s * 1.4426950408889634)), "softmax_scale must be finite, times log2(e) too");
  Place place(stream, c.device);
  Tensor out, lse;
  if (out_given == Py_None) {
    out = fresh(q.sizes(), at::kBFloat16, c.device);
  } else {
    out = tensor(out_given, "out");
    want(out.sizes() == q.sizes() && out.scalar_type() == at::kBFloat16 && out.device() == c.device && out.is_contiguous() && aligned16(out.data_ptr()),
         "out must be a contiguous, 16-byte aligned bfloat16 CUDA tensor of q's shape");
  }
  if (with_lse) lse = fresh({batch, tokens, heads}, at::kFloat, c.device);
  const Tensor x = readable(q);
  tks_queries r = queries_of(x, table);
  r.out = out.data_ptr();
  r.lse = with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
  r.softmax_scale = (float)s;
  check(call(&c.c, &r, place.stream), what);
  if (!with_lse) return THPVariable_Wrap(out);
  return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

void check_q(const Tensor& q, const Paged& c) {
  want(q.dim() == 4 && q.scalar_type() == at::kBFloat16 && q.device() == c.device && q.size(3) == c.c.head_dim,
       "q must be a bfloat16 CUDA tensor [batch, tokens, q_heads, head_dim] on the cache's device");
}

// tree(q, k_cache, v_cache, page_table, ctx_len, tree, draft_len, scales, softmax_scale, out, return_lse, stream)
PyObject* py_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor q = tensor(a[0], "q"), table = tensor(a[3], "page_table"), ctx = tensor(a[4], "ctx_len");
    const std::optional<Tensor> tree = maybe(a[5], "tree"), count = maybe(a[6], "draft_len");
    const Paged c = cache_of(tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), maybe(a[7], "scales"));
    check_q(q, c);
    const int64_t batch = q.size(0), tokens = q.size(1);
    want(tokens <= TKS_DRAFTS_MAX, "too many drafted tokens (TKS_DRAFTS_MAX)");
    const int32_t* p_ctx = ints(ctx, {batch}, c.device, "ctx_len");
    const int32_t* p_count = count ? ints(*count, {batch}, c.device, "draft_len") : nullptr;
    const int32_t* p_tree = tree ? ints(*tree, {batch, tokens, (tokens + 31) / 32}, c.device, "tree") : nullptr;
    return attend(c, q, table, a[8], a[9], a[10] == Py_True, a[11], "tks_tree_attention",
                  [&](const tks_cache* pc, const tks_queries* pq, void* s) { return f_tree(pc, pq, p_ctx, p_count, p_tree, s); });
  });
}

// selected(q, k_cache, v_cache, page_table, indices, kv_len, scales, softmax_scale, out, return_lse, stream)
PyObject* py_selected(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor q = tensor(a[0], "q"), table = tensor(a[3], "page_table"), indices = tensor(a[4], "indices");
    const std::optional<Tensor> limit = maybe(a[5], "kv_len");
    const Paged c = cache_of(tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), maybe(a[6], "scales"));
    check_q(q, c);
    const int64_t batch = q.size(0), tokens = q.size(1);
    want(indices.dim() == 3, "indices must be an int32 CUDA tensor [batch, tokens, k]");
    const int64_t k = indices.size(2);
    const int32_t* p_idx = ints(indices, {batch, tokens, k}, c.device, "indices");
    const int32_t* p_limit = limit ? ints(*limit, {batch}, c.device, "kv_len") : nullptr;
    want(k <= TKS_K_MAX, "too many selected positions (TKS_K_MAX)");
    return attend(c, q, table, a[7], a[8], a[9] == Py_True, a[10], "tks_selected_attention",
                  [&](const tks_cache* pc, const tks_queries* pq, void* s) { return f_selected(pc, pq, p_idx, (int32_t)k, p_limit, s); });
  });
}

// set_library(TksError, write, read, tree, selected): the entry points' addresses
PyObject* py_set(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "set_library takes TksError and four addresses");
    return nullptr;
  }
  void* f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XDECREF(tks_error);
  tks_error = a[0];
  f_write = reinterpret_cast<decltype(f_write)>(f[0]);
  f_read = reinterpret_cast<decltype(f_read)>(f[1]);
  f_tree = reinterpret_cast<decltype(f_tree)>(f[2]);
  f_selected = reinterpret_cast<decltype(f_selected)>(f[3]);
  Py_RETURN_NONE;
}

// The bounds of a cache's blocks, and their device. page_size: the cache's, or 0: made of `block`.
struct Bounds {
  tks_bounds b;
  at::Device device;
};
Bounds bounds_of(const Tensor& t, int64_t page_size, int64_t block) {
  want(t.dim() == 5 && t.is_cuda() && t.scalar_type() == at::kBFloat16 && t.size(3) == 2 && t.is_contiguous() && aligned16(t.data_ptr()),
       "bounds must be a contiguous, 16-byte aligned bfloat16 CUDA tensor [pages, blocks of a page, kv_heads, 2, head_dim]");
  const int64_t pages = t.size(0), of_page = t.size(1), heads = t.size(2), dim = t.size(4);
  want(dim == 64 || dim == 128, "head_dim must be 64 or 128");
  want(pages >= 1 && heads >= 1 && of_page >= 1 && (of_page & (of_page - 1)) == 0, "a page's blocks are a power of two");
  if (page_size) {
    want(of_page <= page_size, "a page has at most as many blocks as tokens");
    block = page_size / of_page;
  }
  want(block >= 1 && (block & (block - 1)) == 0 && block <= INT32_MAX / of_page, "block must be a power of two");
  want(pages <= INT32_MAX && heads <= INT32_MAX, "too many pages or heads");
  Bounds r{tks_bounds{}, t.device()};
  r.b.bounds = t.data_ptr();
  r.b.block = (int32_t)block;
  r.b.pages = (int32_t)pages;
  r.b.page_size = (int32_t)(block * of_page);
  r.b.kv_heads = (int32_t)heads;
  r.b.head_dim = (int32_t)dim;
  return r;
}
Bounds bounds_of(const Tensor& t, const Paged& c) {
  Bounds r = bounds_of(t, c.c.page_size, 0);
  want(r.device == c.device && r.b.pages == c.c.pages && r.b.kv_heads == c.c.kv_heads && r.b.head_dim == c.c.head_dim,
       "bounds must have the cache's pages, heads, head_dim and device");
  return r;
}

int64_t number(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < 0 || v > INT32_MAX) throw Refused(std::string(what) + " must be in [0, 2^31)");
  return v;
}

// bounds(k_cache, page_table, end, bounds, start, scales, stream)
PyObject* py_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity_blocks(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor k = tensor(a[0], "k_cache"), table = tensor(a[1], "page_table"), end = tensor(a[2], "end"), bounds = tensor(a[3], "bounds");
    const std::optional<Tensor> start = maybe(a[4], "start");
    const Paged c = cache_of(k, k, maybe(a[5], "scales"));
    const Bounds b = bounds_of(bounds, c);
    check_table(table, -1, c.device, "page_table must be an int32 CUDA tensor [batch, pages of a sequence] with contiguous rows, on the cache's device");
    const int64_t batch = table.size(0);
    want(batch <= INT32_MAX && table.size(1) <= INT32_MAX, "too many sequences");
    const int32_t* p_end = ints(end, {batch}, c.device, "end");
    const int32_t* p_start = start ? ints(*start, {batch}, c.device, "start") : nullptr;
    Place place(a[6], c.device);
    check(f_bounds(&c.c, &b.b, static_cast<const int32_t*>(table.data_ptr()), step(table, 0), (int32_t)table.size(1), (int32_t)batch, p_start, p_end,
                   place.stream),
          "tks_cache_bounds");
    Py_RETURN_NONE;
  });
}

// scores(q, bounds, page_table, kv_len, block, first, last, n, out, stream) -> (scores, row_len)
PyObject* py_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity_blocks(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor q = tensor(a[0], "q"), table = tensor(a[2], "page_table");
    const std::optional<Tensor> lens = maybe(a[3], "kv_len");
    const Bounds b = bounds_of(tensor(a[1], "bounds"), 0, number(a[4], "block"));
    want(q.dim() == 4 && q.scalar_type() == at::kBFloat16 && q.device() == b.device && q.size(3) == b.b.head_dim,
         "q must be a bfloat16 CUDA tensor [batch, tokens, q_heads, head_dim] on the bounds' device");
    const int64_t batch = q.size(0), tokens = q.size(1), heads = q.size(2);
    want(heads >= 1 && heads % b.b.kv_heads == 0, "q_heads must be a multiple of kv_heads");
    check_table(table, batch, b.device, "page_table must be an int32 CUDA tensor [batch, pages of a sequence] with contiguous rows");
    want(batch <= INT32_MAX && tokens <= INT32_MAX && heads <= INT32_MAX && table.size(1) <= INT32_MAX, "too many queries");
    const int32_t* p_lens = lens ? ints(*lens, {batch, tokens}, b.device, "kv_len") : nullptr;
    const int64_t most = table.size(1) * (b.b.page_size / b.b.block), columns = a[7] == Py_None ? most : number(a[7], "n");
    want(columns <= most && columns <= INT32_MAX, "n must not exceed the blocks of a page table's row");
    const int64_t first = number(a[5], "first"), last = number(a[6], "last");
    Place place(a[9], b.device);
    const int64_t shape[4] = {batch, tokens, b.b.kv_heads, columns};
    Tensor out;
    if (a[8] == Py_None) {
      out = fresh(shape, at::kFloat, b.device);
    } else {
      out = tensor(a[8], "out");
      want(out.sizes() == at::IntArrayRef(shape) && out.scalar_type() == at::kFloat && out.device() == b.device && out.is_contiguous(),
           "out must be a contiguous float32 CUDA tensor [batch, tokens, kv_heads, n]");
    }
    // (an allocation of its own: storage that float32 and int32 tensors share cannot be saved)
    const Tensor row_len = fresh({batch, tokens, b.b.kv_heads}, at::kInt, b.device);
    const Tensor x = readable(q);
    const tks_queries r = queries_of(x, table);
    check(f_scores(&b.b, &r, p_lens, (int32_t)first, (int32_t)last, static_cast<float*>(out.data_ptr()), (int32_t)columns,
                   static_cast<int32_t*>(row_len.data_ptr()), place.stream),
          "tks_block_scores");
    return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(row_len));
  });
}

// block(q, k_cache, v_cache, page_table, blocks, block, kv_len, scales, softmax_scale, out, return_lse, stream)
PyObject* py_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity_blocks(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor q = tensor(a[0], "q"), table = tensor(a[3], "page_table"), blocks = tensor(a[4], "blocks");
    const int64_t block = number(a[5], "block");
    const std::optional<Tensor> lens = maybe(a[6], "kv_len");
    const Paged c = cache_of(tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), maybe(a[7], "scales"));
    check_q(q, c);
    const int64_t batch = q.size(0), tokens = q.size(1);
    want(blocks.dim() == 4, "blocks must be an int32 CUDA tensor [batch, tokens, kv_heads, n]");
    const int64_t count = blocks.size(3);
    const int32_t* p_blocks = ints(blocks, {batch, tokens, c.c.kv_heads, count}, c.device, "blocks");
    const int32_t* p_lens = lens ? ints(*lens, {batch, tokens}, c.device, "kv_len") : nullptr;
    want(block >= 1 && (block & (block - 1)) == 0, "block must be a power of two");
    want(count <= TKS_K_MAX && count * block <= TKS_K_MAX, "too many positions in a list (TKS_K_MAX)");
    return attend(c, q, table, a[8], a[9], a[10] == Py_True, a[11], "tks_block_attention", [&](const tks_cache* pc, const tks_queries* pq, void* s) {
      return f_block(pc, pq, p_blocks, (int32_t)count, (int32_t)block, p_lens, s);
    });
  });
}

// What fork and compact share.
struct Plan {
  Tensor table, lens;
  std::optional<Tensor> keep;
  int64_t rows, width, pages, page;
  const uint8_t* p_keep;
  at::Device device;
};
Plan plan_of(PyObject* table, PyObject* lens, PyObject* pages, PyObject* page_size, PyObject* keep) {
  Plan r{tensor(table, "page_table"), tensor(lens, "lens"), maybe(keep, "keep"), 0, 0, number(pages, "pages"), number(page_size, "page_size"), nullptr,
         at::Device(at::kCPU)};
  r.device = r.table.device();
  check_table(r.table, -1, r.device, "page_table must be an int32 CUDA tensor [sequences, pages of a sequence] with contiguous rows");
  r.rows = r.table.size(0);
  r.width = r.table.size(1);
  want(r.rows <= INT32_MAX && r.width <= INT32_MAX, "too many sequences");
  ints(r.lens, {r.rows}, r.device, "lens");
  want(r.pages >= 1 && r.page >= 1 && (r.page & (r.page - 1)) == 0 && r.pages * r.page <= INT32_MAX,
       "a cache has at least one page, of a power of two of tokens, and fewer than 2^31 in all");
  if (r.keep) {
    want((r.keep->scalar_type() == at::kByte || r.keep->scalar_type() == at::kBool) && r.keep->dim() == 1 && r.keep->size(0) == r.pages &&
             r.keep->device() == r.device && r.keep->is_contiguous(),
         "keep must be a contiguous bool or uint8 CUDA tensor [pages] on the page table's device");
    r.p_keep = static_cast<const uint8_t*>(r.keep->data_ptr());
  }
  return r;
}
// (An allocation for each output and for the scratch buffer: as parts of one, whoever kept one of them would keep them all.)
Tensor new_ints(at::IntArrayRef shape, const at::Device& device) { return fresh(shape, at::kInt, device); }
Tensor table_out(PyObject* given, int64_t rows, int64_t width, const at::Device& device) {
  const int64_t shape[2] = {rows, width};
  if (given == Py_None) return new_ints(shape, device);
  Tensor t = tensor(given, "out");
  ints(t, shape, device, "out");
  return t;
}
int32_t* words(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// fork(page_table, lens, parents, new_lens, pages, page_size, keep, out, stream) -> (table, src, dst)
PyObject* py_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity_blocks(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Plan p = plan_of(a[0], a[1], a[4], a[5], a[6]);
    const Tensor parents = tensor(a[2], "parents"), new_lens = tensor(a[3], "new_lens");
    const int64_t children = parents.numel();
    want(children <= INT32_MAX, "too many children");
    const int32_t* p_parents = ints(parents, {children}, p.device, "parents");
    const int32_t* p_lens = ints(new_lens, {children}, p.device, "new_lens");
    Place place(a[8], p.device);
    Tensor out = table_out(a[7], children, p.width, p.device);
    const Tensor scratch = new_ints({TKS_PAGES_SCRATCH(p.pages, children)}, p.device), src = new_ints({children}, p.device), dst = new_ints({children}, p.device);
    check(f_fork(words(p.table), step(p.table, 0), (int32_t)p.width, (int32_t)p.rows, words(p.lens), p_parents, p_lens, (int32_t)children, p.p_keep,
                 (int32_t)p.pages, (int32_t)p.page, words(out), words(src), words(dst), words(scratch), place.stream),
          "tks_cache_fork");
    return Py_BuildValue("NNN", THPVariable_Wrap(out), THPVariable_Wrap(src), THPVariable_Wrap(dst));
  });
}

// compact(page_table, lens, pages, page_size, keep, out, stream) -> (table, src, dst, count)
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity_blocks(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Plan p = plan_of(a[0], a[1], a[2], a[3], a[4]);
    Place place(a[6], p.device);
    Tensor out = table_out(a[5], p.rows, p.width, p.device);
    const Tensor scratch = new_ints({TKS_PAGES_SCRATCH(p.pages, p.rows)}, p.device), src = new_ints({p.pages / 2}, p.device),
                 dst = new_ints({p.pages / 2}, p.device), count = new_ints({2}, p.device);
    check(f_compact(words(p.table), step(p.table, 0), (int32_t)p.width, (int32_t)p.rows, words(p.lens), p.p_keep, (int32_t)p.pages, (int32_t)p.page,
                    words(out), words(src), words(dst), words(count), words(scratch), place.stream),
          "tks_cache_compact");
    return Py_BuildValue("NNNN", THPVariable_Wrap(out), THPVariable_Wrap(src), THPVariable_Wrap(dst), THPVariable_Wrap(count));
  });
}

// copy(src, dst, k_cache, v_cache, scales, bounds, count, stream)
PyObject* py_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity_blocks(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor src = tensor(a[0], "src"), dst = tensor(a[1], "dst");
    const Paged c = cache_of(tensor(a[2], "k_cache"), tensor(a[3], "v_cache"), maybe(a[4], "scales"));
    const std::optional<Tensor> bounds = maybe(a[5], "bounds"), count = maybe(a[6], "count");
    std::optional<Bounds> b;
    if (bounds) b = bounds_of(*bounds, c);
    const int64_t pairs = src.numel();
    want(pairs <= INT32_MAX, "too many pages");
    const int32_t* p_src = ints(src, {pairs}, c.device, "src");
    const int32_t* p_dst = ints(dst, {pairs}, c.device, "dst");
    if (count)
      want(count->scalar_type() == at::kInt && count->numel() >= 1 && count->is_contiguous() && count->device() == c.device,
           "count must be a contiguous int32 CUDA tensor on the cache's device, whose first element counts");
    Place place(a[7], c.device);
    check(f_copy(&c.c, b ? &b->b : nullptr, p_src, p_dst, (int32_t)pairs, count ? words(*count) : nullptr, place.stream), "tks_cache_copy");
    Py_RETURN_NONE;
  });
}

// set_blocks(TksError, bounds, scores, block attention, fork, compact, copy): the entry points' addresses
PyObject* py_set_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "set_blocks takes TksError and six addresses");
    return nullptr;
  }
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XDECREF(tks_error);
  tks_error = a[0];
  f_bounds = reinterpret_cast<decltype(f_bounds)>(f[0]);
  f_scores = reinterpret_cast<decltype(f_scores)>(f[1]);
  f_block = reinterpret_cast<decltype(f_block)>(f[2]);
  f_fork = reinterpret_cast<decltype(f_fork)>(f[3]);
  f_compact = reinterpret_cast<decltype(f_compact)>(f[4]);
  f_copy = reinterpret_cast<decltype(f_copy)>(f[5]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"set_library", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_set)), METH_FASTCALL, nullptr},
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_write)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_read)), METH_FASTCALL, nullptr},
    {"tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_tree)), METH_FASTCALL, nullptr},
    {"selected", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_selected)), METH_FASTCALL, nullptr},
    {"set_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_set_blocks)), METH_FASTCALL, nullptr},
    {"bounds", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_bounds)), METH_FASTCALL, nullptr},
    {"scores", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_scores)), METH_FASTCALL, nullptr},
    {"block", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_block)), METH_FASTCALL, nullptr},
    {"fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_fork)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_compact)), METH_FASTCALL, nullptr},
    {"copy", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_copy)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tks_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tks_binding() { return PyModule_Create(&module); }
