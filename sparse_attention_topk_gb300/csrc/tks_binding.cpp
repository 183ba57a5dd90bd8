// The Python side of the cache and attention calls: checks of the tensors, the
// outputs' allocation and the call of the C entry point (include/tks_attention.h),
// in one C++ step.  A decode step makes these calls for every layer, and the
// same work in Python took longer than the kernels of a short context (33 us
// of host time a call, 6 so, where the kernels take 9).
//
// The module calls the entry points of the libtks that the package has loaded
// (set_library), so there is no second copy of the library.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <optional>
#include <string>

#include "tks_attention.h"

namespace {

using at::Tensor;

decltype(&tks_cache_write) f_write = nullptr;
decltype(&tks_cache_read) f_read = nullptr;
decltype(&tks_tree_attention) f_tree = nullptr;
decltype(&tks_selected_attention) f_selected = nullptr;
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

bool arity(Py_ssize_t n, Py_ssize_t wanted) {
  if (n == wanted && f_write) return true;
  PyErr_SetString(PyExc_TypeError, f_write ? "wrong number of arguments" : "the library is not set");
  return false;
}

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
        out[i] = at::empty(shape, at::TensorOptions().dtype(type).device(c.device));
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

// What both attention calls share: the queries, the page table, the outputs.
template <typename F>
PyObject* attend(const Paged& c, const Tensor& q, const Tensor& table, PyObject* scale, PyObject* out_given, bool with_lse, PyObject* stream,
                 const char* what, F&& call) {
  const int64_t batch = q.size(0), tokens = q.size(1), heads = q.size(2), dim = q.size(3);
  want(heads >= 1 && heads % c.c.kv_heads == 0, "q_heads must be a multiple of kv_heads");
  want(table.dim() == 2 && table.size(0) == batch && table.scalar_type() == at::kInt && table.device() == c.device &&
           (table.size(1) <= 1 || table.stride(1) == 1),
       "page_table must be an int32 CUDA tensor [batch, pages of a sequence] with contiguous rows");
  want(batch <= INT32_MAX && tokens <= INT32_MAX && heads <= INT32_MAX && table.size(1) <= INT32_MAX, "too many queries");
  const double s = scale == Py_None ? 1.0 / std::sqrt((double)dim) : PyFloat_AsDouble(scale);
  if (PyErr_Occurred()) throw Raised();
  want(std::isfinite((float)((double)(float)s * 1.4426950408889634)), "softmax_scale must be finite, times log2(e) too");
  Place place(stream, c.device);
  Tensor out, lse;
  if (out_given == Py_None) {
    out = at::empty(q.sizes(), at::TensorOptions().dtype(at::kBFloat16).device(c.device));
  } else {
    out = tensor(out_given, "out");
    want(out.sizes() == q.sizes() && out.scalar_type() == at::kBFloat16 && out.device() == c.device && out.is_contiguous() && aligned16(out.data_ptr()),
         "out must be a contiguous, 16-byte aligned bfloat16 CUDA tensor of q's shape");
  }
  if (with_lse) lse = at::empty({batch, tokens, heads}, at::TensorOptions().dtype(at::kFloat).device(c.device));
  const Tensor x = readable(q);
  tks_queries r{};
  r.q = x.data_ptr();
  r.q_batch_stride = step(x, 0);
  r.q_token_stride = step(x, 1);
  r.q_head_stride = step(x, 2);
  r.out = out.data_ptr();
  r.lse = with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
  r.batch = (int32_t)batch;
  r.tokens = (int32_t)tokens;
  r.q_heads = (int32_t)heads;
  r.page_table = static_cast<const int32_t*>(table.data_ptr());
  r.table_stride = step(table, 0);
  r.table_pages = (int32_t)table.size(1);
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

PyMethodDef methods[] = {
    {"set_library", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_set)), METH_FASTCALL, nullptr},
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_write)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_read)), METH_FASTCALL, nullptr},
    {"tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_tree)), METH_FASTCALL, nullptr},
    {"selected", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_selected)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tks_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tks_binding() { return PyModule_Create(&module); }
