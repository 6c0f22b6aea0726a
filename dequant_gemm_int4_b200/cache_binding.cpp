// The tensor side of the int4_cache_* entries as a CPython extension: checks
// of the arguments, outputs and workspace from torch's allocator, the current
// stream, and the call of the C ABI.  dequant_gemm_int4_b200/cache.py wraps
// it and documents the functions.
//
// A decoding step calls these once a layer on a few tokens, where the kernels
// take 2 to 10 us: through ctypes and Python checks a call took 14 us (read)
// to 28 us (attention) on the host, more than the GPU's time.
//
// Functions return None or their outputs, or the C entry's status as an int
// where it is not INT4_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <string>

#include "int4.h"

namespace {

decltype(&int4_cache_write) p_write = nullptr;
decltype(&int4_cache_read) p_read = nullptr;
decltype(&int4_cache_attention) p_attention = nullptr;
decltype(&int4_cache_attention_workspace_size) p_workspace_size = nullptr;

using at::Tensor;

// Argument errors, thrown as C++ and raised as Python exceptions below.
struct BadType { std::string what; };
struct BadValue { std::string what; };
[[noreturn]] void type_error(std::string what) { throw BadType{std::move(what)}; }
[[noreturn]] void value_error(std::string what) { throw BadValue{std::move(what)}; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a truth value");
  }
  return v == 1;
}

// One of the INT4_PATH_* codes, as far as an int32 holds it.
int32_t path_code(PyObject* o) {
  const int64_t v = integer(o, "path");
  if (v < INT32_MIN || v > INT32_MAX) value_error("path must be one of the PATH_* codes");
  return static_cast<int32_t>(v);
}

int dtype_code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return INT4_DTYPE_F32;
    case at::kBFloat16: return INT4_DTYPE_BF16;
    case at::kHalf: return INT4_DTYPE_F16;
    default: return -1;
  }
}

void need_cuda(const Tensor& t, const char* name) {
  if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
}
void need_dense(const Tensor& t, const char* name) {
  need_cuda(t, name);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous (row-major, no padding)");
}

// A cache's tensors, checked, and their C view.
struct Cache {
  int4_cache c;
  c10::DeviceIndex device;

  Cache(PyObject* py_packed, PyObject* py_scales, PyObject* py_zeros, int64_t head_dim, int64_t group) {
    const Tensor& packed = tensor(py_packed, "packed");
    const Tensor& scales = tensor(py_scales, "scales");
    const Tensor* zeros = py_zeros == Py_None ? nullptr : &tensor(py_zeros, "zeros");
    if (group < 1 || head_dim < 1) value_error("group and head_dim must be >= 1");
    if (packed.scalar_type() != at::kByte || packed.dim() != 5 || packed.size(1) != 2 ||
        packed.size(4) != (head_dim + 1) / 2)
      value_error("packed must be uint8 [pages, 2, heads, page_size, ceil(head_dim/2)]");
    if (packed.size(2) < 1 || packed.size(3) < 1) value_error("the cache's heads and page_size must be >= 1");
    const int64_t groups = group >= head_dim ? 1 : (head_dim + group - 1) / group;
    const auto fits = [&](const Tensor& t) {
      return t.dim() == 5 && t.size(0) == packed.size(0) && t.size(1) == 2 && t.size(2) == packed.size(2) &&
             t.size(3) == packed.size(3) && t.size(4) == groups;
    };
    if (scales.scalar_type() != at::kHalf || !fits(scales))
      value_error("scales must be float16 [pages, 2, heads, page_size, ceil(head_dim/group)]");
    if (zeros != nullptr && (zeros->scalar_type() != at::kByte || !fits(*zeros)))
      value_error("zeros must be uint8, shaped as scales");
    if (packed.size(2) > INT32_MAX || packed.size(3) > INT32_MAX || head_dim > INT32_MAX)
      value_error("heads, page_size and head_dim must be below 2^31");
    need_dense(packed, "packed");
    need_dense(scales, "scales");
    device = packed.get_device();
    on(scales, "scales");
    if (zeros != nullptr) {
      need_dense(*zeros, "zeros");
      on(*zeros, "zeros");
    }
    c.packed = packed.data_ptr();
    c.scales = scales.data_ptr();
    c.zeros = zeros == nullptr ? nullptr : zeros->data_ptr();
    // An empty tensor has no address, but the affine scheme stays what it is.
    if (zeros != nullptr && c.zeros == nullptr) c.zeros = reinterpret_cast<void*>(static_cast<uintptr_t>(256));
    c.pages = packed.size(0);
    c.heads = static_cast<int32_t>(packed.size(2));
    c.page_size = static_cast<int32_t>(packed.size(3));
    c.head_dim = static_cast<int32_t>(head_dim);
    c.group = static_cast<int32_t>(group < head_dim ? group : head_dim);
  }
  void on(const Tensor& t, const char* name) const {
    if (t.get_device() != device) value_error(std::string(name) + " must be on the cache's device");
  }
  // t [tokens, heads, head_dim] of a floating type with a dense last dimension.
  void rows(const Tensor& t, const char* name, bool own_heads) const {
    if (t.dim() != 3 || t.size(2) != c.head_dim || (own_heads && t.size(1) != c.heads))
      value_error(std::string(name) + " must be [tokens, heads, head_dim]");
    if (dtype_code(t) < 0) type_error(std::string(name) + " must be float32, bfloat16 or float16");
    need_cuda(t, name);
    if (c.head_dim > 1 && t.stride(2) != 1)
      value_error(std::string(name) + "'s last dimension must be contiguous");
    on(t, name);
  }
  // A dense index tensor of one dimension.
  const Tensor& index(PyObject* o, const char* name, at::ScalarType type, int64_t size) const {
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.dim() != 1 || (size >= 0 && t.size(0) != size))
      value_error(std::string(name) + " must be " + (type == at::kLong ? "int64" : "int32") + " [" +
                  (size >= 0 ? std::to_string(size) : std::string("tokens")) + "]");
    need_dense(t, name);
    on(t, name);
    return t;
  }
};

// The cache's device and its current stream, for the time of a call.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit Place(c10::DeviceIndex device) {
    if (c10::cuda::current_device() != device) guard.set_index(device);
    stream = c10::cuda::getCurrentCUDAStream(device).stream();
  }
};

// A new dense tensor on the cache's device (at::empty's work without its way
// through the dispatcher, which took longer than the rest of a call's checks).
Tensor empty(at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex device) {
  return Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, device), std::nullopt));
}

// Device memory for one call, ordered on its stream.
struct Scratch {
  void* p = nullptr;
  explicit Scratch(size_t n) {
    if (n > 0) p = c10::cuda::CUDACachingAllocator::raw_alloc(n);
  }
  ~Scratch() {
    if (p != nullptr) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
  Scratch(const Scratch&) = delete;
};

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const BadType& e) {
    PyErr_SetString(PyExc_TypeError, e.what.c_str());
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch == nullptr ? nullptr : PyObject_GetAttrString(torch, "OutOfMemoryError");
    if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return false;
}

// write(k, v, packed, scales, slots, group, zeros)
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& k = tensor(a[0], "k");
    const Tensor& v = tensor(a[1], "v");
    if (k.dim() != 3) value_error("k must be [tokens, heads, head_dim]");
    const Cache cache(a[2], a[3], a[6], k.size(2), integer(a[5], "group"));
    cache.rows(k, "k", true);
    cache.rows(v, "v", true);
    if (v.size(0) != k.size(0) || v.scalar_type() != k.scalar_type())
      value_error("v must have k's shape and dtype");
    const Tensor& slots = cache.index(a[4], "slots", at::kLong, k.size(0));
    const Place place(cache.device);
    const int rc = p_write(&cache.c, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                           v.stride(1), dtype_code(k), k.size(0), static_cast<const int64_t*>(slots.data_ptr()),
                           place.stream);
    if (rc != INT4_OK) return PyLong_FromLong(rc);
    Py_RETURN_NONE;
  });
}

// read(packed, scales, slots, head_dim, group, dtype code, zeros, k, v); k and
// v None: new tensors.
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache cache(a[0], a[1], a[6], integer(a[3], "head_dim"), integer(a[4], "group"));
    const Tensor& slots = cache.index(a[2], "slots", at::kLong, -1);
    const int64_t code = integer(a[5], "dtype");
    const at::ScalarType type = code == INT4_DTYPE_F32 ? at::kFloat : code == INT4_DTYPE_BF16 ? at::kBFloat16 : at::kHalf;
    const int64_t shape[3] = {slots.size(0), cache.c.heads, cache.c.head_dim};
    Tensor out[2];
    const Place place(cache.device);
    for (int i = 0; i < 2; ++i) {
      if (a[7 + i] == Py_None) {
        out[i] = empty(shape, type, cache.device);
        continue;
      }
      out[i] = tensor(a[7 + i], "out");
      if (out[i].scalar_type() != type || out[i].sizes() != at::IntArrayRef(shape))
        value_error("out must be two tensors [tokens, heads, head_dim] of dtype");
      need_dense(out[i], "out");
      cache.on(out[i], "out");
    }
    const char* const at[2] = {static_cast<const char*>(out[0].data_ptr()), static_cast<const char*>(out[1].data_ptr())};
    if (at[0] < at[1] + out[1].nbytes() && at[1] < at[0] + out[0].nbytes()) value_error("out's two tensors overlap");
    const int rc = p_read(&cache.c, static_cast<const int64_t*>(slots.data_ptr()), slots.size(0), out[0].data_ptr(),
                          out[1].data_ptr(), static_cast<int32_t>(code), place.stream);
    if (rc != INT4_OK) return PyLong_FromLong(rc);
    PyObject* k = THPVariable_Wrap(std::move(out[0]));
    PyObject* v = THPVariable_Wrap(std::move(out[1]));
    PyObject* both = PyTuple_Pack(2, k, v);
    Py_XDECREF(k);
    Py_XDECREF(v);
    return both;
  });
}

// What the attention and its workspace query check alike.
struct Queries {
  const Tensor& q;
  Cache cache;
  const Tensor& table;
  Queries(PyObject* py_q, PyObject* packed, PyObject* scales, PyObject* py_table, PyObject* zeros, int64_t group)
      : q(query(py_q)), cache(packed, scales, zeros, q.size(2), group), table(tensor(py_table, "page_table")) {
    cache.rows(q, "q", false);
    if (q.size(1) < 1 || q.size(1) % cache.c.heads != 0 || q.size(1) > INT32_MAX)
      value_error("q_heads must be a multiple of the cache's heads");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) > INT32_MAX || table.size(1) > INT32_MAX)
      value_error("page_table must be int32 [batch, max_pages]");
    need_cuda(table, "page_table");
    cache.on(table, "page_table");
    if (table.size(1) > 1 && table.stride(1) != 1) value_error("page_table's rows must be contiguous");
  }
  static const Tensor& query(PyObject* o) {
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 3) value_error("q must be [rows, q_heads, head_dim]");
    return THPVariable_Unpack(o);
  }
  int workspace(int32_t path, size_t* bytes) const {
    return p_workspace_size(&cache.c, dtype_code(q), q.size(0), static_cast<int32_t>(q.size(1)),
                            static_cast<int32_t>(table.size(0)), static_cast<int32_t>(table.size(1)), path, bytes);
  }
};

// workspace_size(q, packed, scales, page_table, group, zeros, path) -> bytes, or -status
PyObject* workspace_size(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const int32_t path = path_code(a[6]);
    const Queries x(a[0], a[1], a[2], a[3], a[5], integer(a[4], "group"));
    const Place place(x.cache.device);
    size_t bytes = 0;
    const int rc = x.workspace(path, &bytes);
    return PyLong_FromLongLong(rc == INT4_OK ? static_cast<long long>(bytes) : -rc);
  });
}

// attention(q, packed, scales, page_table, kv_lens, group, zeros, q_starts,
// causal, window, sm_scale, return_lse, out, lse, path, workspace)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 16)) return nullptr;
  return guarded([&]() -> PyObject* {
    const bool causal = truth(a[8], "causal"), return_lse = truth(a[11], "return_lse");
    const int32_t path = path_code(a[14]);
    const Queries x(a[0], a[1], a[2], a[3], a[6], integer(a[5], "group"));
    const Tensor& q = x.q;
    const Cache& cache = x.cache;
    const int64_t rows = q.size(0), batch = x.table.size(0);
    const Tensor& kv_lens = cache.index(a[4], "kv_lens", at::kInt, batch);
    const Tensor* q_starts = a[7] == Py_None ? nullptr : &cache.index(a[7], "q_starts", at::kInt, batch + 1);
    if (q_starts == nullptr && rows > 0 && (batch == 0 || rows % batch != 0))
      value_error("without q_starts, the batch must divide q's rows");
    int64_t window = a[9] == Py_None ? 0 : integer(a[9], "window");
    if (window < 0) value_error("window must be None or >= 0");
    if (window > INT32_MAX) window = INT32_MAX;
    double scale = 1.0 / std::sqrt(static_cast<double>(cache.c.head_dim));
    if (a[10] != Py_None) {
      scale = PyFloat_AsDouble(a[10]);
      if (scale == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error("sm_scale must be a number");
      }
    }
    if (!std::isfinite(static_cast<float>(scale))) value_error("sm_scale must be finite");

    const Place place(cache.device);
    Tensor out, lse;
    if (a[12] == Py_None) {
      out = empty(q.sizes(), q.scalar_type(), cache.device);
    } else {
      out = tensor(a[12], "out");
      if (out.scalar_type() != q.scalar_type() || out.sizes() != q.sizes())
        value_error("out must have q's shape and dtype");
      need_dense(out, "out");
      cache.on(out, "out");
    }
    if (a[13] != Py_None) {
      lse = tensor(a[13], "lse");
      if (lse.scalar_type() != at::kFloat || lse.sizes() != q.sizes().slice(0, 2))
        value_error("lse must be float32 [rows, q_heads]");
      need_dense(lse, "lse");
      cache.on(lse, "lse");
    } else if (return_lse) {
      lse = empty(q.sizes().slice(0, 2), at::kFloat, cache.device);
    }
    size_t bytes = 0;
    void* workspace = nullptr;
    std::optional<Scratch> scratch;
    if (a[15] == Py_None) {
      const int rc = x.workspace(path, &bytes);
      if (rc != INT4_OK) return PyLong_FromLong(rc);
      scratch.emplace(bytes);
      workspace = scratch->p;
    } else {
      const Tensor& w = tensor(a[15], "workspace");
      need_dense(w, "workspace");
      if (w.scalar_type() != at::kByte || w.get_device() != cache.device)
        value_error("workspace must be a uint8 tensor on the cache's device");
      workspace = w.data_ptr();
      bytes = w.numel();
    }
    const int rc = p_attention(
        &cache.c, q.data_ptr(), q.stride(0), q.stride(1), dtype_code(q), rows, static_cast<int32_t>(q.size(1)),
        static_cast<const int32_t*>(x.table.data_ptr()), x.table.stride(0), static_cast<int32_t>(x.table.size(1)),
        static_cast<const int32_t*>(kv_lens.data_ptr()),
        q_starts == nullptr ? nullptr : static_cast<const int32_t*>(q_starts->data_ptr()), static_cast<int32_t>(batch),
        causal ? 1 : 0, static_cast<int32_t>(window), static_cast<float>(scale), out.data_ptr(),
        lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, path, workspace, bytes, place.stream);
    if (rc != INT4_OK) return PyLong_FromLong(rc);
    PyObject* py_out = a[12] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[12]);
    if (!return_lse) return py_out;
    PyObject* py_lse = a[13] == Py_None ? THPVariable_Wrap(std::move(lse)) : Py_NewRef(a[13]);
    PyObject* both = PyTuple_Pack(2, py_out, py_lse);
    Py_XDECREF(py_out);
    Py_XDECREF(py_lse);
    return both;
  });
}

// bind(addresses of the four C entries)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 4)) return nullptr;
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  p_write = reinterpret_cast<decltype(p_write)>(p[0]);
  p_read = reinterpret_cast<decltype(p_read)>(p[1]);
  p_attention = reinterpret_cast<decltype(p_attention)>(p[2]);
  p_workspace_size = reinterpret_cast<decltype(p_workspace_size)>(p[3]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), nullptr},
                         {"write", FAST(write), nullptr},
                         {"read", FAST(read), nullptr},
                         {"attention", FAST(attention), nullptr},
                         {"workspace_size", FAST(workspace_size), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding() { return PyModule_Create(&module); }
