// The per-step calls of the paged cache as a CPython module: checks of the
// tensors, the launch stream and the call into the C library.
//
// These calls run once per layer and decoding step, on the GPU for two to ten
// microseconds. Written in Python their checks took 2.5 us and the foreign call
// 1.5 us beside the 2 us of a launch, so that the host, not the GPU, set the
// pace; here both take 0.3 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "flashprefill.h"

namespace {

decltype(&fp_cache_write) cache_write_fn;
decltype(&fp_cache_read) cache_read_fn;
decltype(&fp_cache_commit) cache_commit_fn;
decltype(&fp_tree_attention) tree_attention_fn;

struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse(const char* fn, const std::string& what) {
  throw Refused{PyExc_ValueError, std::string(fn) + ": " + what};
}

const at::Tensor& tensor(const char* fn, const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(fn) + ": " + name + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }
std::string cuda_name(long dev) { return "cuda:" + std::to_string(dev); }

bool is_int32(const at::Tensor& t, long dev, int64_t n) {
  return t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == n && device_of(t) == dev && t.is_contiguous();
}
bool is_int32(const at::Tensor& t, long dev, int64_t n, int64_t cols) {
  return t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == n && (cols < 0 || t.size(1) == cols) &&
         device_of(t) == dev && t.is_contiguous();
}

// bf16 [tokens, heads, d] whose tokens are contiguous, at any distance
bool is_rows(const at::Tensor& t, long dev, int64_t tokens, int64_t heads, int64_t d) {
  return t.scalar_type() == at::kBFloat16 && t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads &&
         t.size(2) == d && device_of(t) == dev && t.stride(2) == 1 && (t.stride(1) == d || heads == 1);
}

// Launches go to the current device, on which the tensors have to be; its
// current stream unless the caller names one (None or a torch.cuda.Stream).
void* launch_stream(const char* fn, long dev, PyObject* stream) {
  const int current = c10::cuda::current_device();
  if (current != dev)
    refuse(fn, "tensors are on " + cuda_name(dev) + ", the current device is " + cuda_name(current));
  if (stream == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
  if (!raw) throw Refused{nullptr, ""};
  void* s = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (!s && PyErr_Occurred()) throw Refused{nullptr, ""};
  return s;
}

struct Rows {
  int total;
  long long k_stride, v_stride;
};
Rows packed_rows(const char* fn, const fp_cache_t* c, long dev, const at::Tensor& cu, const at::Tensor& k,
                 const at::Tensor& v) {
  if (!is_int32(cu, dev, c->batch + 1))
    refuse(fn, "cu_tokens must be a contiguous int32 [" + std::to_string(c->batch + 1) + "] on " + cuda_name(dev));
  const int64_t total = k.dim() == 3 ? k.size(0) : -1;
  if (!is_rows(k, dev, total, c->hkv, c->head_dim) || !is_rows(v, dev, total, c->hkv, c->head_dim) || total > INT_MAX)
    refuse(fn, "k and v must be bfloat16 [tokens, " + std::to_string(c->hkv) + ", " + std::to_string(c->head_dim) +
                   "] on " + cuda_name(dev) + ", contiguous within a token");
  // (the stride of a single row is whatever its tensor happens to say)
  const long long row = (long long)c->hkv * c->head_dim;
  return {(int)total, total > 1 ? k.stride(0) : row, total > 1 ? v.stride(0) : row};
}

// Each call's first two arguments: the address of its fp_cache_t, the device.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
const fp_cache_t* cache_at(PyObject* o) { return static_cast<const fp_cache_t*>(PyLong_AsVoidPtr(o)); }

PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> long {
    static const char* fn = "fp_cache_write";
    const fp_cache_t* c = cache_at(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    const at::Tensor &cu = tensor(fn, "cu_tokens", a[2]), &k = tensor(fn, "k", a[3]), &v = tensor(fn, "v", a[4]);
    const Rows r = packed_rows(fn, c, dev, cu, k, v);
    void* s = launch_stream(fn, dev, a[5]);
    return cache_write_fn(c, (const int32_t*)cu.data_ptr(), r.total, k.data_ptr(), r.k_stride, v.data_ptr(),
                          r.v_stride, s);
  });
}

PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> long {
    static const char* fn = "fp_cache_read";
    const fp_cache_t* c = cache_at(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    const at::Tensor &cu = tensor(fn, "cu_tokens", a[2]), &k = tensor(fn, "k", a[3]), &v = tensor(fn, "v", a[4]);
    const Rows r = packed_rows(fn, c, dev, cu, k, v);
    const int32_t* starts = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& t = tensor(fn, "starts", a[5]);
      if (!is_int32(t, dev, c->batch))
        refuse(fn, "starts must be a contiguous int32 [" + std::to_string(c->batch) + "] on " + cuda_name(dev));
      starts = (const int32_t*)t.data_ptr();
    }
    void* s = launch_stream(fn, dev, a[6]);
    return cache_read_fn(c, (const int32_t*)cu.data_ptr(), r.total, starts, k.data_ptr(), r.k_stride, v.data_ptr(),
                         r.v_stride, s);
  });
}

PyObject* cache_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> long {
    static const char* fn = "fp_cache_commit";
    const fp_cache_t* c = cache_at(a[0]);
    const long dev = PyLong_AsLong(a[1]), total = PyLong_AsLong(a[3]);
    if (total == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
    const at::Tensor &cu = tensor(fn, "cu_tokens", a[2]), &accept = tensor(fn, "accept", a[4]),
                     &num = tensor(fn, "num_accept", a[5]), &lens = tensor(fn, "new_lens", a[6]);
    if (!is_int32(cu, dev, c->batch + 1) || !is_int32(num, dev, c->batch) || !is_int32(lens, dev, c->batch) ||
        !is_int32(accept, dev, c->batch, -1)) {
      const std::string R = std::to_string(c->batch);
      refuse(fn, "cu_tokens [" + std::to_string(c->batch + 1) + "], accept [" + R + ", max_accept], num_accept [" + R +
                     "] and new_lens [" + R + "] must be contiguous int32 on " + cuda_name(dev));
    }
    if (total < INT_MIN || total > INT_MAX || accept.size(1) > INT_MAX) return FP_ERR_INVALID_ARG;
    void* s = launch_stream(fn, dev, a[7]);
    return cache_commit_fn(c, (const int32_t*)cu.data_ptr(), (int)total, (const int32_t*)accept.data_ptr(),
                           (const int32_t*)num.data_ptr(), (int)accept.size(1), (int32_t*)lens.data_ptr(), s);
  });
}

std::string shape3(int64_t x, int64_t y, int64_t z) {
  return "(" + std::to_string(x) + ", " + std::to_string(y) + ", " + std::to_string(z) + ")";
}

// cache, device, fp_tree_t, workspace address and bytes, cu_tokens, q, o, mask, lse, stream
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> long {
    static const char* fn = "fp_tree_attention";
    const fp_cache_t* c = cache_at(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    fp_tree_t t = *static_cast<const fp_tree_t*>(PyLong_AsVoidPtr(a[2]));
    const at::Tensor &cu = tensor(fn, "cu_tokens", a[5]), &q = tensor(fn, "q", a[6]), &o = tensor(fn, "o", a[7]);
    const int64_t total = t.total_tokens, d = c->head_dim;
    if (!is_int32(cu, dev, c->batch + 1))
      refuse(fn, "cu_tokens must be a contiguous int32 [" + std::to_string(c->batch + 1) + "] on " + cuda_name(dev));
    // (a stride of 0, of an expanded tensor, would mean packed rows to the library)
    if (!is_rows(q, dev, total, t.hq, d) || (total > 1 && q.stride(0) == 0))
      refuse(fn, "q must be bfloat16 " + shape3(total, t.hq, d) + " on " + cuda_name(dev) + ", contiguous within a token");
    if (!is_rows(o, dev, total, t.hq, d) || !o.is_contiguous())
      refuse(fn, "o must be contiguous bfloat16 " + shape3(total, t.hq, d) + " on " + cuda_name(dev));
    t.mask = nullptr;
    t.mask_words = 0;
    if (a[8] != Py_None) {
      const at::Tensor& m = tensor(fn, "mask", a[8]);
      if (!is_int32(m, dev, total, -1) || m.size(1) > INT_MAX)
        refuse(fn, "mask must be contiguous int32 [" + std::to_string(total) + ", words] on " + cuda_name(dev));
      t.mask = (const uint32_t*)m.data_ptr();
      t.mask_words = (int)m.size(1);
    }
    float* lse = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor& l = tensor(fn, "lse", a[9]);
      if (l.scalar_type() != at::kFloat || l.dim() != 2 || l.size(0) != t.hq || l.size(1) != total ||
          device_of(l) != dev || !l.is_contiguous())
        refuse(fn, "lse must be contiguous float32 (" + std::to_string(t.hq) + ", " + std::to_string(total) + ") on " +
                       cuda_name(dev));
      lse = (float*)l.data_ptr();
    }
    t.cu_tokens = (const int32_t*)cu.data_ptr();
    t.q_stride = total > 1 ? q.stride(0) : 0;
    void* s = launch_stream(fn, dev, a[10]);
    return tree_attention_fn(c, &t, q.data_ptr(), o.data_ptr(), lse, PyLong_AsVoidPtr(a[3]), PyLong_AsSize_t(a[4]), s);
  });
}

// The library whose functions are called from now on.
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  auto get = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    return f != nullptr;
  };
  if (!get(cache_write_fn, "fp_cache_write") || !get(cache_read_fn, "fp_cache_read") ||
      !get(cache_commit_fn, "fp_cache_commit") || !get(tree_attention_fn, "fp_tree_attention")) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks a paged-cache function");
    return nullptr;
  }
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"cache_write", fast(cache_write), METH_FASTCALL, nullptr},
                         {"cache_read", fast(cache_read), METH_FASTCALL, nullptr},
                         {"cache_commit", fast(cache_commit), METH_FASTCALL, nullptr},
                         {"tree_attention", fast(tree_attention), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers (tensor layout, inline accessors) this file was compiled with.
PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FP_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
