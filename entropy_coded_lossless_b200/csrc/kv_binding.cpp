// kv_binding.cpp — the Python calls of the paged KV cache (include/shn_kv.h): tensor checks and argument marshalling.
//
// A decoding step makes these calls for every layer, each with a dozen tensors, and the kernels of a small batch take a few
// microseconds: checked and marshalled in Python (0.5 us a tensor, 3 us for ctypes' 18 arguments) the calls would take longer
// than their work. Functions take positional arguments, tensors and None, and return the shn_status; what a check
// refuses is raised as ValueError before anything is enqueued. kv.py documents and wraps them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/shn_kv.h"

namespace {

using at::Tensor;

// A call's arguments, taken one after another.
struct Args {
  PyObject* const* v;
  Py_ssize_t n;
  int device = -1;  // index of the CUDA device all tensors are on

  void count(Py_ssize_t want) const {
    if (n != want) throw std::invalid_argument("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
  }
  bool none(int i) const { return v[i] == Py_None; }
  uint64_t u(int i) const {
    const unsigned long long x = PyLong_AsUnsignedLongLong(v[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw std::invalid_argument("an integer argument is negative, too large or no integer");
    }
    return x;
  }
  float f(int i) const {
    const double x = PyFloat_AsDouble(v[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw std::invalid_argument("a number was expected");
    }
    return (float)x;
  }
  const Tensor& tensor(int i, const char* name) const {
    if (!THPVariable_Check(v[i])) throw std::invalid_argument(std::string(name) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(v[i]);
    if (!t.is_cuda() || (device >= 0 && t.get_device() != device))
      throw std::invalid_argument(std::string(name) + " must be a CUDA tensor" + (device >= 0 ? " on cuda:" + std::to_string(device) : ""));
    return t;
  }
  // Address of a contiguous tensor of this type; shape: what it must be (-1: any size), nullptr: any.
  void* dev(int i, const char* name, at::ScalarType type, int64_t size = -1) const {
    const Tensor& t = tensor(i, name);
    if (t.scalar_type() != type) throw std::invalid_argument(std::string(name) + " must be " + c10::toString(type) + ", not " + c10::toString(t.scalar_type()));
    if (!t.is_contiguous()) throw std::invalid_argument(std::string(name) + " must be contiguous");
    if (size >= 0 && (t.dim() != 1 || t.numel() != size))
      throw std::invalid_argument(std::string(name) + " must have the shape (" + std::to_string(size) + ",)");
    return t.data_ptr();
  }
  int32_t* i32(int i, const char* name, int64_t size = -1) const { return static_cast<int32_t*>(dev(i, name, at::kInt, size)); }
  // bf16 rows [tokens, heads, head_dim] whose heads are contiguous; heads, tokens: what they must be, -1: any
  struct Rows {
    uint16_t* p;
    uint64_t stride;
    int64_t tokens, heads;
  };
  Rows rows(int i, const char* name, int64_t head_dim, int64_t heads = -1, int64_t tokens = -1) const {
    const Tensor& t = tensor(i, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3) throw std::invalid_argument(std::string(name) + " must be bfloat16 [tokens, heads, head_dim]");
    const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
    if (d != head_dim || (heads >= 0 && h != heads) || (tokens >= 0 && n != tokens))
      throw std::invalid_argument(std::string(name) + " has the shape [" + std::to_string(n) + ", " + std::to_string(h) + ", " + std::to_string(d) +
                                  "]; expected [" + (tokens < 0 ? "tokens" : std::to_string(tokens)) + ", " +
                                  (heads < 0 ? "heads" : std::to_string(heads)) + ", " + std::to_string(head_dim) + "]");
    if (t.stride(2) != 1 || (h > 1 && t.stride(1) != d)) throw std::invalid_argument(std::string(name) + ": the heads of a token must be contiguous");
    const int64_t s = n > 1 ? t.stride(0) : h * d;  // (the stride of a single token means nothing)
    if (s < h * d) throw std::invalid_argument(std::string(name) + ": tokens overlap");
    return {static_cast<uint16_t*>(t.data_ptr()), (uint64_t)s, n, h};
  }
  struct Table {
    int32_t* p;
    uint32_t width;
  };
  Table table(int i, int64_t reqs) const {
    const Tensor& t = tensor(i, "block_table");
    if (t.dim() != 2 || t.size(0) != reqs || t.size(1) > UINT32_MAX)
      throw std::invalid_argument("block_table must be [" + std::to_string(reqs) + ", max_blocks]");
    return {i32(i, "block_table"), (uint32_t)t.size(1)};
  }
  void* work(int i, size_t& bytes) const {
    void* p = dev(i, "work", at::kByte);
    bytes = (size_t)THPVariable_Unpack(v[i]).numel();
    return p;
  }
  // (address of the C struct, device index), as Cache holds them
  const shn_kv_cache* cache(int i) {
    device = (int)u(i + 1);
    return reinterpret_cast<const shn_kv_cache*>((uintptr_t)u(i));
  }
};

// The call's device made current around it, and its stream: the caller's, or the device's current one. What may be refused is
// asked first, so that a refusal leaves the device as it was; and putting it back raises nothing, whatever the call met.
struct On {
  void* stream;
  int before;
  bool changed;
  On(const Args& a, int i)
      : stream(a.none(i) ? static_cast<void*>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)a.device).stream()) : reinterpret_cast<void*>((uintptr_t)a.u(i))),
        before(c10::cuda::current_device()),
        changed(before != a.device) {
    if (changed) c10::cuda::set_device((c10::DeviceIndex)a.device);
  }
  ~On() {
    if (changed) (void)c10::cuda::SetDevice((c10::DeviceIndex)before);
  }
};

// No C++ exception passes into the interpreter.
template <typename F>
PyObject* guarded(PyObject* const* v, Py_ssize_t n, F f) {
  try {
    Args a{v, n};
    return PyLong_FromLong(f(a));
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// plan(ctx_len, new_len, page_tokens, block_table, free_pages, free_head, free_next, cu_new, kv_len, positions, slots, work, stream)
PyObject* plan(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, [](Args& a) {
    a.count(13);
    a.device = a.tensor(0, "ctx_len").get_device();
    const int64_t reqs = THPVariable_Unpack(a.v[0]).numel();
    const auto t = a.table(3, reqs);
    const int64_t tokens = a.tensor(10, "slots").numel();
    size_t bytes;
    void* w = a.work(11, bytes);
    const int32_t *ctx = a.i32(0, "ctx_len", reqs), *fresh = a.i32(1, "new_len", reqs), *free_pages = a.i32(4, "free_pages"),
                  *head = a.i32(5, "free_head", 1);
    int32_t *next = a.i32(6, "free_next", 1), *cu = a.i32(7, "cu_new", reqs + 1), *len = a.i32(8, "kv_len", reqs),
            *pos = a.i32(9, "positions", tokens), *slots = a.i32(10, "slots", tokens);
    const int64_t n_free = THPVariable_Unpack(a.v[4]).numel();
    if (n_free > UINT32_MAX || tokens > UINT32_MAX || reqs > UINT32_MAX) throw std::invalid_argument("a buffer is too long");
    const uint64_t pt = a.u(2);
    if (pt > 1024) return (int)SHN_ERR_INVALID_ARG;
    const On on(a, 12);
    return shn_kv_plan(ctx, fresh, (uint32_t)reqs, (uint32_t)pt, t.p, t.width, free_pages, (uint32_t)n_free, head, next, cu, len, pos, slots,
                       (uint32_t)tokens, w, bytes, on.stream);
  });
}

// store(cache, device, q, k, v, positions, slots, q_out, work, q_weight, k_weight, eps, cos_sin, pairs, stream)
PyObject* store(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, [](Args& a) {
    a.count(15);
    const shn_kv_cache* c = a.cache(0);
    const int64_t d = c->head_dim;
    const auto k = a.rows(3, "k", d, c->kv_heads);
    const auto x = a.rows(4, "v", d, c->kv_heads, k.tokens);
    Args::Rows q = {nullptr, 0, 0, 0}, o = {nullptr, 0, 0, 0};
    if (!a.none(2)) {
      q = a.rows(2, "q", d, -1, k.tokens);
      o = a.rows(7, "q_out", d, q.heads, k.tokens);
    }
    const int32_t *pos = a.none(5) ? nullptr : a.i32(5, "positions", k.tokens), *slots = a.i32(6, "slots", k.tokens);
    size_t bytes;
    void* w = a.work(8, bytes);
    const uint16_t* wq = a.none(9) ? nullptr : static_cast<uint16_t*>(a.dev(9, "q_weight", at::kBFloat16, d));
    const uint16_t* wk = a.none(10) ? nullptr : static_cast<uint16_t*>(a.dev(10, "k_weight", at::kBFloat16, d));
    const float* cs = nullptr;
    int64_t n_pos = 0, rot = 0;
    if (!a.none(12)) {
      const Tensor& t = a.tensor(12, "cos_sin");
      if (t.dim() != 2) throw std::invalid_argument("cos_sin must be [positions, rot_dim]");
      cs = static_cast<float*>(a.dev(12, "cos_sin", at::kFloat));
      n_pos = t.size(0), rot = t.size(1);
    }
    if (k.tokens > UINT32_MAX || n_pos > UINT32_MAX || rot > UINT32_MAX || q.heads > UINT32_MAX) throw std::invalid_argument("a tensor is too long");
    const int pairs = PyObject_IsTrue(a.v[13]);
    if (pairs < 0) {
      PyErr_Clear();
      throw std::invalid_argument("pairs must be true or false");
    }
    const On on(a, 14);
    return shn_kv_store(q.p, q.stride, (uint32_t)q.heads, k.p, k.stride, x.p, x.stride, (uint32_t)k.tokens, pos, slots, wq, wk, a.f(11), cs,
                        (uint32_t)n_pos, (uint32_t)rot, (uint32_t)pairs, c, o.p, o.stride, w, bytes, on.stream);
  });
}

// load(cache, device, slots, k_out, v_out, work, stream)
PyObject* load(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, [](Args& a) {
    a.count(7);
    const shn_kv_cache* c = a.cache(0);
    const int32_t* slots = a.i32(2, "slots");
    const int64_t tokens = THPVariable_Unpack(a.v[2]).numel();
    Args::Rows k = {nullptr, 0, 0, 0}, x = {nullptr, 0, 0, 0};
    if (!a.none(3)) k = a.rows(3, "k_out", c->head_dim, c->kv_heads, tokens);
    if (!a.none(4)) x = a.rows(4, "v_out", c->head_dim, c->kv_heads, tokens);
    size_t bytes;
    void* w = a.work(5, bytes);
    if (tokens > UINT32_MAX) throw std::invalid_argument("a tensor is too long");
    const On on(a, 6);
    return shn_kv_load(c, slots, (uint32_t)tokens, k.p, k.stride, x.p, x.stride, w, bytes, on.stream);
  });
}

struct Attn {
  Args::Rows q, o;
  Args::Table t;
  int32_t* len;
  int64_t reqs;
};
// q at 2, block_table, kv_len and out at the places given
Attn attention(Args& a, const shn_kv_cache* c, int table, int kv_len, int out) {
  Attn x;
  x.q = a.rows(2, "q", c->head_dim);
  x.o = a.rows(out, "out", c->head_dim, x.q.heads, x.q.tokens);
  x.len = a.i32(kv_len, "kv_len");
  x.reqs = THPVariable_Unpack(a.v[kv_len]).numel();
  x.t = a.table(table, x.reqs);
  if (x.q.tokens > UINT32_MAX || x.q.heads > UINT32_MAX || x.reqs > UINT32_MAX) throw std::invalid_argument("a tensor is too long");
  return x;
}

// attn_prompt(cache, device, q, block_table, cu_q, kv_len, scale, out, work, stream)
PyObject* attn_prompt(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, [](Args& a) {
    a.count(10);
    const shn_kv_cache* c = a.cache(0);
    const Attn x = attention(a, c, 3, 5, 7);
    const int32_t* cu = a.i32(4, "cu_q", x.reqs + 1);
    size_t bytes;
    void* w = a.work(8, bytes);
    const On on(a, 9);
    return shn_kv_attn_prompt(x.q.p, x.q.stride, (uint32_t)x.q.tokens, (uint32_t)x.q.heads, c, x.t.p, x.t.width, cu, x.len, (uint32_t)x.reqs, a.f(6),
                              x.o.p, x.o.stride, w, bytes, on.stream);
  });
}

// attn_shared(cache, device, q, prefix_pages, prefix_len, block_table, kv_len, scale, out, work, stream)
PyObject* attn_shared(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, [](Args& a) {
    a.count(11);
    const shn_kv_cache* c = a.cache(0);
    const Attn x = attention(a, c, 5, 6, 8);
    if (x.q.tokens != x.reqs)
      throw std::invalid_argument("q has " + std::to_string(x.q.tokens) + " queries for " + std::to_string(x.reqs) + " requests");
    const int32_t* pages = a.none(3) ? nullptr : a.i32(3, "prefix_pages");
    const int64_t n_pages = a.none(3) ? 0 : THPVariable_Unpack(a.v[3]).numel();
    if (n_pages > UINT32_MAX) throw std::invalid_argument("a tensor is too long");
    const int32_t* plen = a.i32(4, "prefix_len", 1);
    size_t bytes;
    void* w = a.work(9, bytes);
    const On on(a, 10);
    return shn_kv_attn_shared(x.q.p, x.q.stride, (uint32_t)x.reqs, (uint32_t)x.q.heads, c, pages, (uint32_t)n_pages, plen, x.t.p, x.t.width, x.len,
                              a.f(7), x.o.p, x.o.stride, w, bytes, on.stream);
  });
}

PyMethodDef kMethods[] = {
    {"plan", (PyCFunction)(void (*)(void))plan, METH_FASTCALL, nullptr},
    {"store", (PyCFunction)(void (*)(void))store, METH_FASTCALL, nullptr},
    {"load", (PyCFunction)(void (*)(void))load, METH_FASTCALL, nullptr},
    {"attn_prompt", (PyCFunction)(void (*)(void))attn_prompt, METH_FASTCALL, nullptr},
    {"attn_shared", (PyCFunction)(void (*)(void))attn_shared, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kv", "Tensor checks and marshalling of the paged KV cache calls.", -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__kv(void) { return PyModule_Create(&kModule); }
