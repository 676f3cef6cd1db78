// sg_attn_torch.cpp -- the calls of attention.py on torch tensors, in one step each:
// checks, outputs, the C ABI (include/scaled_attention.h).
//
// A decode step of a small batch runs in 5 to 10 us on the GPU; the same marshalling in Python
// took 12 to 20 us a call, most of it for outputs, the stream and the checks.  Nothing is
// computed here.  Every entry catches C++ exceptions and raises them in Python.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <exception>
#include <string>

#include "scaled_attention.h"

namespace {

PyObject* g_status_error = nullptr;  // raised with (status, call)

struct Plan {
  sg_attn_t handle;
  int64_t q_heads, kv_heads, dim, page;
  int device;
  sg_rotary_t rotary;
};

struct Cache {
  sg_kv_cache_t args;
  int64_t heads, page, dim;
  int device;
};

constexpr const char* kPlan = "sg_attn plan";
constexpr const char* kCache = "sg_attn cache";

struct BadArgument {
  std::string what;
};

template <typename T>
void free_capsule(PyObject* c) {
  delete static_cast<T*>(PyCapsule_GetPointer(c, PyCapsule_GetName(c)));
}

// Runs f; what it throws becomes a Python exception.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const BadArgument& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw BadArgument{std::string(what) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

bool on(const at::Tensor& t, int device) { return t.is_cuda() && t.device().index() == device; }

struct Rows {
  const void* data;
  int64_t n, stride;
};

// q, k or v: bfloat16 [tokens, heads, dim], heads next to each other.
Rows rows(PyObject* o, int64_t heads, const Plan& p, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 3 || t.scalar_type() != at::kBFloat16 || !on(t, p.device))
    throw BadArgument{std::string(what) + " must be a bfloat16 [tokens, heads, dim] tensor on the plan's device"};
  const auto size = t.sizes(), step = t.strides();
  if (size[1] != heads || size[2] != p.dim || step[2] != 1 || (heads > 1 && step[1] != p.dim))
    throw BadArgument{std::string(what) + " must be [tokens, " + std::to_string(heads) + ", " + std::to_string(p.dim) +
                      "] with its heads next to each other"};
  return {t.data_ptr(), size[0], size[0] > 1 ? step[0] : heads * p.dim};
}

const int32_t* ints(PyObject* o, int64_t n, const Plan& p, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !on(t, p.device) || !t.is_contiguous())
    throw BadArgument{std::string(what) + " must be a contiguous int32 [" + std::to_string(n) + "] tensor on the plan's device"};
  return static_cast<const int32_t*>(t.data_ptr());
}

int64_t length(PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 1) throw BadArgument{std::string(what) + " must have one dimension"};
  return t.size(0);
}

const int32_t* table(PyObject* o, int64_t batch, const Plan& p, int64_t* width) {
  const at::Tensor& t = tensor(o, "block_table");
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != batch || !on(t, p.device) || !t.is_contiguous())
    throw BadArgument{"block_table must be a contiguous int32 [" + std::to_string(batch) + ", pages] tensor on the plan's device"};
  *width = t.size(1);
  return static_cast<const int32_t*>(t.data_ptr());
}

// The stream that a call runs on; torch's current one, and whether the two differ.
struct Streams {
  sg_stream_t handle;
  c10::cuda::CUDAStream current;
  bool side;
};

Streams streams(PyObject* o, const Plan& p) {
  const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(p.device));
  const sg_stream_t now = current.stream();
  if (o == Py_None) return {now, current, false};
  const auto s = static_cast<sg_stream_t>(PyLong_AsVoidPtr(o));
  if (PyErr_Occurred()) throw BadArgument{"stream"};
  return {s, current, s != now};
}

// An output that the caller has, or a new one.  On a stream of the caller's choice a new one is that stream's memory, so
// whoever used it before or gets it next is ordered there; and it is recorded on the current stream, where results are
// read as a rule, so that dropping it does not give it away before the reads so far.
at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const Plan& p, const Streams& s, const char* what) {
  if (o == Py_None) {
    const auto options = at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(p.device)));
    if (!s.side) return at::empty(shape, options);
    const c10::cuda::CUDAStreamGuard guard(
        c10::cuda::getStreamFromExternal(s.handle, static_cast<c10::DeviceIndex>(p.device)));
    const at::Tensor t = at::empty(shape, options);
    t.record_stream(s.current.unwrap());
    return t;
  }
  const at::Tensor& t = tensor(o, what);
  if (t.sizes() != shape || t.scalar_type() != type || !on(t, p.device) || !t.is_contiguous())
    throw BadArgument{std::string(what) + " must be a contiguous tensor of the result's shape and type on the plan's device"};
  return t;
}

const Plan& plan(PyObject* o) {
  auto* p = static_cast<Plan*>(PyCapsule_GetPointer(o, kPlan));
  if (!p) throw BadArgument{"not a plan"};
  return *p;
}

const sg_kv_cache_t* cache(PyObject* o, const Plan& p) {
  auto* c = static_cast<Cache*>(PyCapsule_GetPointer(o, kCache));
  if (!c) throw BadArgument{"not a cache"};
  if (c->heads != p.kv_heads || c->page != p.page || c->dim != p.dim || c->device != p.device)
    throw BadArgument{"the cache's layout differs from the plan's"};
  return &c->args;
}

int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw BadArgument{"number"};
  return v;
}

float scale_or(PyObject* o, const Plan& p) {
  const double v = o == Py_None ? 1.0 / std::sqrt(static_cast<double>(p.dim)) : PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw BadArgument{"scale"};
  return static_cast<float>(v);
}

void check(sg_status_t s, const char* call) {
  if (s == SG_OK) return;
  PyObject* e = g_status_error ? PyObject_CallFunction(g_status_error, "is", static_cast<int>(s), call) : nullptr;
  if (e) {
    PyErr_SetObject(g_status_error, e);
    Py_DECREF(e);
  }
  throw BadArgument{call};
}

void arity(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) throw BadArgument{"expected " + std::to_string(want) + " arguments"};
}

PyObject* pair(const at::Tensor& a, PyObject* b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* t = x && b ? PyTuple_Pack(2, x, b) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(b);
  return t;
}

// set_error(type)
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_status_error);
  g_status_error = type;
  Py_RETURN_NONE;
}

// plan(handle, q_heads, kv_heads, dim, page, device, rotary pointer, max_pos, rot, interleaved)
PyObject* make_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 10);
    int64_t v[10];
    for (int i = 0; i < 10; ++i) v[i] = number(a[i]);
    auto* p = new Plan{reinterpret_cast<sg_attn_t>(v[0]), v[1], v[2], v[3], v[4], static_cast<int>(v[5]),
                       {reinterpret_cast<const float*>(v[6]), v[7], static_cast<int32_t>(v[8]), static_cast<int32_t>(v[9])}};
    return PyCapsule_New(p, kPlan, free_capsule<Plan>);
  });
}

// cache(k, v, k_scale, v_scale pointers, num_pages, k and v page strides, heads, page, dim, device)
PyObject* make_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 11);
    int64_t v[11];
    for (int i = 0; i < 11; ++i) v[i] = number(a[i]);
    auto* c = new Cache{{reinterpret_cast<void*>(v[0]), reinterpret_cast<void*>(v[1]), reinterpret_cast<uint8_t*>(v[2]),
                         reinterpret_cast<uint8_t*>(v[3]), v[4], v[5], v[6]},
                        v[7], v[8], v[9], static_cast<int>(v[10])};
    return PyCapsule_New(c, kCache, free_capsule<Cache>);
  });
}

// append(plan, q, k, v, cache, block_table, ctx_lens, cu_seqlens, k_out, q_out, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 11);
    const Plan& p = plan(a[0]);
    const Rows q = rows(a[1], p.q_heads, p, "q"), k = rows(a[2], p.kv_heads, p, "k"), v = rows(a[3], p.kv_heads, p, "v");
    if (k.n != q.n || v.n != q.n) throw BadArgument{"q, k and v must have the same number of rows"};
    const sg_kv_cache_t* c = cache(a[4], p);
    const int64_t batch = length(a[6], "ctx_lens");
    int64_t width;
    const int32_t* t = table(a[5], batch, p, &width);
    const int32_t* ctx = ints(a[6], batch, p, "ctx_lens");
    const int32_t* cu = ints(a[7], batch + 1, p, "cu_seqlens");
    const Streams s = streams(a[10], p);
    const at::Tensor q_out = output(a[9], {q.n, p.q_heads, p.dim}, at::kBFloat16, p, s, "q_out");
    at::Tensor k_out;
    if (a[8] == Py_True || (a[8] != Py_None && a[8] != Py_False))
      k_out = output(a[8] == Py_True ? Py_None : a[8], {q.n, p.kv_heads, p.dim}, at::kBFloat16, p, s, "k_out");
    check(scaled_attn_append(p.handle, c, &p.rotary, q.data, q.stride, k.data, k.stride, v.data, v.stride, t, width, ctx, cu,
                             q.n, batch, q_out.data_ptr(), k_out.defined() ? k_out.data_ptr() : nullptr, s.handle),
          "scaled_attn_append");
    PyObject* second = Py_None;
    if (k_out.defined())
      second = THPVariable_Wrap(k_out);
    else
      Py_INCREF(second);
    return pair(q_out, second);
  });
}

// decode(plan, q, cache, block_table, kv_lens, q_tokens, scale, out, lse, stream)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 10);
    const Plan& p = plan(a[0]);
    const Rows q = rows(a[1], p.q_heads, p, "q");
    const sg_kv_cache_t* c = cache(a[2], p);
    const int64_t batch = length(a[4], "kv_lens"), qn = number(a[5]);
    if (qn < 0 || q.n != batch * qn)
      throw BadArgument{"q must have q_tokens = " + std::to_string(qn) + " rows for each of " + std::to_string(batch) + " sequences"};
    int64_t width;
    const int32_t* t = table(a[3], batch, p, &width);
    const int32_t* lens = ints(a[4], batch, p, "kv_lens");
    const float scale = scale_or(a[6], p);
    const Streams s = streams(a[9], p);
    const at::Tensor out = output(a[7], {q.n, p.q_heads, p.dim}, at::kBFloat16, p, s, "out");
    const at::Tensor lse = output(a[8], {q.n, p.q_heads}, at::kFloat, p, s, "lse");
    check(scaled_attn_decode(p.handle, c, q.data, q.stride, qn, t, width, lens, batch, scale, out.data_ptr(),
                             static_cast<float*>(lse.data_ptr()), s.handle),
          "scaled_attn_decode");
    return pair(out, THPVariable_Wrap(lse));
  });
}

// prompt(plan, q, k, v, cu_q, cu_k, causal, scale, out, lse, stream)
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 11);
    const Plan& p = plan(a[0]);
    const Rows q = rows(a[1], p.q_heads, p, "q"), k = rows(a[2], p.kv_heads, p, "k"), v = rows(a[3], p.kv_heads, p, "v");
    if (k.n != v.n) throw BadArgument{"k and v must have the same number of rows"};
    const int64_t batch = length(a[4], "cu_q") - 1;
    const int32_t* cu_q = ints(a[4], batch + 1, p, "cu_q");
    const int32_t* cu_k = a[5] == Py_None ? cu_q : ints(a[5], batch + 1, p, "cu_k");
    const int causal = PyObject_IsTrue(a[6]);
    if (causal < 0) throw BadArgument{"causal"};
    const float scale = scale_or(a[7], p);
    const Streams s = streams(a[10], p);
    const at::Tensor out = output(a[8], {q.n, p.q_heads, p.dim}, at::kBFloat16, p, s, "out");
    const at::Tensor lse = output(a[9], {q.n, p.q_heads}, at::kFloat, p, s, "lse");
    check(scaled_attn_prompt(p.handle, q.data, q.stride, k.data, k.stride, v.data, v.stride, cu_q, cu_k, q.n, k.n, batch, causal,
                             scale, out.data_ptr(), static_cast<float*>(lse.data_ptr()), s.handle),
          "scaled_attn_prompt");
    return pair(out, THPVariable_Wrap(lse));
  });
}

PyMethodDef g_methods[] = {
    {"set_error", set_error, METH_O, nullptr},
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(make_plan)), METH_FASTCALL, nullptr},
    {"cache", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(make_cache)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"prompt", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prompt)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn() { return PyModule_Create(&g_module); }
