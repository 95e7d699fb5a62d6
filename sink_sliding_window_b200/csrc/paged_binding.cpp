// Python binding of the paged-cache calls (include/sink_attn.h).
//
// Argument marshalling only, like the ctypes binding of the other calls: torch
// CUDA tensors are checked, results are allocated, and the C-ABI entry points
// do the work on the current stream of the tensors' device.  A serving step
// makes these calls once per layer beside kernels of a few microseconds, which
// a call through ctypes took longer than (planning 18 us, append 12 us).
//
// A function returns its results, or the status (an int) of a call that the
// library refused; tensors that do not fit the call raise ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "sink_attn.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

constexpr int64_t kAny = -1;  // any length
constexpr int kHeadDim = 64;

std::string text(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + (v[i] == kAny ? std::string("any") : std::to_string(v[i]));
  return s + ")";
}

[[noreturn]] void refuse(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int device,
                         bool strides) {
  const std::string n = name;
  if (!t.is_cuda()) throw Refused(n + ": expected a CUDA tensor, got one on " + t.device().str());
  if (t.get_device() != device)
    throw Refused(n + " is on " + t.device().str() + ", the call's other tensors are on cuda:" + std::to_string(device));
  if (t.scalar_type() != type)
    throw Refused(n + ": expected " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  bool same = t.dim() == static_cast<int64_t>(shape.size());
  for (size_t i = 0; same && i < shape.size(); ++i) same = shape[i] == kAny || shape[i] == t.size(i);
  if (!same) throw Refused(n + ": expected shape " + text(shape) + ", got " + text(t.sizes()));
  if (!strides && !t.is_contiguous()) throw Refused(n + " is not contiguous");
  throw Refused(n + ": not a tensor of this call");
}

// A tensor of one type, shape and device; dense, unless strides are the call's to give.
void check(const Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, int device,
           bool strides = false) {
  bool fine = t.is_cuda() && t.get_device() == device && t.scalar_type() == type &&
              t.dim() == static_cast<int64_t>(shape.size()) && (strides || t.is_contiguous());
  int i = 0;
  for (int64_t n : shape) {
    if (!fine) break;
    fine = n == kAny || n == t.size(i);
    ++i;
  }
  if (!fine) refuse(t, name, type, at::IntArrayRef(shape.begin(), shape.size()), device, strides);
}

// The stride of a dimension; of one with a single element, which no address
// needs, any multiple of a row.
int64_t stride_of(const Tensor& t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : kHeadDim; }

// bf16 [T][heads][64] whose tokens are contiguous; returns the token stride.
int64_t check_heads(const Tensor& t, const char* name, int64_t tokens, int64_t heads, int device) {
  check(t, name, at::kBFloat16, {tokens, heads, kHeadDim}, device, true);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != kHeadDim))
    throw Refused(std::string(name) + ": the heads of a token are not contiguous");
  return stride_of(t, 0);
}

int as_int(int64_t v, const char* name) {
  if (v < INT_MIN || v > INT_MAX) throw Refused(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

// One call's arguments.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) throw Refused("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
  }
  bool none(int i) const { return a_[i] == Py_None; }
  const Tensor& tensor(int i, const char* name) const {
    if (!THPVariable_Check(a_[i])) throw Refused(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(a_[i]);
  }
  int64_t integer(int i, const char* name) const {
    const long long v = PyLong_AsLongLong(a_[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused(std::string(name) + ": expected a whole number");
    }
    return v;
  }
  double real(int i, const char* name) const {
    const double v = PyFloat_AsDouble(a_[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused(std::string(name) + ": expected a number");
    }
    return v;
  }
  PyObject* object(int i) const { return a_[i]; }

 private:
  PyObject* const* a_;
};

struct Cache {
  bool codes;
  int device;
  int64_t pages, page, heads;
  const Tensor *k, *v;
  const float *k_scale, *v_scale;
};

Cache cache_of(const Args& a, int k, int v, int ks, int vs) {
  Cache c;
  c.k = &a.tensor(k, "k_cache");
  c.v = &a.tensor(v, "v_cache");
  const at::ScalarType type = c.k->scalar_type();
  c.codes = type == at::kByte || type == at::kFloat8_e4m3fn;
  if (!c.codes && type != at::kBFloat16)
    throw Refused(std::string("k_cache: expected bfloat16, float8_e4m3fn or uint8 codes, got ") + c10::toString(type));
  c.device = c.k->is_cuda() ? c.k->get_device() : -1;
  check(*c.k, "k_cache", type, {kAny, kAny, kAny, kHeadDim}, c.device, true);
  c.pages = c.k->size(0), c.page = c.k->size(1), c.heads = c.k->size(2);
  check(*c.v, "v_cache", type, {c.pages, c.page, c.heads, kHeadDim}, c.device, true);
  bool same = c.k->stride(3) == 1 && c.v->stride(3) == 1;
  for (int i = 0; i < 3; ++i) same = same && stride_of(*c.k, i) == stride_of(*c.v, i);
  if (!same)
    throw Refused("k_cache and v_cache need the same strides, with contiguous rows");
  c.k_scale = c.v_scale = nullptr;
  if (c.codes) {
    if (a.none(ks) || a.none(vs)) throw Refused("an e4m3 cache needs k_scale and v_scale");
    check(a.tensor(ks, "k_scale"), "k_scale", at::kFloat, {c.heads}, c.device);
    check(a.tensor(vs, "v_scale"), "v_scale", at::kFloat, {c.heads}, c.device);
    c.k_scale = a.tensor(ks, "k_scale").const_data_ptr<float>();
    c.v_scale = a.tensor(vs, "v_scale").const_data_ptr<float>();
  } else if (!a.none(ks) || !a.none(vs)) {
    throw Refused("a bf16 cache takes no scales");
  }
  return c;
}

void fill(sink_attn_paged_dims* d, const Cache& c) {
  d->num_kv_heads = as_int(c.heads, "key/value heads");
  d->head_dim = kHeadDim;
  d->page_size = as_int(c.page, "page_size");
  d->num_pages = as_int(c.pages, "num_pages");
  d->page_stride = stride_of(*c.k, 0);
  d->token_stride = stride_of(*c.k, 1);
  d->head_stride = stride_of(*c.k, 2);
}

// Frees the interpreter for other threads, and takes it back however the scope
// is left: an exception is turned into Python's by code that needs it.
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  Released() = default;
  Released(const Released&) = delete;
  ~Released() { PyEval_RestoreThread(state); }
};

// The C call, with the interpreter free for other threads.  What can be refused
// (an address of a tensor without memory, a number out of range) is worked out
// before it.
template <typename F>
sink_attn_status run(F&& f) {
  const Released released;
  return f();
}

int* ints(const Tensor& t) { return t.data_ptr<int>(); }

// (cached_lens, new_lens, block_table, free_pages, pool, page_size, max_tokens,
// window, first_page, cu_seqlens, kv_lens, slot_map, pool_out, first_page_out)
PyObject* plan(const Args& a) {
  const Tensor& cached = a.tensor(0, "cached_lens");
  const int dev = cached.is_cuda() ? cached.get_device() : -1;
  const int64_t B = cached.numel();
  check(cached, "cached_lens", at::kInt, {B}, dev);
  const Tensor &fresh = a.tensor(1, "new_lens"), &table = a.tensor(2, "block_table"), &ring = a.tensor(3, "free_pages"),
               &pool = a.tensor(4, "pool");
  check(fresh, "new_lens", at::kInt, {B}, dev);
  check(table, "block_table", at::kInt, {B, kAny}, dev);
  check(ring, "free_pages", at::kInt, {kAny}, dev);
  check(pool, "pool", at::kInt, {2}, dev);
  const int64_t max_tokens = a.integer(6, "max_tokens");
  const int window = as_int(a.integer(7, "window"), "window");
  const bool has_first = !a.none(8);
  if (has_first)
    check(a.tensor(8, "first_page"), "first_page", at::kInt, {B}, dev);
  else if (window > 0 || !a.none(13))
    throw Refused("giving back a window's pages needs first_page");
  if (max_tokens < 0) throw Refused("max_tokens is negative");
  sink_attn_plan_dims d;
  d.batch = as_int(B, "requests");
  d.max_tokens = as_int(max_tokens, "max_tokens");
  d.max_pages = as_int(table.size(1), "max_pages");
  d.page_size = as_int(a.integer(5, "page_size"), "page_size");
  d.num_pages = as_int(ring.numel(), "num_pages");
  const int *const cached_p = ints(cached), *const fresh_p = ints(fresh), *const pool_p = ints(pool);
  int *const table_p = ints(table), *const ring_p = ints(ring);
  const int* const first_p = has_first ? ints(a.tensor(8, "first_page")) : nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  static const char* const names[5] = {"cu_seqlens", "kv_lens", "slot_map", "pool_out", "first_page_out"};
  const int64_t sizes[5] = {B + 1, B, max_tokens, 2, B};
  Tensor out[5];
  const int outs = has_first ? 5 : 4;
  for (int i = 0; i < outs; ++i) {
    if (a.none(9 + i)) {
      out[i] = at::empty({sizes[i]}, cached.options());
    } else {
      out[i] = a.tensor(9 + i, names[i]);
      check(out[i], names[i], at::kInt, {sizes[i]}, dev);
    }
  }
  if (B == 0) {
    out[0].zero_();
    out[2].fill_(-1);
    out[3].copy_(pool);
  } else {
    void* const stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    int* to[5] = {};
    for (int i = 0; i < outs; ++i) to[i] = ints(out[i]);
    const sink_attn_status st = run([&] {
      return sink_attn_paged_plan(&d, cached_p, fresh_p, table_p, ring_p, pool_p, first_p, window, to[0], to[1], to[2],
                                  to[3], to[4], stream);
    });
    if (st != SINK_ATTN_OK) return PyLong_FromLong(st);
  }
  PyObject* r = PyTuple_New(5);
  if (!r) return nullptr;
  for (int i = 0; i < 5; ++i) {
    PyObject* o = i < outs ? THPVariable_Wrap(std::move(out[i])) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// (k_new, v_new, slot_map, k_cache, v_cache, k_scale, v_scale)
PyObject* append(const Args& a) {
  const Cache c = cache_of(a, 3, 4, 5, 6);
  const Tensor &k = a.tensor(0, "k_new"), &v = a.tensor(1, "v_new"), &slots = a.tensor(2, "slot_map");
  const int64_t ks = check_heads(k, "k_new", kAny, c.heads, c.device);
  const int64_t T = k.size(0);
  const int64_t vs = check_heads(v, "v_new", T, c.heads, c.device);
  check(slots, "slot_map", at::kInt, {T}, c.device);
  sink_attn_paged_dims d = {};
  d.total_tokens = as_int(T, "tokens");
  fill(&d, c);
  const void *const k_p = k.data_ptr(), *const v_p = v.data_ptr();
  const int* const slots_p = ints(slots);
  void *const kc_p = c.k->data_ptr(), *const vc_p = c.v->data_ptr();
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
  void* const stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  const sink_attn_status st = run([&] {
    return c.codes ? sink_attn_paged_append_e4m3(&d, k_p, v_p, ks, vs, slots_p, kc_p, vc_p, c.k_scale, c.v_scale, stream)
                   : sink_attn_paged_append(&d, k_p, v_p, ks, vs, slots_p, kc_p, vc_p, stream);
  });
  if (st != SINK_ATTN_OK) return PyLong_FromLong(st);
  return PyTuple_Pack(2, a.object(3), a.object(4));
}

// (q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, sinks, window, scale,
// max_new, k_scale, v_scale, out, lse, workspace)
PyObject* attn(const Args& a) {
  const Cache c = cache_of(a, 1, 2, 10, 11);
  const Tensor &q = a.tensor(0, "q"), &table = a.tensor(3, "block_table"), &cu = a.tensor(4, "cu_seqlens"),
               &lens = a.tensor(5, "kv_lens"), &sinks = a.tensor(6, "sinks");
  const int64_t qs = check_heads(q, "q", kAny, q.dim() == 3 ? q.size(1) : kAny, c.device);
  const int64_t T = q.size(0), Hq = q.size(1), B = lens.numel();
  check(table, "block_table", at::kInt, {B, kAny}, c.device);
  check(cu, "cu_seqlens", at::kInt, {B + 1}, c.device);
  check(lens, "kv_lens", at::kInt, {B}, c.device);
  check(sinks, "sinks", at::kFloat, {Hq}, c.device);
  const int window = as_int(a.integer(7, "window"), "window");
  const float scale = a.none(8) ? 0.125f : static_cast<float>(a.real(8, "scale"));
  sink_attn_paged_dims d = {};
  d.batch = as_int(B, "requests");
  d.total_tokens = as_int(T, "tokens");
  d.max_new = a.none(9) ? std::max(d.total_tokens, 1) : as_int(a.integer(9, "max_new"), "max_new");
  d.num_q_heads = as_int(Hq, "query heads");
  d.max_pages = as_int(table.size(1), "max_pages");
  d.q_stride = qs;
  fill(&d, c);
  const void *const q_p = q.data_ptr(), *const kc_p = c.k->data_ptr(), *const vc_p = c.v->data_ptr();
  const int *const table_p = ints(table), *const cu_p = ints(cu), *const lens_p = ints(lens);
  const float* const sinks_p = sinks.data_ptr<float>();
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
  Tensor out, lse, ws;
  if (a.none(12)) {
    out = at::empty({T, Hq, kHeadDim}, q.options());
  } else {
    out = a.tensor(12, "out");
    check(out, "out", at::kBFloat16, {T, Hq, kHeadDim}, c.device);
  }
  if (a.none(13)) {
    lse = at::empty({Hq, T}, sinks.options());
  } else {
    lse = a.tensor(13, "lse");
    check(lse, "lse", at::kFloat, {Hq, T}, c.device);
  }
  if (a.none(14)) {
    ws = at::empty({static_cast<int64_t>(sink_attn_paged_workspace_size(&d) / 4 + 1)}, sinks.options());
  } else {
    ws = a.tensor(14, "workspace");
    if (!ws.is_cuda() || ws.get_device() != c.device || !ws.is_contiguous())
      throw Refused("workspace: expected a contiguous tensor on cuda:" + std::to_string(c.device) + ", got one on " +
                    ws.device().str());
  }
  void* const stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  void *const out_p = out.data_ptr(), *const ws_p = ws.data_ptr();
  float* const lse_p = lse.data_ptr<float>();
  const size_t ws_bytes = ws.nbytes();
  const sink_attn_status st = run([&] {
    return c.codes ? sink_attn_paged_attn_e4m3(&d, q_p, kc_p, vc_p, table_p, cu_p, lens_p, c.k_scale, c.v_scale, sinks_p,
                                               window, scale, out_p, lse_p, ws_p, ws_bytes, stream)
                   : sink_attn_paged_attn(&d, q_p, kc_p, vc_p, table_p, cu_p, lens_p, sinks_p, window, scale, out_p,
                                          lse_p, ws_p, ws_bytes, stream);
  });
  if (st != SINK_ATTN_OK) return PyLong_FromLong(st);
  PyObject* o = a.none(12) ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a.object(12));
  PyObject* l = a.none(13) ? THPVariable_Wrap(std::move(lse)) : Py_NewRef(a.object(13));
  PyObject* r = o && l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(l);
  return r;
}

template <PyObject* (*kCall)(const Args&), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return kCall(Args(args, n, kArgs));
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*kCall)(const Args&), int kArgs>
PyCFunction function() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<kCall, kArgs>));
}

PyMethodDef kMethods[] = {
    {"plan", function<plan, 14>(), METH_FASTCALL, "sink_attn_paged_plan"},
    {"append", function<append, 7>(), METH_FASTCALL, "sink_attn_paged_append, _e4m3"},
    {"attn", function<attn, 15>(), METH_FASTCALL, "sink_attn_paged_attn, _e4m3"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", "Binding of the paged-cache calls.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&kModule); }
