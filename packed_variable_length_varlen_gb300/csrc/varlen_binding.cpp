// varlen_binding.cpp -- the short way from Python into the entry points around a
// step of the paged attention: reads the tensors' types, shapes and places,
// allocates what the call returns and calls the C function, without going through
// Python attributes and ctypes for each of them.
//
// A small call is the host's.  A step of 16 rows, one call after another, through
// ctypes and through this: rotary_cache_write 15.9 -> 4.9 us (its kernel 2.5),
// cache_plan 5.5 -> 3.4 (3.1), cache_move and cache_trim 12.0 -> 6.3, tree attention
// of 52 rows 27 -> 14.7 (its kernels 14.6).  Everything here is a shortcut for calls that are as usual: where
// anything is not (a wrong type or shape, another device than the current one, a
// stream of the caller's own), a function returns NotImplemented before it has done
// anything, and varlen_attn.py goes its own way, which also words the refusals.  A
// status other than VARLEN_OK is returned as a number.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <vector>

#include "varlen_attn.h"

namespace {

// The library's functions, as the process has loaded it (bind).
struct Entries {
  decltype(&varlen_attn_rotary) rotary;
  decltype(&varlen_attn_rotary_cache_write) write;
  decltype(&varlen_attn_cache_plan) plan;
  decltype(&varlen_attn_cache_trim) trim;
  decltype(&varlen_attn_cache_move) move;
  decltype(&varlen_attn_fwd_paged_tree) tree;
  decltype(&varlen_attn_fwd_paged_workspace_size) workspace;
} g_entry = {};

using Args = PyObject* const*;

struct Refuse {};  // the call is not as usual

int64_t number(PyObject* o) {
  if (!PyLong_Check(o)) throw Refuse();
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refuse();
  }
  return v;
}

void* address(PyObject* o) { return o == Py_None ? nullptr : reinterpret_cast<void*>(static_cast<uintptr_t>(number(o))); }

// A handle's `at`: the address of its C description, which the caller keeps, and its device's index.
template <class T>
struct Handle {
  const T* at;
  int64_t dev;
  explicit Handle(PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) throw Refuse();
    at = static_cast<const T*>(address(PyTuple_GET_ITEM(o, 0)));
    dev = number(PyTuple_GET_ITEM(o, 1));
  }
};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refuse();
  return THPVariable_Unpack(o);
}

bool on(const at::Tensor& t, int64_t dev) { return t.is_cuda() && t.get_device() == dev; }

// Packed rows [rows, heads, dim] (heads < 0: any number).
const at::Tensor& rows_of(PyObject* o, int64_t dev, int64_t rows, int64_t heads, int64_t dim) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 3 || t.scalar_type() != at::kBFloat16 || t.size(0) != rows || t.size(2) != dim || t.stride(2) != 1 ||
      (heads >= 0 && t.size(1) != heads) || t.size(1) > INT32_MAX || !on(t, dev))
    throw Refuse();
  return t;
}

void* list_of(PyObject* o, int64_t dev, int64_t n, at::ScalarType type) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 1 || t.size(0) != n || t.scalar_type() != type || !t.is_contiguous() || !on(t, dev)) throw Refuse();
  return t.data_ptr();
}
void* list_or_null(PyObject* o, int64_t dev, int64_t n, at::ScalarType type) {
  return o == Py_None ? nullptr : list_of(o, dev, n, type);
}

varlen_stride strides(const at::Tensor& t) { return varlen_stride{t.stride(0), t.stride(1)}; }

at::Tensor fresh(const at::Tensor& like, at::IntArrayRef sizes, at::ScalarType type) {
  return at::empty(sizes, like.options().dtype(type).requires_grad(false));
}

// The current stream of device `dev`, which has to be the current one.
void* stream_of(int64_t dev) {
  if (dev < 0 || c10::cuda::current_device() != dev) throw Refuse();
  return static_cast<void*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

int32_t in32(int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) throw Refuse();
  return static_cast<int32_t>(v);
}

template <class F>
PyObject* answer(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refuse&) {
    Py_RETURN_NOTIMPLEMENTED;
  }
  END_HANDLE_TH_ERRORS
}

// Calls an entry point without the interpreter's lock.
template <class F, class... A>
int call(F entry, A... args) {
  PyThreadState* state = PyEval_SaveThread();
  const int st = entry(args...);
  PyEval_RestoreThread(state);
  return st;
}

PyObject* status(int st) { return PyLong_FromLong(st); }

PyObject* wrapped(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = wrapped(a);
  PyObject* y = wrapped(b);
  PyObject* both = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
}

// rotary(rope, inverse, q, k or None, positions or None, cu or None, q_out or None, k_out or None): (q_out, k_out)
PyObject* rotary(PyObject*, Args a, Py_ssize_t n) {
  return answer([&]() -> PyObject* {
    if (n != 8) throw Refuse();
    const Handle<varlen_rotary> rope(a[0]);
    const int64_t dev = rope.dev;
    void* stream = stream_of(dev);
    const at::Tensor& first = tensor(a[2]);
    if (first.dim() != 3) throw Refuse();
    const int64_t total = in32(first.size(0)), dim = in32(first.size(2));
    const at::Tensor& q = rows_of(a[2], dev, total, -1, dim);
    const bool has_k = a[3] != Py_None;
    const at::Tensor& k = has_k ? rows_of(a[3], dev, total, -1, dim) : q;
    const auto* pos = static_cast<const int32_t*>(list_or_null(a[4], dev, total, at::kInt));
    const int32_t* cu = nullptr;
    int64_t batch = 0;
    if (pos == nullptr) {
      batch = tensor(a[5]).numel() - 1;
      cu = static_cast<const int32_t*>(list_of(a[5], dev, batch + 1, at::kInt));
    }
    const at::Tensor qo = a[6] == Py_None ? fresh(q, q.sizes(), at::kBFloat16) : rows_of(a[6], dev, total, q.size(1), dim);
    at::Tensor ko;
    if (has_k) ko = a[7] == Py_None ? fresh(k, k.sizes(), at::kBFloat16) : rows_of(a[7], dev, total, k.size(1), dim);
    const varlen_stride none{0, 0};
    const int st = call(g_entry.rotary, static_cast<const void*>(q.data_ptr()), strides(q),
                        static_cast<const void*>(has_k ? k.data_ptr() : nullptr), has_k ? strides(k) : none, pos, cu, in32(batch),
                        in32(total), in32(q.size(1)), has_k ? in32(k.size(1)) : 0, (int32_t)dim, rope.at, in32(number(a[1])),
                        qo.data_ptr(), strides(qo), has_k ? ko.data_ptr() : nullptr, has_k ? strides(ko) : none, stream);
    if (st != VARLEN_OK) return status(st);
    return pair(qo, ko);
  });
}

// rotary_cache_write(cache, q or None, k, v, rope, positions, slots, q_out or None): q_out or None
PyObject* rotary_cache_write(PyObject*, Args a, Py_ssize_t n) {
  return answer([&]() -> PyObject* {
    if (n != 8) throw Refuse();
    const Handle<varlen_kv_cache> cache(a[0]);
    const Handle<varlen_rotary> rope(a[4]);
    const int64_t dev = cache.dev;
    void* stream = stream_of(dev);
    if (rope.dev != dev) throw Refuse();
    const at::Tensor& first = tensor(a[2]);
    if (first.dim() != 3) throw Refuse();
    const int64_t total = in32(first.size(0)), dim = cache.at->head_dim;
    const at::Tensor& k = rows_of(a[2], dev, total, cache.at->num_kv_heads, dim);
    const at::Tensor& v = rows_of(a[3], dev, total, cache.at->num_kv_heads, dim);
    const bool has_q = a[1] != Py_None;
    const at::Tensor& q = has_q ? rows_of(a[1], dev, total, -1, dim) : k;
    const auto* pos = static_cast<const int32_t*>(list_of(a[5], dev, total, at::kInt));
    const auto* slots = static_cast<const int64_t*>(list_of(a[6], dev, total, at::kLong));
    at::Tensor qo;
    if (has_q) qo = a[7] == Py_None ? fresh(q, q.sizes(), at::kBFloat16) : rows_of(a[7], dev, total, q.size(1), dim);
    const varlen_stride none{0, 0};
    const int st = call(g_entry.write, static_cast<const void*>(has_q ? q.data_ptr() : nullptr), has_q ? strides(q) : none,
                        static_cast<const void*>(k.data_ptr()), strides(k), static_cast<const void*>(v.data_ptr()), strides(v), pos,
                        slots, in32(total), has_q ? in32(q.size(1)) : 0, cache.at, rope.at,
                        has_q ? qo.data_ptr() : nullptr, has_q ? strides(qo) : none, stream);
    if (st != VARLEN_OK) return status(st);
    return wrapped(qo);
  });
}

// cache_plan(pool, batch, new_lens, parents or None, total, StepPlan.args): status
PyObject* cache_plan(PyObject*, Args a, Py_ssize_t n) {
  return answer([&]() -> PyObject* {
    if (n != 6 || !PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 8) throw Refuse();
    const Handle<varlen_page_pool> pool(a[0]);
    const int64_t batch = number(a[1]), total = number(a[4]);
    void* stream = stream_of(pool.dev);
    auto arg = [&](int i) { return PyTuple_GET_ITEM(a[5], i); };
    return status(call(g_entry.plan, pool.at, static_cast<const int32_t*>(list_of(a[2], pool.dev, batch, at::kInt)), in32(batch),
                       static_cast<const int32_t*>(list_or_null(a[3], pool.dev, total, at::kInt)), in32(total),
                       static_cast<int32_t*>(address(arg(0))), static_cast<int64_t*>(address(arg(1))),
                       static_cast<int32_t*>(address(arg(2))), static_cast<int32_t*>(address(arg(3))),
                       static_cast<uint32_t*>(address(arg(4))), in32(number(arg(5))), address(arg(6)),
                       static_cast<size_t>(number(arg(7))), stream));
  });
}

// cache_trim(pool, batch, lens, cu or None): status
PyObject* cache_trim(PyObject*, Args a, Py_ssize_t n) {
  return answer([&]() -> PyObject* {
    if (n != 4) throw Refuse();
    const Handle<varlen_page_pool> pool(a[0]);
    const int64_t batch = number(a[1]);
    void* stream = stream_of(pool.dev);
    return status(call(g_entry.trim, pool.at, static_cast<const int32_t*>(list_of(a[2], pool.dev, batch, at::kInt)),
                       static_cast<const int32_t*>(list_or_null(a[3], pool.dev, batch + 1, at::kInt)), in32(batch), stream));
  });
}

// cache_move([cache, ...], batch, cu, kept, kept_lens): status
PyObject* cache_move(PyObject*, Args a, Py_ssize_t n) {
  return answer([&]() -> PyObject* {
    if (n != 5 || !PyList_Check(a[0]) || PyList_GET_SIZE(a[0]) < 1) throw Refuse();
    const Py_ssize_t count = PyList_GET_SIZE(a[0]);
    const int64_t dev = Handle<varlen_kv_cache>(PyList_GET_ITEM(a[0], 0)).dev;
    void* stream = stream_of(dev);
    std::vector<varlen_kv_cache> caches;
    caches.reserve(static_cast<size_t>(count));
    for (Py_ssize_t i = 0; i < count; ++i) {
      const Handle<varlen_kv_cache> cache(PyList_GET_ITEM(a[0], i));
      if (cache.dev != dev) throw Refuse();
      caches.push_back(*cache.at);
    }
    const int64_t batch = number(a[1]);
    const at::Tensor& kept = tensor(a[3]);
    if (kept.dim() != 2 || kept.scalar_type() != at::kInt || kept.size(0) != batch || !on(kept, dev) ||
        (kept.size(1) > 1 && kept.stride(1) != 1))
      throw Refuse();
    return status(call(g_entry.move, static_cast<const varlen_kv_cache*>(caches.data()), in32(count),
                       static_cast<const int32_t*>(list_of(a[2], dev, batch + 1, at::kInt)), in32(batch), INT32_MAX,
                       static_cast<const int32_t*>(kept.data_ptr()), kept.stride(0),
                       static_cast<const int32_t*>(list_of(a[4], dev, batch, at::kInt)), in32(kept.size(1)), stream));
  });
}

// attention_fwd_paged_tree(cache, batch, q, cu, masks, max_seqlen_q, scale or None, window_left, positions or None): (out, lse)
PyObject* attention_fwd_paged_tree(PyObject*, Args a, Py_ssize_t n) {
  return answer([&]() -> PyObject* {
    if (n != 9) throw Refuse();
    const Handle<varlen_kv_cache> cache(a[0]);
    const int64_t dev = cache.dev, batch = number(a[1]);
    void* stream = stream_of(dev);
    const at::Tensor& first = tensor(a[2]);
    if (first.dim() != 3) throw Refuse();
    const int64_t total = in32(first.size(0));
    const int32_t dim = cache.at->head_dim;
    const at::Tensor& q = rows_of(a[2], dev, total, -1, dim);
    const int32_t heads = in32(q.size(1));
    const auto* cu = static_cast<const int32_t*>(list_of(a[3], dev, batch + 1, at::kInt));
    const at::Tensor& masks = tensor(a[4]);
    if (masks.dim() != 2 || masks.scalar_type() != at::kInt || masks.size(0) != total || !masks.is_contiguous() || !on(masks, dev))
      throw Refuse();
    if (a[6] != Py_None && !PyFloat_Check(a[6])) throw Refuse();
    const double scale = a[6] == Py_None ? std::pow(static_cast<double>(dim), -0.5) : PyFloat_AS_DOUBLE(a[6]);
    const auto* pos = static_cast<const int32_t*>(list_or_null(a[8], dev, total, at::kInt));
    const int32_t most = in32(number(a[5])), left = in32(std::max<int64_t>(number(a[7]), -1));
    const size_t bytes = g_entry.workspace(in32(batch), in32(total), heads, cache.at->num_kv_heads, dim);
    const at::Tensor out = fresh(q, q.sizes(), at::kBFloat16), lse = fresh(q, {heads, total}, at::kFloat);
    const at::Tensor ws = fresh(q, {static_cast<int64_t>(bytes)}, at::kByte);
    const int st = call(g_entry.tree, static_cast<const void*>(q.data_ptr()), strides(q), cu, in32(batch), in32(total), heads, most,
                        cache.at, static_cast<float>(scale), static_cast<const uint32_t*>(masks.data_ptr()), in32(masks.size(1)), pos,
                        left, out.data_ptr(), strides(out), static_cast<float*>(lse.data_ptr()), ws.data_ptr(), bytes, stream);
    return st != VARLEN_OK ? status(st) : pair(out, lse);
  });
}

// bind(addresses of the library's functions, in the order of Entries)
PyObject* bind(PyObject*, Args a, Py_ssize_t n) {
  return answer([&]() -> PyObject* {
    if (n != 7) throw Refuse();
    auto take = [&](auto& f, int i) { f = reinterpret_cast<std::decay_t<decltype(f)>>(static_cast<uintptr_t>(number(a[i]))); };
    take(g_entry.rotary, 0);
    take(g_entry.write, 1);
    take(g_entry.plan, 2);
    take(g_entry.trim, 3);
    take(g_entry.move, 4);
    take(g_entry.tree, 5);
    take(g_entry.workspace, 6);
    Py_RETURN_NONE;
  });
}

#define VARLEN_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {VARLEN_METHOD(bind),       VARLEN_METHOD(rotary),     VARLEN_METHOD(rotary_cache_write),
                           VARLEN_METHOD(cache_plan), VARLEN_METHOD(cache_trim), VARLEN_METHOD(cache_move),
                           VARLEN_METHOD(attention_fwd_paged_tree), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_varlen_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__varlen_binding() { return PyModule_Create(&g_module); }
