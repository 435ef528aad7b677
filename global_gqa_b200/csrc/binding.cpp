// The quick way into the paged-cache calls from Python.
//
// A decode step makes several of these calls per layer, each a few microseconds
// on the GPU; through ctypes the checks of a call's tensors, its outputs and the
// conversion of its arguments take 10 to 20 us of host time, here about 5.  Each
// function checks what the Python wrappers check and makes the library call on
// the device's current stream; whatever is not as expected (a wrong type, shape
// or place, another current device, a refusal by the library) returns None, and
// the wrapper takes its ordinary way, which words the error.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "../../include/g3attn.h"

namespace {

constexpr int kMaxDevices = 64;
PyObject* g_status[kMaxDevices] = {};  // error words of each device's calls (owned references), set by the wrapper

using at::kBFloat16;
using at::kChar;
using at::kFloat;
using at::kInt;

const at::Tensor* tensor_of(PyObject* o, int64_t dims) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.dim() == dims ? &t : nullptr;
}

// One call's tensors: everything on one GPU, which is the current one.
struct Call {
  bool ok = true;
  int dev = -1;

  void on(const at::Tensor* t) {
    ok = ok && t != nullptr && t->is_cuda();
    if (!ok) return;
    dev = t->device().index();
    ok = dev >= 0 && dev < kMaxDevices && c10::cuda::current_device() == dev;
  }
  void* ptr(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (!ok) return nullptr;
    const at::Tensor* t = tensor_of(o, (int64_t)shape.size());
    ok = t != nullptr && t->scalar_type() == type && t->is_cuda() && t->device().index() == dev && t->is_contiguous() &&
         t->sizes().equals(at::IntArrayRef(shape));
    return ok ? t->data_ptr() : nullptr;
  }
  int32_t* status(PyObject* o) {
    if (ok && o == Py_None) o = g_status[dev];
    if (o == nullptr) ok = false;  // not made yet
    return static_cast<int32_t*>(ptr(o, kInt, {2}));
  }
  int32_t number(PyObject* o) {
    if (!ok) return 0;
    const long v = PyLong_AsLong(o);
    if ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX) {
      PyErr_Clear();
      ok = false;
    }
    return (int32_t)v;
  }
  float real(PyObject* o) {
    if (!ok) return 0.f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)v;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
  at::Tensor empty(std::initializer_list<int64_t> shape, at::ScalarType type) const {
    return at::detail::empty_cuda(at::IntArrayRef(shape), type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
  }
};

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "%zd arguments instead of %zd", n, want);
  try {
    return body();
  } catch (const std::exception& e) {  // out of memory: as torch would say it
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (old_lens, new_lens, block_table, free_pages, free_state, page_size, n_pages, max_tokens, status)
PyObject* page_map(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor *old = tensor_of(a[0], 1), *table = tensor_of(a[2], 2), *ring = tensor_of(a[3], 1);
    Call c;
    c.on(old);
    if (!c.ok || table == nullptr || ring == nullptr) Py_RETURN_NONE;
    const int64_t B = old->size(0), pages = table->size(1), cap = ring->size(0);
    void *po = c.ptr(a[0], kInt, {B}), *pn = c.ptr(a[1], kInt, {B}), *pt = c.ptr(a[2], kInt, {B, pages}),
         *pf = c.ptr(a[3], kInt, {cap}), *ps = c.ptr(a[4], kInt, {2});
    const int32_t P = c.number(a[5]), n_pages = c.number(a[6]), T = c.number(a[7]);
    int32_t* status = c.status(a[8]);
    if (!c.ok || T < 1 || B > INT32_MAX || pages > INT32_MAX || cap > INT32_MAX) Py_RETURN_NONE;
    // One allocation of tensors that share its storage, on 256-byte boundaries; a second one (0.6 of 6 us of host time)
    // for the token rows where there are many, so that kept lengths do not keep a prompt's rows alive.
    const int64_t sizes[5] = {B, B + 1, T, T, 2};
    const int apart = T > 8192 ? 1 : 0;
    const int in[5] = {0, 0, apart, apart, 0};
    int64_t total[2] = {0, 0}, begin[5];
    for (int i = 0; i < 5; ++i) {
      begin[i] = total[in[i]];
      total[in[i]] += (sizes[i] + 63) / 64 * 64;
    }
    at::Tensor all[2];
    for (int k = 0; k <= apart; ++k) all[k] = c.empty({total[k]}, kInt);
    at::Tensor out[5];
    for (int i = 0; i < 5; ++i) {
      const at::Tensor& t = all[in[i]];
      out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
      out[i].unsafeGetTensorImpl()->set_storage_offset(begin[i]);
      out[i].unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(&sizes[i], 1));
    }
    auto i32 = [](void* p) { return static_cast<int32_t*>(p); };
    auto o32 = [&](int i) { return static_cast<int32_t*>(out[i].data_ptr()); };
    if (g3attn_page_map(i32(po), i32(pn), (int32_t)B, i32(pt), (int32_t)pages, i32(pf), (int32_t)cap, i32(ps), P, n_pages, T,
                        o32(0), o32(1), o32(2), o32(3), o32(4), status, c.stream()) != G3_OK)
      Py_RETURN_NONE;
    static PyObject* const names[5] = {PyUnicode_InternFromString("seq_lens"), PyUnicode_InternFromString("cu_tokens"),
                                       PyUnicode_InternFromString("slots"), PyUnicode_InternFromString("positions"),
                                       PyUnicode_InternFromString("free_state")};
    PyObject* d = PyDict_New();
    for (int i = 0; d != nullptr && i < 5; ++i) {
      PyObject* t = THPVariable_Wrap(out[i]);
      if (t == nullptr || PyDict_SetItem(d, names[i], t) != 0) Py_CLEAR(d);
      Py_XDECREF(t);
    }
    return d;
  });
}

// (k, v, k_gamma, positions, slots, k_pages, v_pages, rope_base, interp_factor, q, q_gamma, status): q_hat, or True without q
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor *k = tensor_of(a[0], 3), *pool = tensor_of(a[5], 4), *q = a[9] == Py_None ? nullptr : tensor_of(a[9], 3);
    Call c;
    c.on(k);
    if (!c.ok || pool == nullptr || (a[9] == Py_None) != (q == nullptr) || (q == nullptr && a[10] != Py_None)) Py_RETURN_NONE;
    const int64_t T = k->size(0), Hkv = k->size(1), D = k->size(2), n_pages = pool->size(0), P = pool->size(2);
    const int64_t Hq = q == nullptr ? 0 : q->size(1);
    void *pk = c.ptr(a[0], kBFloat16, {T, Hkv, D}), *pv = c.ptr(a[1], kBFloat16, {T, Hkv, D}), *pg = c.ptr(a[2], kFloat, {D}),
         *pp = c.ptr(a[3], kInt, {T}), *ps = c.ptr(a[4], kInt, {T}), *kp = c.ptr(a[5], kBFloat16, {n_pages, Hkv, P, D}),
         *vp = c.ptr(a[6], kBFloat16, {n_pages, Hkv, P, D});
    const float base = c.real(a[7]), interp = c.real(a[8]);
    void *pq = nullptr, *qg = nullptr;
    if (q != nullptr) {
      pq = c.ptr(a[9], kBFloat16, {T, Hq, D});
      qg = c.ptr(a[10], kFloat, {D});
    }
    int32_t* status = c.status(a[11]);
    if (!c.ok || T > INT32_MAX || n_pages > INT32_MAX) Py_RETURN_NONE;
    at::Tensor q_hat;
    if (q != nullptr) q_hat = c.empty({T, Hq, D}, kBFloat16);
    if (g3attn_paged_append(pq, pk, pv, static_cast<float*>(qg), static_cast<float*>(pg), static_cast<int32_t*>(pp),
                            static_cast<int32_t*>(ps), kp, vp, (int32_t)n_pages, (int32_t)P, base, interp, (int32_t)T, (int32_t)Hq,
                            (int32_t)Hkv, (int32_t)D, q != nullptr ? q_hat.data_ptr() : nullptr, status, c.stream()) != G3_OK)
      Py_RETURN_NONE;
    if (q == nullptr) Py_RETURN_TRUE;
    return THPVariable_Wrap(q_hat);
  });
}

// (k_pages, block_table, old_lens, seq_lens, bounds, exps, status): True
PyObject* page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor *pool = tensor_of(a[0], 4), *table = tensor_of(a[1], 2);
    Call c;
    c.on(pool);
    if (!c.ok || table == nullptr) Py_RETURN_NONE;
    const int64_t n_pages = pool->size(0), Hkv = pool->size(1), P = pool->size(2), D = pool->size(3);
    const int64_t B = table->size(0), pages = table->size(1);
    void *kp = c.ptr(a[0], kBFloat16, {n_pages, Hkv, P, D}), *pt = c.ptr(a[1], kInt, {B, pages}), *po = c.ptr(a[2], kInt, {B}),
         *pl = c.ptr(a[3], kInt, {B}), *pb = c.ptr(a[4], kChar, {n_pages, Hkv, 2, D}), *pe = c.ptr(a[5], kChar, {n_pages, Hkv});
    int32_t* status = c.status(a[6]);
    if (!c.ok || n_pages > INT32_MAX || B > INT32_MAX || pages > INT32_MAX) Py_RETURN_NONE;
    if (g3attn_page_bounds(kp, static_cast<int32_t*>(pt), static_cast<int32_t*>(po), static_cast<int32_t*>(pl), (int32_t)B,
                           (int32_t)pages, (int32_t)n_pages, (int32_t)P, (int32_t)Hkv, (int32_t)D, static_cast<int8_t*>(pb),
                           static_cast<int8_t*>(pe), status, c.stream()) != G3_OK)
      Py_RETURN_NONE;
    Py_RETURN_TRUE;
  });
}

// (q_hat, bounds, exps, block_table, seq_lens, page_size, n_select, status): pages
PyObject* page_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor *q = tensor_of(a[0], 3), *exps = tensor_of(a[2], 2), *table = tensor_of(a[3], 2);
    Call c;
    c.on(q);
    if (!c.ok || exps == nullptr || table == nullptr) Py_RETURN_NONE;
    const int64_t B = q->size(0), Hq = q->size(1), D = q->size(2), n_pages = exps->size(0), Hkv = exps->size(1), pages = table->size(1);
    void *pq = c.ptr(a[0], kBFloat16, {B, Hq, D}), *pb = c.ptr(a[1], kChar, {n_pages, Hkv, 2, D}), *pe = c.ptr(a[2], kChar, {n_pages, Hkv}),
         *pt = c.ptr(a[3], kInt, {B, pages}), *pl = c.ptr(a[4], kInt, {B});
    const int32_t P = c.number(a[5]), sel = c.number(a[6]);
    int32_t* status = c.status(a[7]);
    if (!c.ok || sel < 1 || n_pages > INT32_MAX || B > INT32_MAX || pages > INT32_MAX) Py_RETURN_NONE;
    const size_t ws_bytes = g3attn_page_select_workspace_size((int32_t)B, (int32_t)Hkv, (int32_t)pages);
    if (ws_bytes == 0) Py_RETURN_NONE;
    const at::Tensor out = c.empty({B, Hkv, sel}, kInt), ws = c.empty({(int64_t)ws_bytes}, at::kByte);
    if (g3attn_page_select(pq, static_cast<int8_t*>(pb), static_cast<int8_t*>(pe), static_cast<int32_t*>(pt), static_cast<int32_t*>(pl),
                           (int32_t)B, (int32_t)pages, (int32_t)n_pages, P, (int32_t)Hq, (int32_t)Hkv, (int32_t)D, sel,
                           static_cast<int32_t*>(out.data_ptr()), ws.data_ptr(), ws_bytes, status, c.stream()) != G3_OK)
      Py_RETURN_NONE;
    return THPVariable_Wrap(out);
  });
}

// (q_hat, k_pages, v_pages, block_table, seq_lens, layer_kind, window, pages, return_lse, status): out, or (out, lse)
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor *q = tensor_of(a[0], 3), *pool = tensor_of(a[1], 4), *table = tensor_of(a[3], 2);
    const at::Tensor* list = a[7] == Py_None ? nullptr : tensor_of(a[7], 3);
    Call c;
    c.on(q);
    if (!c.ok || pool == nullptr || table == nullptr || (a[7] == Py_None) != (list == nullptr)) Py_RETURN_NONE;
    const int64_t B = q->size(0), Hq = q->size(1), D = q->size(2), n_pages = pool->size(0), Hkv = pool->size(1), P = pool->size(2);
    const int64_t pages = table->size(1), sel = list == nullptr ? 0 : list->size(2);
    void *pq = c.ptr(a[0], kBFloat16, {B, Hq, D}), *kp = c.ptr(a[1], kBFloat16, {n_pages, Hkv, P, D}),
         *vp = c.ptr(a[2], kBFloat16, {n_pages, Hkv, P, D}), *pt = c.ptr(a[3], kInt, {B, pages}), *pl = c.ptr(a[4], kInt, {B});
    const int32_t kind = c.number(a[5]), window = c.number(a[6]);
    void* pp = list == nullptr ? nullptr : c.ptr(a[7], kInt, {B, Hkv, sel});
    int32_t* status = c.status(a[9]);
    if (!c.ok || n_pages > INT32_MAX || B > INT32_MAX || pages > INT32_MAX || sel > INT32_MAX || (list != nullptr && sel == 0))
      Py_RETURN_NONE;
    const size_t ws_bytes = g3attn_paged_decode_workspace_size((int32_t)D);
    if (ws_bytes == 0) Py_RETURN_NONE;
    const int with_lse = PyObject_IsTrue(a[8]);
    if (with_lse < 0) return nullptr;
    const at::Tensor out = c.empty({B, Hq, D}, kBFloat16), ws = c.empty({(int64_t)ws_bytes}, at::kByte);
    at::Tensor lse;
    if (with_lse) lse = c.empty({B, Hq}, kFloat);
    if (g3attn_paged_decode(pq, kp, vp, static_cast<int32_t*>(pt), static_cast<int32_t*>(pl), static_cast<int32_t*>(pp), (int32_t)sel,
                            static_cast<g3_layer_kind>(kind), window, (int32_t)B, (int32_t)pages, (int32_t)n_pages, (int32_t)P,
                            (int32_t)Hq, (int32_t)Hkv, (int32_t)D, out.data_ptr(), with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                            ws.data_ptr(), ws_bytes, status, c.stream()) != G3_OK)
      Py_RETURN_NONE;
    PyObject* o = THPVariable_Wrap(out);
    if (!with_lse || o == nullptr) return o;
    PyObject* l = THPVariable_Wrap(lse);
    PyObject* both = l == nullptr ? nullptr : PyTuple_Pack(2, o, l);
    Py_DECREF(o);
    Py_XDECREF(l);
    return both;
  });
}

// (device index, int32 [2] tensor): the error words used where a call is given none
PyObject* set_status(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    const long dev = PyLong_AsLong(a[0]);
    if (dev < 0 || dev >= kMaxDevices || !THPVariable_Check(a[1])) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a device index and its error words");
      return nullptr;
    }
    Py_INCREF(a[1]);
    Py_XSETREF(g_status[dev], a[1]);
    Py_RETURN_NONE;
  });
}

#define ENTRY(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {ENTRY(page_map),     ENTRY(paged_append), ENTRY(page_bounds),
                         ENTRY(page_select),  ENTRY(paged_decode), ENTRY(set_status), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
