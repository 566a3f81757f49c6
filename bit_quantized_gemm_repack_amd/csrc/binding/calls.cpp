// The short calls of the binding, natively: their outputs' allocation, checks
// and launch from one C function each.  Through ctypes a call with two outputs
// costs the host 6.8 us (3 of them the allocations in Python, 2.4 the launch),
// through this 4.6, where the kernels take 2 to 4.
//
// Each function takes the ordinary call: contiguous tensors of the right types
// and sizes on the current device.  It returns None for any other and after any
// error, and the Python function behind it then checks and calls again, with its
// messages.  Other Python threads run while it allocates and launches, which wait
// where memory or the launch queue is full (as ctypes lets them).  The library's entry points come in by address (bind), so nothing
// here links to it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "hq.h"

namespace {

decltype(&hq_quantize_blocks) quantize_fn;
decltype(&hq_route_topk) route_fn;
decltype(&hq_gemm) gemm_fn;
decltype(&hq_plan_workspace_bytes) workspace_fn;
decltype(&hq_rms_norm) norm_fn;
decltype(&hq_route_experts) route_experts_fn;

const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.is_contiguous() ? &t : nullptr;
}

bool current(const at::Tensor& t) { return t.device().index() == c10::hip::current_device(); }

void* stream(const at::Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

// 16-bit types as the library counts them, or -1.
int act_type(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? HQ_BF16 : (t.scalar_type() == at::kHalf ? HQ_F16 : -1);
}

PyObject* pair(at::Tensor a, at::Tensor b) {
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(a)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(b)));
  return r;
}

// Python's lock given up for a scope, for what may wait and touches no Python object.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// f(), or None where it throws (an allocation that fails).
template <typename F>
PyObject* guarded(F&& f) {
  try {
    if (PyObject* r = f()) return r;
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// quantize_blocks(x, silu_mul)
PyObject* quantize_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* x = n == 2 ? tensor(a[0]) : nullptr;
    if (!x || x->dim() != 2 || act_type(*x) < 0 || !current(*x)) return nullptr;
    const int silu = PyObject_IsTrue(a[1]);
    const int64_t m = x->size(0), k = silu ? x->size(1) / 2 : x->size(1);
    if (silu < 0 || k % 128 || (silu && x->size(1) % 2)) return nullptr;
    at::Tensor codes, scales;
    {
      const Unlocked unlocked;
      codes = at::empty({m, k}, x->options().dtype(at::kByte));
      scales = at::empty({k / 128, m}, x->options().dtype(at::kFloat));
      if (quantize_fn(m, k, (hq_dtype)act_type(*x), silu, x->data_ptr(), codes.data_ptr(), static_cast<float*>(scales.data_ptr()),
                      stream(*x)) != HQ_OK)
        return nullptr;
    }
    return pair(std::move(codes), std::move(scales));
  });
}

// route_topk(logits, topk, renormalize)
PyObject* route_topk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* x = n == 3 && PyLong_Check(a[1]) ? tensor(a[0]) : nullptr;
    if (!x || x->dim() != 2 || !current(*x)) return nullptr;
    const int type = x->scalar_type() == at::kFloat ? HQ_F32 : act_type(*x);
    const int64_t t = x->size(0), topk = PyLong_AsLongLong(a[1]);
    const int renorm = PyObject_IsTrue(a[2]);
    if (type < 0 || topk < 1 || topk > 64 || x->size(1) > 1024 || renorm < 0) return nullptr;
    at::Tensor ids, w;
    {
      const Unlocked unlocked;
      ids = at::empty({t, topk}, x->options().dtype(at::kInt));
      w = at::empty({t, topk}, x->options().dtype(at::kFloat));
      if (route_fn(t, (int)x->size(1), (int)topk, (hq_dtype)type, x->data_ptr(), renorm, static_cast<int32_t*>(ids.data_ptr()),
                   static_cast<float*>(w.data_ptr()), stream(*x)) != HQ_OK)
        return nullptr;
    }
    return pair(std::move(ids), std::move(w));
  });
}

// Rows [m, k] of x's type and device, contiguous inside; the step from one to the next (of one
// row it says nothing).
const at::Tensor* rows(PyObject* o, const at::Tensor* like) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1)) return nullptr;
  if (like && (t.device() != like->device() || t.scalar_type() != like->scalar_type() || t.sizes() != like->sizes())) return nullptr;
  return &t;
}
int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// rms_norm(x, weight, eps, residual or None, kind, residual_out or None)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* x = n == 6 && PyFloat_Check(a[2]) && PyLong_Check(a[4]) ? rows(a[0], nullptr) : nullptr;
    if (!x || act_type(*x) < 0 || !current(*x)) return nullptr;
    const int64_t m = x->size(0), k = x->size(1);
    const at::Tensor* w = tensor(a[1]);
    if (!w || w->dim() != 1 || w->size(0) != k || w->device() != x->device() ||
        (w->scalar_type() != x->scalar_type() && w->scalar_type() != at::kFloat))
      return nullptr;
    const bool add = a[3] != Py_None, given = a[5] != Py_None;
    const at::Tensor* res = add ? rows(a[3], x) : nullptr;
    const at::Tensor* into = given ? rows(a[5], x) : nullptr;
    if ((add && !res) || (given && (!into || !add))) return nullptr;
    const auto kind = (hq_norm_kind)PyLong_AsLong(a[4]);
    const float eps = (float)PyFloat_AS_DOUBLE(a[2]);
    const bool blocks = kind == HQ_NORM_FP8_BLOCK || kind == HQ_NORM_MXFP4;
    if (kind < HQ_NORM_SAME || kind > HQ_NORM_MXFP4 || (blocks && k % 128)) return nullptr;
    at::Tensor h, y, scale;
    {
      const Unlocked unlocked;
      if (add) h = given ? *into : at::empty({m, k}, x->options());
      if (kind == HQ_NORM_SAME)
        y = at::empty({m, k}, x->options());
      else
        y = at::empty({m, kind == HQ_NORM_MXFP4 ? k / 2 : k}, x->options().dtype(kind == HQ_NORM_INT8 ? at::kChar : at::kByte));
      if (kind == HQ_NORM_MXFP4)
        scale = at::empty({k / 128, m, 4}, x->options().dtype(at::kByte));
      else if (blocks)
        scale = at::empty({k / 128, m}, x->options().dtype(at::kFloat));
      else if (kind != HQ_NORM_SAME)
        scale = at::empty({m}, x->options().dtype(at::kFloat));
      const auto type = (hq_dtype)act_type(*x);
      if (norm_fn(m, k, type, x->data_ptr(), row_stride(*x), add ? res->data_ptr() : nullptr, add ? row_stride(*res) : 0,
                  w->scalar_type() == at::kFloat ? HQ_F32 : type, w->data_ptr(), eps, kind, add ? h.data_ptr() : nullptr,
                  add ? row_stride(h) : 0, y.data_ptr(), scale.defined() ? scale.data_ptr() : nullptr, stream(*x)) != HQ_OK)
        return nullptr;
    }
    if (!add) return scale.defined() ? pair(std::move(y), std::move(scale)) : THPVariable_Wrap(std::move(y));
    if (!scale.defined()) return pair(std::move(y), std::move(h));
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(y)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(scale)));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(h)));
    return r;
  });
}

// route_experts(logits, topk, bias or None, scoring, groups, group_topk, group_best, renormalize, scale)
PyObject* route_experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* x = n == 9 ? tensor(a[0]) : nullptr;
    if (!x || x->dim() != 2 || !current(*x) || !PyFloat_Check(a[8])) return nullptr;
    for (int i : {1, 3, 4, 5, 6})
      if (!PyLong_Check(a[i])) return nullptr;
    const int type = x->scalar_type() == at::kFloat ? HQ_F32 : act_type(*x);
    const int64_t t = x->size(0), experts = x->size(1), topk = PyLong_AsLongLong(a[1]);
    int64_t v[4];
    for (int i = 0; i < 4; ++i) {
      v[i] = PyLong_AsLongLong(a[3 + i]);
      if (v[i] < 0 || v[i] > 1024) return nullptr;
    }
    const int renorm = PyObject_IsTrue(a[7]);
    if (type < 0 || topk < 1 || topk > 64 || experts > 1024 || renorm < 0) return nullptr;
    const at::Tensor* bias = a[2] != Py_None ? tensor(a[2]) : nullptr;
    if (a[2] != Py_None && (!bias || bias->device() != x->device() || bias->scalar_type() != at::kFloat || bias->dim() != 1 || bias->size(0) != experts))
      return nullptr;
    at::Tensor ids, w;
    {
      const Unlocked unlocked;
      ids = at::empty({t, topk}, x->options().dtype(at::kInt));
      w = at::empty({t, topk}, x->options().dtype(at::kFloat));
      if (route_experts_fn(t, (int)experts, (int)topk, (hq_dtype)type, x->data_ptr(), (hq_score)v[0],
                           bias ? static_cast<const float*>(bias->data_ptr()) : nullptr, (int)v[1], (int)v[2], (int)v[3], renorm,
                           (float)PyFloat_AS_DOUBLE(a[8]), static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(w.data_ptr()),
                           stream(*x)) != HQ_OK)
        return nullptr;
    }
    return pair(std::move(ids), std::move(w));
  });
}

// gemm_block(plan, n, k, bf16, a, a_scale, w, meta): a w8a8_block GEMM with its
// output and workspace
PyObject* gemm_block(PyObject*, PyObject* const* v, Py_ssize_t count) {
  return guarded([&]() -> PyObject* {
    if (count != 8) return nullptr;
    const auto* plan = static_cast<const hq_plan*>(PyLong_AsVoidPtr(v[0]));
    const int64_t n = PyLong_AsLongLong(v[1]), k = PyLong_AsLongLong(v[2]);
    const at::Tensor *a = tensor(v[4]), *s = tensor(v[5]), *w = tensor(v[6]), *meta = tensor(v[7]);
    if (!plan || n < 1 || k < 128 || !a || !s || !w || !meta || !current(*a)) return nullptr;
    if (s->device() != a->device() || w->device() != a->device() || meta->device() != a->device()) return nullptr;
    const auto type = a->scalar_type();
    if (type != at::kByte && type != at::kFloat8_e4m3fn && type != at::kChar) return nullptr;
    if (a->dim() != 2 || a->size(1) != k) return nullptr;
    const int64_t m = a->size(0);
    if (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != k / 128 || s->size(1) != m) return nullptr;
    if ((int64_t)w->nbytes() < n * k || (int64_t)meta->nbytes() < (n + 127) / 128 * (k / 128) * 4) return nullptr;
    const auto out_type = PyObject_IsTrue(v[3]) ? at::kBFloat16 : at::kHalf;
    at::Tensor out, ws;
    {
      const Unlocked unlocked;
      size_t need = 0;
      if (workspace_fn(plan, m, &need) != HQ_OK) return nullptr;
      out = at::empty({m, n}, a->options().dtype(out_type));
      if (need) ws = at::empty({(int64_t)need}, a->options().dtype(at::kByte));
      if (gemm_fn(plan, m, a->data_ptr(), s->data_ptr(), w->data_ptr(), meta->data_ptr(), out.data_ptr(),
                  need ? ws.data_ptr() : nullptr, need, stream(*a)) != HQ_OK)
        return nullptr;
    }
    return THPVariable_Wrap(std::move(out));
  });
}

// bind(addresses of hq_quantize_blocks, hq_route_topk, hq_gemm, hq_plan_workspace_bytes)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  quantize_fn = reinterpret_cast<decltype(quantize_fn)>(PyLong_AsVoidPtr(a[0]));
  route_fn = reinterpret_cast<decltype(route_fn)>(PyLong_AsVoidPtr(a[1]));
  gemm_fn = reinterpret_cast<decltype(gemm_fn)>(PyLong_AsVoidPtr(a[2]));
  workspace_fn = reinterpret_cast<decltype(workspace_fn)>(PyLong_AsVoidPtr(a[3]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// bind_norm_route(addresses of hq_rms_norm, hq_route_experts)
PyObject* bind_norm_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "bind_norm_route takes two addresses");
    return nullptr;
  }
  norm_fn = reinterpret_cast<decltype(norm_fn)>(PyLong_AsVoidPtr(a[0]));
  route_experts_fn = reinterpret_cast<decltype(route_experts_fn)>(PyLong_AsVoidPtr(a[1]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"bind_norm_route", fast(bind_norm_route), METH_FASTCALL, nullptr},
                         {"quantize_blocks", fast(quantize_blocks), METH_FASTCALL, nullptr},
                         {"route_topk", fast(route_topk), METH_FASTCALL, nullptr},
                         {"rms_norm", fast(rms_norm), METH_FASTCALL, nullptr},
                         {"route_experts", fast(route_experts), METH_FASTCALL, nullptr},
                         {"gemm_block", fast(gemm_block), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  // the torch whose headers this was compiled with; the binding uses it with no other
  if (m && PyModule_AddStringConstant(m, "built_for", HQ_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
