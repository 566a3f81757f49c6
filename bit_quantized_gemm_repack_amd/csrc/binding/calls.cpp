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

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"quantize_blocks", fast(quantize_blocks), METH_FASTCALL, nullptr},
                         {"route_topk", fast(route_topk), METH_FASTCALL, nullptr},
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
