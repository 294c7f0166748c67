// moe_ext.cpp -- the common call of each operator of gmm_moe.h from Python:
// arguments checked, outputs allocated and the C entry point called without a
// Python step in between (a dispatch call of a decode step takes 4 us on the
// GPU; marshalling it in Python takes longer than launching it).
//
// Every function takes what is plain -- dense device tensors of fitting rank
// and type, outputs to be made, the current stream -- and returns None for
// anything else, a refused call included: the caller (_moe.py) then goes the
// long way, which serves the other forms and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gmm_moe.h"

namespace {

constexpr int kDevices = 64;
gmm_handle* g_handles[kDevices];

struct Entry {
  decltype(&gmm_sort_tokens_workspace) sort_workspace;
  decltype(&gmm_sort_tokens_run) sort;
  decltype(&gmm_dispatch_run) dispatch;
  decltype(&gmm_combine_run) combine;
  decltype(&gmm_combine_grad_run) combine_grad;
  decltype(&gmm_quant_mxfp4_run) quant;
  decltype(&gmm_widen_mxfp4_run) widen;
} g_entry;

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return GMM_F32;
    case at::kBFloat16: return GMM_BF16;
    case at::kFloat8_e4m3fn: return GMM_F8E4M3FN;
    case at::kFloat8_e5m2: return GMM_F8E5M2;
    case at::kFloat8_e8m0fnu: return GMM_E8M0;
    case at::kInt: return GMM_I32;
    case at::kLong: return GMM_I64;
    case at::kChar: return GMM_I8;
    default: return -1;
  }
}

gmm_tensor view(const at::Tensor& t, int code) {
  gmm_tensor v{t.numel() ? t.const_data_ptr() : nullptr, code, (int32_t)t.dim(), {0, 0, 0, 0}};
  for (int i = 0; i < v.ndim; ++i) v.shape[i] = t.size(i);
  return v;
}

// Packed fp4 codes: two elements a byte.
gmm_tensor view_packed(const at::Tensor& t) {
  gmm_tensor v = view(t, GMM_F4E2M1);
  v.shape[v.ndim - 1] *= 2;
  return v;
}

// The arguments of one call, read before the interpreter lock is let go.
struct Args {
  PyObject* const* args;
  int dev = -1;
  gmm_handle* handle = nullptr;
  bool ok = true;

  // A dense tensor of rank `dim` on the first one's device.
  at::Tensor tensor(int i, int64_t dim) {
    if (!ok || !THPVariable_Check(args[i])) {
      ok = false;
      return {};
    }
    at::Tensor t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || t.layout() != at::kStrided || t.dim() != dim || !t.is_contiguous()) ok = false;
    if (ok && dev < 0) {
      dev = t.get_device();
      handle = dev < kDevices ? g_handles[dev] : nullptr;
    }
    if (ok && (t.get_device() != dev || !handle)) ok = false;
    return t;
  }
  long long number(int i) {
    const long long v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  void* pointer(int i) {
    void* const v = PyLong_AsVoidPtr(args[i]);
    if (!v && PyErr_Occurred()) ok = false;
    return v;
  }
};

// Lets other Python threads run while outputs are allocated and the call is
// queued (the allocator and the launch may have to wait for the device).
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

PyObject* none() { Py_RETURN_NONE; }
PyObject* give(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* give(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// Runs a function's body; what it throws (an allocation that fails) is left to
// the long way to meet again and report.
template <class Body>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Body body) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    PyObject* r = body();
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_XDECREF(r);
      return none();
    }
    return r;
  } catch (...) {
    PyErr_Clear();
    return none();
  }
}

// sort_tokens(expert_ids, groups, stream)
PyObject* sort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor ids = x.tensor(0, 2);
    const long long groups = x.number(1);
    void* const stream = x.pointer(2);
    if (!x.ok || (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong)) return none();
    size_t bytes = 0;
    if (g_entry.sort_workspace(ids.numel(), groups, &bytes) != GMM_OK) return none();
    at::Tensor sizes, slot_row;
    {
      Unlocked u;
      sizes = at::empty({groups}, ids.options().dtype(at::kInt));
      slot_row = at::empty(ids.sizes(), ids.options().dtype(at::kInt));
      at::Tensor work;
      if (bytes) work = at::empty({(int64_t)bytes}, ids.options().dtype(at::kByte));
      const gmm_tensor iv = view(ids, code_of(ids.scalar_type())), gv = view(sizes, GMM_I32), sv = view(slot_row, GMM_I32);
      if (g_entry.sort(x.handle, &iv, &gv, &sv, bytes ? work.mutable_data_ptr() : nullptr, bytes, stream)) x.ok = false;
    }
    return x.ok ? give(sizes, slot_row) : none();
  });
}

// dispatch(x, slot_row, stream)
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor t = x.tensor(0, 2), slots = x.tensor(1, 2);
    void* const stream = x.pointer(2);
    if (!x.ok) return none();
    // (bytes, packed fp4 codes among them, are only copied)
    const int code = t.scalar_type() == at::kByte ? GMM_I8 : code_of(t.scalar_type()), scode = code_of(slots.scalar_type());
    if (code < 0 || scode < 0) return none();
    at::Tensor out;
    {
      Unlocked u;
      out = at::empty({slots.numel(), t.size(1)}, t.options());
      const gmm_tensor xv = view(t, code), sv = view(slots, scode), ov = view(out, code);
      if (g_entry.dispatch(x.handle, &xv, &sv, &ov, stream)) x.ok = false;
    }
    return x.ok ? give(out) : none();
  });
}

// combine(rows, slot_row, weights or None, output code or -1, stream)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor rows = x.tensor(0, 2), slots = x.tensor(1, 2);
    const bool weighted = a[2] != Py_None;
    at::Tensor w;
    if (weighted) w = x.tensor(2, 2);
    const long long want = x.number(3);
    void* const stream = x.pointer(4);
    if (!x.ok) return none();
    const int code = code_of(rows.scalar_type());
    if (code < 0 || (want != -1 && want != GMM_F32 && want != GMM_BF16)) return none();
    const at::ScalarType type = want == -1 ? rows.scalar_type() : want == GMM_F32 ? at::kFloat : at::kBFloat16;
    at::Tensor out;
    {
      Unlocked u;
      out = at::empty({slots.size(0), rows.size(1)}, rows.options().dtype(type));
      const gmm_tensor rv = view(rows, code), sv = view(slots, code_of(slots.scalar_type())), ov = view(out, code_of(type));
      gmm_tensor wv{};
      if (weighted) wv = view(w, code_of(w.scalar_type()));
      if (g_entry.combine(x.handle, &rv, &sv, weighted ? &wv : nullptr, &ov, stream)) x.ok = false;
    }
    return x.ok ? give(out) : none();
  });
}

// combine_grad(dout, rows, slot_row, weights, stream)
PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor dout = x.tensor(0, 2), rows = x.tensor(1, 2), slots = x.tensor(2, 2), w = x.tensor(3, 2);
    void* const stream = x.pointer(4);
    if (!x.ok) return none();
    const int rcode = code_of(rows.scalar_type()), wcode = code_of(w.scalar_type());
    if (rcode < 0 || wcode < 0) return none();
    at::Tensor drows, dw;
    {
      Unlocked u;
      drows = at::empty(rows.sizes(), rows.options());
      dw = at::empty(w.sizes(), w.options());
      const gmm_tensor gv = view(dout, code_of(dout.scalar_type())), rv = view(rows, rcode);
      const gmm_tensor sv = view(slots, code_of(slots.scalar_type())), wv = view(w, wcode);
      const gmm_tensor ov = view(drows, rcode), dv = view(dw, wcode);
      if (g_entry.combine_grad(x.handle, &gv, &rv, &sv, &wv, &ov, &dv, stream)) x.ok = false;
    }
    return x.ok ? give(drows, dw) : none();
  });
}

// quant_mxfp4(x, rank, stream)
PyObject* quant_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Args x{a};
    const long long dim = x.number(1);
    const at::Tensor t = x.tensor(0, dim);
    void* const stream = x.pointer(2);
    if (!x.ok || code_of(t.scalar_type()) < 0) return none();
    const int64_t K = t.size(dim - 1);
    at::Tensor q, scale;
    {
      Unlocked u;
      const auto q8 = t.options().dtype(at::kByte), e8 = t.options().dtype(at::kFloat8_e8m0fnu);
      q = dim == 2 ? at::empty({t.size(0), K / 2}, q8) : at::empty({t.size(0), t.size(1), K / 2}, q8);
      scale = dim == 2 ? at::empty({t.size(0), K / 32}, e8) : at::empty({t.size(0), K / 32, 1, t.size(1)}, e8);
      const gmm_tensor xv = view(t, code_of(t.scalar_type())), qv = view_packed(q), sv = view(scale, GMM_E8M0);
      if (g_entry.quant(x.handle, &xv, &qv, &sv, stream)) x.ok = false;
    }
    return x.ok ? give(q, scale) : none();
  });
}

// widen_mxfp4(q, scale, rank of q, output code, stream)
PyObject* widen_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Args x{a};
    const long long dim = x.number(2), want = x.number(3);
    const at::Tensor q = x.tensor(0, dim), scale = x.tensor(1, dim == 2 ? 2 : 4);
    void* const stream = x.pointer(4);
    if (!x.ok || q.scalar_type() != at::kByte || (want != GMM_F32 && want != GMM_BF16)) return none();
    std::vector<int64_t> shape(q.sizes().begin(), q.sizes().end());
    shape.back() *= 2;
    at::Tensor y;
    {
      Unlocked u;
      y = at::empty(shape, q.options().dtype(want == GMM_F32 ? at::kFloat : at::kBFloat16));
      const gmm_tensor qv = view_packed(q), sv = view(scale, code_of(scale.scalar_type())), yv = view(y, (int)want);
      if (g_entry.widen(x.handle, &qv, &sv, &yv, stream)) x.ok = false;
    }
    return x.ok ? give(y) : none();
  });
}

// bind(entry addresses in Entry's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);
  if (n != kEntries) {
    PyErr_SetString(PyExc_TypeError, "wrong number of entry points");
    return nullptr;
  }
  void* at[kEntries];
  for (Py_ssize_t i = 0; i < n; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  static_assert(sizeof at == sizeof g_entry, "entry points");
  memcpy(&g_entry, at, sizeof at);
  for (auto& h : g_handles) h = nullptr;
  return none();
}

// set_handle(device, handle)
PyObject* set_handle(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  const long long dev = PyLong_AsLongLong(a[0]);
  void* const h = PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return nullptr;
  if (dev >= 0 && dev < kDevices) g_handles[dev] = static_cast<gmm_handle*>(h);
  return none();
}

#define GMM_METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {GMM_METHOD(bind),         GMM_METHOD(set_handle),  GMM_METHOD(sort_tokens),
                           GMM_METHOD(dispatch),     GMM_METHOD(combine),     GMM_METHOD(combine_grad),
                           GMM_METHOD(quant_mxfp4),  GMM_METHOD(widen_mxfp4), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_moe_ext", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_ext() { return PyModule_Create(&g_module); }
