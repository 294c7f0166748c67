// moe_ext.cpp -- the common call of each operator of gmm_moe.h and gmm_layer.h from Python:
// arguments checked, outputs allocated and the C entry point called without a
// Python step in between (a dispatch call of a decode step takes 4 us on the
// GPU; marshalling it in Python takes longer than launching it).
//
// Every function takes what is plain -- dense device tensors of fitting rank
// and type, outputs to be made, the current stream -- and returns None for
// anything else, a refused call included: the caller (_moe.py, _layer.py) then goes the
// long way, which serves the other forms and says what is wrong.  (A call that failed
// is made again that way: it writes the same outputs.  Not so a step, see adamw.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gmm_layer.h"
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

struct LayerEntry {
  decltype(&gmm_route_run) route;
  decltype(&gmm_balance_loss_workspace) balance_workspace;
  decltype(&gmm_balance_loss_run) balance;
  decltype(&gmm_router_grad_run) router_grad;
  decltype(&gmm_gmv_workspace) gmv_workspace;
  decltype(&gmm_gmv_run) gmv;
  decltype(&gmm_adamw_run) adamw;
} g_layer;

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
  // The same, or nothing where the argument is None.
  at::Tensor maybe(int i, int64_t dim) { return args[i] == Py_None ? at::Tensor() : tensor(i, dim); }
  // A tensor of rank 2 or 3.
  at::Tensor matrix_or_more(int i) {
    const bool three = ok && THPVariable_Check(args[i]) && THPVariable_Unpack(args[i]).dim() == 3;
    return tensor(i, three ? 3 : 2);
  }
  double real(int i) {
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return v;
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

// ---------------------------------------------------------------------------
// gmm_layer.h

// The view of a tensor that may be missing.
struct Maybe {
  gmm_tensor v{};
  bool there = false;
  Maybe(const at::Tensor& t, int code) : there(t.defined()) {
    if (there) v = view(t, code);
  }
  explicit Maybe(const at::Tensor& t) : Maybe(t, t.defined() ? code_of(t.scalar_type()) : -1) {}
  const gmm_tensor* at() const { return there ? &v : nullptr; }
};

bool ids_type(const at::Tensor& t) { return t.scalar_type() == at::kInt || t.scalar_type() == at::kLong; }
// One byte a token: bool, int8 or uint8.
bool flags_type(const at::Tensor& t) {
  return !t.defined() || t.scalar_type() == at::kBool || t.scalar_type() == at::kChar || t.scalar_type() == at::kByte;
}

PyObject* give(const at::Tensor& a, const at::Tensor& b, const at::Tensor& c) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  PyObject* z = THPVariable_Wrap(c);
  PyObject* r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  Py_XDECREF(z);
  return r;
}

// route(logits, k, bias, valid, scores, renormalize, scale, stream)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor z = x.tensor(0, 2);
    const long long k = x.number(1);
    const at::Tensor bias = x.maybe(2, 1), valid = x.maybe(3, 1);
    const long long scores = x.number(4), renorm = x.number(5);
    const double scale = x.real(6);
    void* const stream = x.pointer(7);
    if (!x.ok || k < 1 || k > z.size(1) || !flags_type(valid)) return none();
    const int code = code_of(z.scalar_type());
    at::Tensor ids, w;
    {
      Unlocked u;
      ids = at::empty({z.size(0), (int64_t)k}, z.options().dtype(at::kInt));
      w = at::empty({z.size(0), (int64_t)k}, z.options().dtype(at::kFloat));
      const gmm_tensor zv = view(z, code), iv = view(ids, GMM_I32), wv = view(w, GMM_F32);
      const Maybe bv(bias), vv(valid, GMM_I8);
      if (g_layer.route(x.handle, &zv, bv.at(), vv.at(), (int)scores, renorm != 0, (float)scale, &iv, &wv, stream)) x.ok = false;
    }
    return x.ok ? give(ids, w) : none();
  });
}

// balance_loss(logits, expert_ids, valid, scores, coef, z_coef, stream)
PyObject* balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor z = x.tensor(0, 2), ids = x.tensor(1, 2), valid = x.maybe(2, 1);
    const long long scores = x.number(3);
    const double coef = x.real(4), z_coef = x.real(5);
    void* const stream = x.pointer(6);
    if (!x.ok || !ids_type(ids) || !flags_type(valid)) return none();
    size_t bytes = 0;
    if (g_layer.balance_workspace(z.size(0), z.size(1), &bytes) != GMM_OK) return none();
    at::Tensor loss, counts, tokens;
    {
      Unlocked u;
      const auto i32 = z.options().dtype(at::kInt);
      loss = at::empty({1}, z.options().dtype(at::kFloat));
      counts = at::empty({z.size(1)}, i32);
      tokens = at::empty({1}, i32);
      at::Tensor work;
      if (bytes) work = at::empty({(int64_t)bytes}, z.options().dtype(at::kByte));
      const gmm_tensor zv = view(z, code_of(z.scalar_type())), iv = view(ids, code_of(ids.scalar_type()));
      const gmm_tensor lv = view(loss, GMM_F32), cv = view(counts, GMM_I32), tv = view(tokens, GMM_I32);
      const Maybe vv(valid, GMM_I8);
      if (g_layer.balance(x.handle, &zv, &iv, vv.at(), (int)scores, (float)coef, (float)z_coef, &lv, &cv, &tv,
                          bytes ? work.mutable_data_ptr() : nullptr, bytes, stream))
        x.ok = false;
    }
    return x.ok ? give(loss, counts, tokens) : none();
  });
}

// router_grad(logits, expert_ids, valid, scores, dweights, renormalize, scale, counts, tokens, dloss, coef, z_coef, stream)
PyObject* router_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor z = x.tensor(0, 2), ids = x.tensor(1, 2), valid = x.maybe(2, 1);
    const long long scores = x.number(3);
    const at::Tensor dw = x.maybe(4, 2);
    const long long renorm = x.number(5);
    const double scale = x.real(6);
    const at::Tensor counts = x.maybe(7, 1), tokens = x.maybe(8, 1), dloss = x.maybe(9, 1);
    const double coef = x.real(10), z_coef = x.real(11);
    void* const stream = x.pointer(12);
    if (!x.ok || !ids_type(ids) || !flags_type(valid)) return none();
    const int code = code_of(z.scalar_type());
    at::Tensor dz;
    {
      Unlocked u;
      dz = at::empty(z.sizes(), z.options());
      const gmm_tensor zv = view(z, code), iv = view(ids, code_of(ids.scalar_type())), ov = view(dz, code);
      const Maybe vv(valid, GMM_I8), wv(dw), cv(counts), tv(tokens), lv(dloss);
      if (g_layer.router_grad(x.handle, &zv, &iv, vv.at(), (int)scores, wv.at(), renorm != 0, (float)scale, cv.at(), tv.at(),
                              lv.at(), (float)coef, (float)z_coef, &ov, stream))
        x.ok = false;
    }
    return x.ok ? give(dz) : none();
  });
}

// gmv(x, rhs, format code, rhs_scale, rhs_zero, expert_ids, weights, output code, stream)
PyObject* gmv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Args x{a};
    const at::Tensor t = x.matrix_or_more(0), rhs = x.tensor(1, 3);
    const long long format = x.number(2);
    const at::Tensor scale = x.tensor(3, 4), zero = x.maybe(4, 4), ids = x.maybe(5, 2), w = x.maybe(6, 2);
    const long long want = x.number(7);
    void* const stream = x.pointer(8);
    if (!x.ok || rhs.scalar_type() != at::kByte || (ids.defined() && !ids_type(ids)) || (want != GMM_F32 && want != GMM_BF16))
      return none();
    const int64_t T = t.size(0), k = ids.defined() ? ids.size(1) : 1, N = rhs.size(1);
    if (k < 1 || k > 64 || T > (1 << 20)) return none();
    size_t bytes = 0;
    if (g_layer.gmv_workspace(T * k, N, w.defined(), &bytes) != GMM_OK) return none();
    at::Tensor out;
    {
      Unlocked u;
      const auto type = t.options().dtype(want == GMM_F32 ? at::kFloat : at::kBFloat16);
      out = w.defined() ? at::empty({T, N}, type) : at::empty({T, k, N}, type);
      at::Tensor work;
      if (bytes) work = at::empty({(int64_t)bytes}, t.options().dtype(at::kByte));
      gmm_tensor rv = view(rhs, (int)format);
      rv.shape[2] *= 2;
      const gmm_tensor xv = view(t, code_of(t.scalar_type())), sv = view(scale, code_of(scale.scalar_type()));
      const gmm_tensor ov = view(out, (int)want);
      const Maybe zv(zero), iv(ids), wv(w);
      if (g_layer.gmv(x.handle, &xv, &rv, &sv, zv.at(), iv.at(), wv.at(), &ov, bytes ? work.mutable_data_ptr() : nullptr, bytes,
                      stream))
        x.ok = false;
    }
    return x.ok ? give(out) : none();
  });
}

// One role's tensors of a step, read off a list or tuple.
struct Column {
  PyObject* seq;
  explicit Column(PyObject* o) : seq(PyList_Check(o) || PyTuple_Check(o) ? o : nullptr) {}
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// adamw(params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies, step, lr, beta1, beta2, eps,
//       weight_decay, grad_scale, stream): True, None, or the status of a step that may have been queued in part (it
//       reads what it writes, so it must not be asked for again as a refused one is)
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    Args x{a};
    const Column params(a[0]);
    if (!params.seq || params.size() == 0) return none();
    const Py_ssize_t count = params.size();
    std::vector<gmm_adamw_item> items(count);
    gmm_adamw_args args{};
    for (int role = 0; role < 7; ++role) {
      if (role >= 4 && a[role] == Py_None) continue;
      const Column c(a[role]);
      if (!c.seq || c.size() != count) return none();
      at::ScalarType type{};
      for (Py_ssize_t i = 0; i < count; ++i) {
        if (!THPVariable_Check(c[i])) return none();
        const at::Tensor& t = THPVariable_Unpack(c[i]);
        if (!t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) return none();
        if (x.dev < 0) {
          x.dev = t.get_device();
          x.handle = x.dev < kDevices ? g_handles[x.dev] : nullptr;
          if (!x.handle) return none();
        }
        if (t.get_device() != x.dev || (i > 0 && t.scalar_type() != type)) return none();
        type = t.scalar_type();
        gmm_adamw_item& item = items[i];
        const int64_t elems = t.numel();
        if (role == 0) item.n = elems;
        if (elems != (role == 4 || role == 5 ? (item.n + GMM_ADAMW_BLOCK - 1) / GMM_ADAMW_BLOCK : item.n)) return none();
        // (what is written becomes the tensor's own first, if it is a lazy copy)
        void* const at = !elems ? nullptr : role == 1 ? const_cast<void*>(t.const_data_ptr()) : t.mutable_data_ptr();
        switch (role) {
          case 0: item.param = at; break;
          case 1: item.grad = at; break;
          case 2: item.exp_avg = at; break;
          case 3: item.exp_avg_sq = at; break;
          case 4: item.exp_avg_scale = static_cast<float*>(at); break;
          case 5: item.exp_avg_sq_scale = static_cast<float*>(at); break;
          default: item.copy = at;
        }
      }
      const int code = code_of(type);
      switch (role) {
        case 0: args.param_dtype = code; break;
        case 1: args.grad_dtype = code; break;
        case 2: args.state_dtype = code; break;
        case 3:
          if (code != args.state_dtype) return none();
          break;
        case 4:
        case 5:
          if (type != at::kFloat) return none();
          break;
        default:
          if (type != at::kBFloat16) return none();
      }
    }
    // a number, or one element in device memory
    const auto one = [&](int i, at::ScalarType type) -> const void* {
      const at::Tensor& t = THPVariable_Unpack(a[i]);
      if (!t.is_cuda() || t.get_device() != x.dev || t.scalar_type() != type || t.numel() != 1) x.ok = false;
      return x.ok ? t.const_data_ptr() : nullptr;
    };
    if (THPVariable_Check(a[7]))
      args.step_at = static_cast<const int32_t*>(one(7, at::kInt));
    else
      args.step = x.number(7);
    if (THPVariable_Check(a[8]))
      args.lr_at = static_cast<const float*>(one(8, at::kFloat));
    else
      args.lr = x.real(8);
    args.beta1 = x.real(9);
    args.beta2 = x.real(10);
    args.eps = x.real(11);
    args.weight_decay = x.real(12);
    if (a[13] != Py_None) {
      if (!THPVariable_Check(a[13])) return none();
      args.grad_scale = static_cast<const float*>(one(13, at::kFloat));
    }
    void* const stream = x.pointer(14);
    if (!x.ok) return none();
    gmm_status status;
    {
      Unlocked u;
      status = g_layer.adamw(x.handle, items.data(), count, &args, stream);
    }
    if (status == GMM_E_INVALID || status == GMM_E_UNSUPPORTED) return none();
    // What has been (or may have been) written is another version to autograd.
    for (const int role : {0, 2, 3, 4, 5, 6}) {
      if (a[role] == Py_None) continue;
      const Column c(a[role]);
      for (Py_ssize_t i = 0; i < c.size(); ++i) {
        if (!THPVariable_Check(c[i])) continue;  // (a list is read as it is by now)
        const at::Tensor& t = THPVariable_Unpack(c[i]);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
      }
    }
    if (status != GMM_OK) return PyLong_FromLong(status);
    Py_RETURN_TRUE;
  });
}

// bind(entry addresses in Entry's order); bind_layer(those of LayerEntry)
template <class E>
PyObject* bind_entries(E& entries, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(E) / sizeof(void*);
  if (n != kEntries) {
    PyErr_SetString(PyExc_TypeError, "wrong number of entry points");
    return nullptr;
  }
  void* at[kEntries];
  for (Py_ssize_t i = 0; i < n; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  static_assert(sizeof at == sizeof entries, "entry points");
  memcpy(&entries, at, sizeof at);
  return none();
}
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  PyObject* r = bind_entries(g_entry, a, n);
  if (r)
    for (auto& h : g_handles) h = nullptr;
  return r;
}
PyObject* bind_layer(PyObject*, PyObject* const* a, Py_ssize_t n) { return bind_entries(g_layer, a, n); }

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
                           GMM_METHOD(quant_mxfp4),  GMM_METHOD(widen_mxfp4), GMM_METHOD(bind_layer),
                           GMM_METHOD(route),        GMM_METHOD(balance_loss), GMM_METHOD(router_grad),
                           GMM_METHOD(gmv),          GMM_METHOD(adamw),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_moe_ext", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_ext() { return PyModule_Create(&g_module); }
