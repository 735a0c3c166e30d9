// The Python side of the small calls (norms, row quantiser, 8-bit products, the
// share for a few tokens), whose kernels take 4 to 20 us, less than the checks
// and allocations around them in Python: the same checks on the tensors
// themselves, the outputs, and the call of the C entry point. Calling thread per
// call, ctypes -> here (a launch alone is 3.2 us): norm before the block
// 8.4 -> 4.5 us, after it with two outputs 11.9 -> 5.4, quantiser 9 -> 5.3,
// product 8.6 -> 4.6, few tokens 14.6 -> 8.3 (two launches), 8-bit MLPs 20.5 ->
// 16.7 (four).
//
// Each function returns None where its arguments do not fit (or the tensors
// are not on the current device): the caller's checks then say why. A status
// other than 0 is returned as an int, else the outputs.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// The C entry points, by address: the one library the binding has loaded.
struct {
  decltype(&moe_norm_pre) norm_pre;
  decltype(&moe_norm_post) norm_post;
  decltype(&moe_quantize_rows) quantize_rows;
  decltype(&moe_gemm_i8) gemm_i8;
  decltype(&moe_expert_ffn_i8_workspace_size) expert_ffn_i8_workspace_size;
  decltype(&moe_expert_ffn_i8) expert_ffn_i8;
  decltype(&moe_few_workspace_size) few_workspace_size;
  decltype(&moe_forward_few) forward_few;
  decltype(&moe_forward_few_f32) forward_few_f32;
} entry;

// One call's tensors, all on the current device.
struct Call {
  int index = -1;
  bool ok = true;

  // An argument: its tensor, or none (also for None).
  const Tensor* arg(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  // The first tensor, of n dimensions that are ints to the library: its device
  // has to be the current one.
  const Tensor* first(PyObject* o, int64_t n) {
    const Tensor* t = arg(o);
    ok = ok && t != nullptr && t->is_cuda() && t->dim() == n && t->is_contiguous();
    if (!ok) return nullptr;
    for (const int64_t s : t->sizes()) ok = ok && s <= INT_MAX;
    index = t->get_device();
    ok = ok && index == c10::hip::current_device();
    return t;
  }
  bool is(const Tensor* t, ScalarType type, IntArrayRef shape) {
    return t != nullptr && t->scalar_type() == type && t->sizes() == shape && t->is_cuda() && t->get_device() == index &&
           t->is_contiguous();
  }
  void need(const Tensor* t, ScalarType type, IntArrayRef shape) { ok = ok && is(t, type, shape); }
  void may(const Tensor* t, ScalarType type, IntArrayRef shape) { ok = ok && (t == nullptr || is(t, type, shape)); }
  Tensor out(const Tensor* t, ScalarType type, IntArrayRef shape) const {
    return t ? *t : at::empty(shape, at::TensorOptions(type).device(at::kCUDA, c10::DeviceIndex(index)));
  }
  // The caller's workspace where it is large enough, or a new one.
  Tensor workspace(const Tensor* t, size_t bytes) {
    if (t) {
      ok = ok && t->is_cuda() && t->get_device() == index && t->is_contiguous() && t->nbytes() >= bytes;
      return *t;
    }
    return at::empty({std::max<int64_t>(int64_t(bytes), 1)},
                     at::TensorOptions(at::kByte).device(at::kCUDA, c10::DeviceIndex(index)));
  }
  hipStream_t stream() const { return c10::hip::getCurrentHIPStream(c10::DeviceIndex(index)).stream(); }
};

bool either(const Tensor* t) {
  return t != nullptr && (t->scalar_type() == at::kBFloat16 || t->scalar_type() == at::kFloat);
}
int type_of(const Tensor& t) { return t.scalar_type() == at::kFloat ? MOE_TYPE_F32 : MOE_TYPE_BF16; }

template <typename T>
const T* in(const Tensor* t) {
  return t ? static_cast<const T*>(t->const_data_ptr()) : nullptr;
}
template <typename T>
T* to(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.mutable_data_ptr()) : nullptr;
}

bool number(PyObject* o, float& v) {
  const double d = PyFloat_AsDouble(o);
  v = float(d);
  return !(d == -1.0 && PyErr_Occurred());
}
bool count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
  return false;
}

// f() without the interpreter's lock, which is held again where f throws (a
// tensor without storage has no data pointer)
template <typename F>
int unlocked(F f) {
  struct Unlock {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlock() { PyEval_RestoreThread(state); }
  } unlock;
  return f();
}
PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject *pa = wrap(a), *pb = wrap(b);
  PyObject* t = pa && pb ? PyTuple_Pack(2, pa, pb) : nullptr;
  Py_XDECREF(pa);
  Py_XDECREF(pb);
  return t;
}

// norm_pre(r, w, eps, out)
PyObject* norm_pre(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 4)) return nullptr;
  Call c;
  const Tensor* r = c.first(a[0], 2);
  if (!c.ok || !either(r)) Py_RETURN_NONE;
  const Tensor *w = c.arg(a[1]), *o = c.arg(a[3]);
  const int64_t T = r->size(0), H = r->size(1);
  c.need(w, at::kFloat, {H});
  c.may(o, at::kBFloat16, {T, H});
  if (!c.ok) Py_RETURN_NONE;
  float eps;
  if (!number(a[2], eps)) return nullptr;
  const Tensor out = c.out(o, at::kBFloat16, {T, H});
  const int st = unlocked([&] {
    return entry.norm_pre(in<void>(r), type_of(*r), in<float>(w), eps, int(T), int(H), to<moe_bf16>(out), c.stream());
  });
  return st == MOE_OK ? wrap(out) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// norm_post(y, residual, w_post, gate, residual_scale, w_next, eps, out, normed)
PyObject* norm_post(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 9)) return nullptr;
  Call c;
  const Tensor* y = c.first(a[0], 2);
  if (!c.ok || !either(y)) Py_RETURN_NONE;
  const Tensor *r = c.arg(a[1]), *w_post = c.arg(a[2]), *gate = c.arg(a[3]), *w_next = c.arg(a[5]), *o = c.arg(a[7]),
               *nm = c.arg(a[8]);
  if (!c.ok || !either(r) || (nm && !w_next)) Py_RETURN_NONE;
  const int64_t T = y->size(0), H = y->size(1);
  c.need(r, r->scalar_type(), {T, H});
  c.may(w_post, at::kFloat, {H});
  c.may(w_next, at::kFloat, {H});
  c.may(o, r->scalar_type(), {T, H});
  c.may(nm, at::kBFloat16, {T, H});
  const int kind = !gate                              ? MOE_GATE_NONE
                   : gate->sizes() == IntArrayRef{T, 1} ? MOE_GATE_TOKEN
                   : gate->dim() == 1                   ? MOE_GATE_CHANNEL
                                                        : MOE_GATE_FULL;
  if (kind == MOE_GATE_TOKEN) c.need(gate, at::kFloat, {T, 1});
  if (kind == MOE_GATE_CHANNEL) c.need(gate, at::kFloat, {H});
  if (kind == MOE_GATE_FULL) c.need(gate, at::kFloat, {T, H});
  if (!c.ok) Py_RETURN_NONE;
  float scale, eps;
  if (!number(a[4], scale) || !number(a[6], eps)) return nullptr;
  const Tensor out = c.out(o, r->scalar_type(), {T, H});
  const Tensor normed = w_next ? c.out(nm, at::kBFloat16, {T, H}) : Tensor();
  const int st = unlocked([&] {
    return entry.norm_post(in<void>(y), type_of(*y), in<void>(r), type_of(*r), in<float>(w_post), in<float>(gate), kind,
                           scale, in<float>(w_next), eps, int(T), int(H), to<void>(out), to<moe_bf16>(normed),
                           c.stream());
  });
  return st == MOE_OK ? pair(out, normed) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// quantize_rows(x, q, scale)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 3)) return nullptr;
  Call c;
  const Tensor* x = c.first(a[0], 2);
  if (!c.ok || x->scalar_type() != at::kBFloat16) Py_RETURN_NONE;
  const Tensor *qo = c.arg(a[1]), *so = c.arg(a[2]);
  const int64_t M = x->size(0), K = x->size(1);
  c.may(qo, at::kChar, {M, K});
  c.may(so, at::kFloat, {M});
  if (!c.ok) Py_RETURN_NONE;
  const Tensor q = c.out(qo, at::kChar, {M, K}), scale = c.out(so, at::kFloat, {M});
  const int st = unlocked([&] {
    return entry.quantize_rows(in<moe_bf16>(x), M, int(K), to<int8_t>(q), to<float>(scale), c.stream());
  });
  return st == MOE_OK ? pair(q, scale) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// gemm_i8(a, a_scale, w, w_scale, offsets, out)
PyObject* gemm_i8(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 6)) return nullptr;
  Call c;
  const Tensor* a = c.first(p[0], 2);
  if (!c.ok || a->scalar_type() != at::kChar) Py_RETURN_NONE;
  const Tensor *as = c.arg(p[1]), *w = c.arg(p[2]), *ws = c.arg(p[3]), *offsets = c.arg(p[4]), *o = c.arg(p[5]);
  if (!c.ok || !w || w->dim() != 3) Py_RETURN_NONE;
  const int64_t M = a->size(0), K = a->size(1), E = w->size(0), N = w->size(1);
  c.need(as, at::kFloat, {M});
  c.need(w, at::kChar, {E, N, K});
  c.need(ws, at::kFloat, {E, N});
  c.may(offsets, at::kInt, {E + 1});
  c.may(o, at::kBFloat16, {M, N});
  if (!c.ok || N > INT_MAX || E > INT_MAX || (!offsets && E != 1)) Py_RETURN_NONE;
  const Tensor out = c.out(o, at::kBFloat16, {M, N});
  const int st = unlocked([&] {
    return entry.gemm_i8(in<int8_t>(a), in<float>(as), in<int32_t>(offsets), in<int8_t>(w), in<float>(ws), M, int(N),
                         int(K), int(E), to<moe_bf16>(out), c.stream());
  });
  return st == MOE_OK ? wrap(out) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// expert_ffn_i8(x_perm, offsets, w_gate_up, s_gate_up, w_down, s_down, out, workspace)
PyObject* expert_ffn_i8(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 8)) return nullptr;
  Call c;
  const Tensor* x = c.first(p[0], 2);
  if (!c.ok || x->scalar_type() != at::kBFloat16) Py_RETURN_NONE;
  const Tensor *offsets = c.arg(p[1]), *gu = c.arg(p[2]), *sg = c.arg(p[3]), *dn = c.arg(p[4]), *sd = c.arg(p[5]),
               *o = c.arg(p[6]), *w = c.arg(p[7]);
  if (!c.ok || !gu || gu->dim() != 3 || gu->size(1) % 2 != 0) Py_RETURN_NONE;
  const int64_t cap = x->size(0), H = x->size(1), E = gu->size(0), I = gu->size(1) / 2;
  c.need(offsets, at::kInt, {E + 1});
  c.need(gu, at::kChar, {E, 2 * I, H});
  c.need(sg, at::kFloat, {E, 2 * I});
  c.need(dn, at::kChar, {E, H, I});
  c.need(sd, at::kFloat, {E, H});
  c.may(o, at::kBFloat16, {cap, H});
  if (!c.ok || E > INT_MAX || I > INT_MAX) Py_RETURN_NONE;
  const Tensor ws = c.workspace(w, entry.expert_ffn_i8_workspace_size(int(H), int(I), cap));
  if (!c.ok) Py_RETURN_NONE;
  const Tensor out = c.out(o, at::kBFloat16, {cap, H});
  const int st = unlocked([&] {
    return entry.expert_ffn_i8(in<moe_bf16>(x), in<int32_t>(offsets), in<int8_t>(gu), in<float>(sg), in<int8_t>(dn),
                               in<float>(sd), int(H), int(I), int(E), cap, to<moe_bf16>(out), to<void>(ws), ws.nbytes(),
                               c.stream());
  });
  return st == MOE_OK ? pair(out, ws) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// forward_few(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize, y, workspace)
template <bool F32>
PyObject* forward_few(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 10)) return nullptr;
  Call c;
  const Tensor* x = c.first(p[0], 2);
  if (!c.ok || x->scalar_type() != at::kBFloat16) Py_RETURN_NONE;
  const Tensor *wr = c.arg(p[1]), *bias = c.arg(p[2]), *gu = c.arg(p[3]), *dn = c.arg(p[4]), *o = c.arg(p[8]),
               *w = c.arg(p[9]);
  if (!c.ok || !wr || wr->dim() != 2 || !gu || gu->dim() != 3 || gu->size(2) % 2 != 0) Py_RETURN_NONE;
  const int64_t T = x->size(0), H = x->size(1), E = wr->size(0), El = gu->size(0), I = gu->size(2) / 2;
  const ScalarType type = F32 ? at::kFloat : at::kBFloat16;
  c.need(wr, at::kFloat, {E, H});
  c.may(bias, at::kFloat, {E});
  c.need(gu, at::kBFloat16, {El, H, 2 * I});
  c.need(dn, at::kBFloat16, {El, I, H});
  c.may(o, type, {T, H});
  if (!c.ok || E > INT_MAX || I > INT_MAX || !PyLong_Check(p[5]) || !PyLong_Check(p[6])) Py_RETURN_NONE;
  int over_k, over_e;
  const int64_t k = PyLong_AsLongLongAndOverflow(p[5], &over_k), e0 = PyLong_AsLongLongAndOverflow(p[6], &over_e);
  if (over_k || over_e || k < 1 || k > E || e0 < 0 || e0 > E - El) Py_RETURN_NONE;
  const int renormalize = PyObject_IsTrue(p[7]);
  if (renormalize < 0) return nullptr;
  const Tensor ws = c.workspace(w, entry.few_workspace_size(int(T), int(H), int(I), int(E), int(k), int(El)));
  if (!c.ok) Py_RETURN_NONE;
  const Tensor y = c.out(o, type, {T, H});
  const int st = unlocked([&] {
    if constexpr (F32)
      return entry.forward_few_f32(in<moe_bf16>(x), in<float>(wr), in<float>(bias), in<moe_bf16>(gu), in<moe_bf16>(dn),
                                   int(T), int(H), int(I), int(E), int(k), int(e0), int(El), renormalize, to<float>(y),
                                   to<void>(ws), ws.nbytes(), c.stream());
    else
      return entry.forward_few(in<moe_bf16>(x), in<float>(wr), in<float>(bias), in<moe_bf16>(gu), in<moe_bf16>(dn),
                               int(T), int(H), int(I), int(E), int(k), int(e0), int(El), renormalize, to<moe_bf16>(y),
                               to<void>(ws), ws.nbytes(), c.stream());
  });
  return st == MOE_OK ? pair(y, ws) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points, in the order of `entry`)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[sizeof(entry) / sizeof(void*)];
  static_assert(sizeof(at) == sizeof(entry), "an address each");
  if (!count(n, sizeof(at) / sizeof(void*))) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  memcpy(&entry, at, sizeof(entry));
  Py_RETURN_NONE;
}

typedef PyObject* (*Fast)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"norm_pre", fast(norm_pre), METH_FASTCALL, nullptr},
                         {"norm_post", fast(norm_post), METH_FASTCALL, nullptr},
                         {"quantize_rows", fast(quantize_rows), METH_FASTCALL, nullptr},
                         {"gemm_i8", fast(gemm_i8), METH_FASTCALL, nullptr},
                         {"expert_ffn_i8", fast(expert_ffn_i8), METH_FASTCALL, nullptr},
                         {"forward_few", fast(forward_few<false>), METH_FASTCALL, nullptr},
                         {"forward_few_f32", fast(forward_few<true>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// MOE_BUILT_FOR names the torch and the interpreter whose object layouts and C++
// ABI are compiled in here; the binding calls nothing before it has compared it.
PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
