// Python binding of the gated delta rule: argument checks, allocation of
// outputs and workspaces, and the call of the C ABI on the current stream of the
// tensors' device. A token of decoding is a call of a few microseconds, and a
// forward of a short prompt two launches: marshalled in Python, the checks and
// allocations took twice as long as the launches (step 12 us, of which 4 were the
// call's own; forward 21, of which 9).
//
// The entry points come as addresses from the loaded library (`bind`), so that
// this module links against torch alone.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/torch.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>

#include "kata.h"

namespace {

struct {
  decltype(&kata_fwd_gated_delta_workspace_bytes) fwd_bytes;
  decltype(&kata_fwd_gated_delta) fwd;
  decltype(&kata_bwd_gated_delta_workspace_bytes) bwd_bytes;
  decltype(&kata_bwd_gated_delta) bwd;
  decltype(&kata_gated_delta_step) step;
} abi;

const at::Tensor none;

// A tensor argument; None gives the undefined tensor where it is allowed.
const at::Tensor &tensor(PyObject *o, const char *name, bool optional = false) {
  if (optional && o == Py_None) return none;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

struct Shape {
  int B, H_k, H, T, d_k, d_v;
  kata_dtype_t dtype;
  c10::DeviceIndex index;
  at::ScalarType type;
};

// Shapes and types of the inputs; `n` dimensions (3: one token, no token axis).
Shape shapes(const at::Tensor &q, const at::Tensor &k, const at::Tensor &v, const at::Tensor &g,
             const at::Tensor &beta, int n) {
  TORCH_CHECK_VALUE(q.dim() == n && k.sizes() == q.sizes() && v.dim() == n && v.size(0) == q.size(0) &&
                        (n == 3 || v.size(2) == q.size(2)),
                    "expected q, k ", n == 4 ? "[B, H_k, T, d_k]" : "[B, H_k, d_k]", " and v ",
                    n == 4 ? "[B, H, T, d_v]" : "[B, H, d_v]", "; got ", q.sizes(), ", ", k.sizes(), ", ", v.sizes());
  Shape s;
  s.type = q.scalar_type();
  TORCH_CHECK_TYPE(k.scalar_type() == s.type && v.scalar_type() == s.type, "q, k, v must share one dtype");
  for (int64_t x : q.sizes()) TORCH_CHECK_VALUE(x <= INT_MAX, "sizes must fit in 32 bits, got ", q.sizes());
  for (int64_t x : v.sizes()) TORCH_CHECK_VALUE(x <= INT_MAX, "sizes must fit in 32 bits, got ", v.sizes());
  s.B = (int)q.size(0);
  s.H_k = (int)q.size(1);
  s.H = (int)v.size(1);
  s.T = n == 4 ? (int)q.size(2) : 1;
  s.d_k = (int)q.size(n - 1);
  s.d_v = (int)v.size(n - 1);
  TORCH_CHECK_VALUE(s.H == 0 || (s.H_k > 0 && s.H % s.H_k == 0), "the ", s.H,
                    " value heads must be a multiple of the ", s.H_k, " key heads");
  const auto tokens = v.sizes().slice(0, n - 1);
  TORCH_CHECK_VALUE(g.sizes() == tokens && beta.sizes() == tokens, "g and beta must be ", tokens, " fp32, got ",
                    g.sizes(), " and ", beta.sizes());
  TORCH_CHECK_TYPE(s.type == at::kFloat || s.type == at::kBFloat16, "unsupported dtype ", q.dtype(),
                   "; use float32 or bfloat16");
  s.dtype = s.type == at::kFloat ? KATA_DTYPE_F32 : KATA_DTYPE_BF16;
  s.index = q.is_cuda() ? q.get_device() : -1;
  return s;
}

// An output or a state: shape and type as they have to be (or undefined).
void like(const at::Tensor &t, at::IntArrayRef sizes, at::ScalarType type, const char *name) {
  TORCH_CHECK_VALUE(!t.defined() || (t.sizes() == sizes && t.scalar_type() == type), name, " must be ", sizes, " ",
                    type, ", got ", t.sizes(), " ", t.scalar_type());
}

// Device pointer of a contiguous tensor on q's device (null for an undefined one).
template <typename P = void> P *ptr(const at::Tensor &t, const char *name, const Shape &s, at::ScalarType type) {
  if (!t.defined()) return nullptr;
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
  TORCH_CHECK_VALUE(t.get_device() == s.index, name, " is on ", t.device(), ", q is not");
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return static_cast<P *>(t.data_ptr());
}

struct Workspace {
  at::Tensor held;
  void *p;
  size_t bytes;
};
Workspace workspace(const at::Tensor &given, size_t need, const Shape &s, const at::Tensor &q) {
  if (given.defined())
    return {given, ptr(given, "workspace", s, given.scalar_type()), (size_t)given.numel() * given.element_size()};
  TORCH_CHECK_VALUE(need > 0, "unsupported shape for the gated delta rule: B, H_k, H, T, d_k, d_v = ", s.B, ", ",
                    s.H_k, ", ", s.H, ", ", s.T, ", ", s.d_k, ", ", s.d_v);
  at::Tensor t = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
  void *p = t.data_ptr();
  return {std::move(t), p, need};
}

kata_stream_t stream(const Shape &s) {
  return reinterpret_cast<kata_stream_t>(c10::cuda::getCurrentCUDAStream(s.index).stream());
}

PyObject *wrap(const at::Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// (status, tensors ...)
template <size_t N> PyObject *result(kata_status_t status, const at::Tensor *const (&out)[N]) {
  PyObject *tuple = PyTuple_New(N + 1);
  if (!tuple) return nullptr;
  PyTuple_SET_ITEM(tuple, 0, PyLong_FromLong((long)status));
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(tuple, i + 1, wrap(*out[i]));
  return tuple;
}
void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// fwd(q, k, v, g, beta, S0, want_state, o, S_out, workspace): o None allocates o
// and, if want_state, S_out.
PyObject *fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &g = tensor(a[3], "g"),
                   &beta = tensor(a[4], "beta"), &S0 = tensor(a[5], "S0", true);
  const Shape s = shapes(q, k, v, g, beta, 4);
  const int64_t state[4] = {s.B, s.H, s.d_k, s.d_v};
  at::Tensor o = tensor(a[7], "o", true), S = tensor(a[8], "S_out", true);
  like(o, v.sizes(), s.type, "o");
  like(S0, state, at::kFloat, "S0");
  like(S, state, at::kFloat, "S_out");
  const void *pq = ptr(q, "q", s, s.type), *pk = ptr(k, "k", s, s.type), *pv = ptr(v, "v", s, s.type);
  const float *pg = ptr<float>(g, "g", s, at::kFloat), *pb = ptr<float>(beta, "beta", s, at::kFloat),
              *p0 = ptr<float>(S0, "S0", s, at::kFloat);
  const c10::cuda::CUDAGuard guard(s.index);
  if (!o.defined()) {
    o = at::empty_like(v);
    if (a[6] == Py_True) S = at::empty(state, v.options().dtype(at::kFloat));
  }
  void *po = ptr(o, "o", s, s.type);
  float *pS = ptr<float>(S, "S_out", s, at::kFloat);
  const at::Tensor &given = tensor(a[9], "workspace", true);
  const Workspace ws = workspace(
      given, given.defined() ? 0 : abi.fwd_bytes(s.B, s.H_k, s.H, s.T, s.d_k, s.d_v, s.dtype), s, q);
  const kata_status_t st = abi.fwd(pq, pk, pv, pg, pb, po, s.B, s.H_k, s.H, s.T, s.d_k, s.d_v, s.dtype, p0, pS, ws.p,
                                   ws.bytes, stream(s));
  return result(st, {&o, &S});
  END_HANDLE_TH_ERRORS
}

// bwd(q, k, v, g, beta, dout, S0, dS, dq, dk, dv, dg, dbeta, dS0, workspace): dq None
// allocates all gradients (dS0 if S0 is given).
PyObject *bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &g = tensor(a[3], "g"),
                   &beta = tensor(a[4], "beta"), &dout = tensor(a[5], "dout"), &S0 = tensor(a[6], "S0", true),
                   &dS = tensor(a[7], "dS", true);
  const Shape s = shapes(q, k, v, g, beta, 4);
  const int64_t state[4] = {s.B, s.H, s.d_k, s.d_v};
  const bool make = a[8] == Py_None;
  at::Tensor dq = tensor(a[8], "dq", true), dk = tensor(a[9], "dk", make), dv = tensor(a[10], "dv", make),
             dg = tensor(a[11], "dg", make), dbeta = tensor(a[12], "dbeta", make), dS0 = tensor(a[13], "dS0", true);
  like(dout, v.sizes(), s.type, "dout");
  like(dq, q.sizes(), s.type, "dq");
  like(dk, k.sizes(), s.type, "dk");
  like(dv, v.sizes(), s.type, "dv");
  like(dg, g.sizes(), at::kFloat, "dg");
  like(dbeta, g.sizes(), at::kFloat, "dbeta");
  like(S0, state, at::kFloat, "S0");
  like(dS, state, at::kFloat, "dS");
  like(dS0, state, at::kFloat, "dS0");
  const void *pq = ptr(q, "q", s, s.type), *pk = ptr(k, "k", s, s.type), *pv = ptr(v, "v", s, s.type),
             *po = ptr(dout, "dout", s, s.type);
  const float *pg = ptr<float>(g, "g", s, at::kFloat), *pb = ptr<float>(beta, "beta", s, at::kFloat),
              *p0 = ptr<float>(S0, "S0", s, at::kFloat), *pS = ptr<float>(dS, "dS", s, at::kFloat);
  const c10::cuda::CUDAGuard guard(s.index);
  if (make) {
    dq = at::empty_like(q);
    dk = at::empty_like(k);
    dv = at::empty_like(v);
    dg = at::empty_like(g);
    dbeta = at::empty_like(beta);
    if (S0.defined()) dS0 = at::empty_like(S0);
  }
  void *oq = ptr(dq, "dq", s, s.type), *ok = ptr(dk, "dk", s, s.type), *ov = ptr(dv, "dv", s, s.type);
  float *og = ptr<float>(dg, "dg", s, at::kFloat), *ob = ptr<float>(dbeta, "dbeta", s, at::kFloat),
        *o0 = ptr<float>(dS0, "dS0", s, at::kFloat);
  const at::Tensor &given = tensor(a[14], "workspace", true);
  const Workspace ws = workspace(
      given, given.defined() ? 0 : abi.bwd_bytes(s.B, s.H_k, s.H, s.T, s.d_k, s.d_v, s.dtype), s, q);
  const kata_status_t st = abi.bwd(pq, pk, pv, pg, pb, po, p0, pS, oq, ok, ov, og, ob, o0, s.B, s.H_k, s.H, s.T,
                                   s.d_k, s.d_v, s.dtype, ws.p, ws.bytes, stream(s));
  return result(st, {&dq, &dk, &dv, &dg, &dbeta, &dS0});
  END_HANDLE_TH_ERRORS
}

// step(q, k, v, g, beta, S, y): y None allocates it.
PyObject *step(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &g = tensor(a[3], "g"),
                   &beta = tensor(a[4], "beta"), &S = tensor(a[5], "S");
  const Shape s = shapes(q, k, v, g, beta, 3);
  const int64_t state[4] = {s.B, s.H, s.d_k, s.d_v};
  at::Tensor y = tensor(a[6], "y", true);
  like(y, v.sizes(), s.type, "y");
  like(S, state, at::kFloat, "S");
  const void *pq = ptr(q, "q", s, s.type), *pk = ptr(k, "k", s, s.type), *pv = ptr(v, "v", s, s.type);
  const float *pg = ptr<float>(g, "g", s, at::kFloat), *pb = ptr<float>(beta, "beta", s, at::kFloat);
  float *pS = ptr<float>(S, "S", s, at::kFloat);
  const c10::cuda::CUDAGuard guard(s.index);
  if (!y.defined()) y = at::empty_like(v);
  const kata_status_t st = abi.step(pq, pk, pv, pg, pb, pS, ptr(y, "y", s, s.type), s.B, s.H_k, s.H, s.d_k, s.d_v,
                                    s.dtype, stream(s));
  return result(st, {&y});
  END_HANDLE_TH_ERRORS
}

// bind(addresses): those of the five entry points, in the order of `abi`.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5);
  void *p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_ValueError, "null entry point"), nullptr);
  }
  abi.fwd_bytes = reinterpret_cast<decltype(abi.fwd_bytes)>(p[0]);
  abi.fwd = reinterpret_cast<decltype(abi.fwd)>(p[1]);
  abi.bwd_bytes = reinterpret_cast<decltype(abi.bwd_bytes)>(p[2]);
  abi.bwd = reinterpret_cast<decltype(abi.bwd)>(p[3]);
  abi.step = reinterpret_cast<decltype(abi.step)>(p[4]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(bind)), METH_FASTCALL, nullptr},
    {"fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(fwd)), METH_FASTCALL, nullptr},
    {"bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(bwd)), METH_FASTCALL, nullptr},
    {"step", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(step)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
