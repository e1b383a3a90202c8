// The packed-batch helpers of sala.py below their Python signatures: checks of
// what the C entry points cannot see (shapes, types, devices), outputs and
// workspaces from torch's allocator, and the call.
//
// In C++ because these calls are made once per decode token: with the checks,
// allocations and the call in Python a single-token step of 4 requests took
// 15 us of host time against 3 us on the GPU.
//
// Every function takes positional arguments (sala.py has the signatures), works
// on the tensors' device and its current stream, and returns its outputs, or the
// sala_status of a refused call as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/sala.h"

namespace {

using at::Tensor;

struct Refused {};      // a Python error is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused{};
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw Refused{};
  }
  return THPVariable_Unpack(o);
}

const Tensor& ranked(PyObject* o, const char* name, int64_t dim) {
  const Tensor& t = tensor(o, name);
  if (t.dim() != dim) refuse(std::string(name) + ": shape " + shape_text(t.sizes()) + ", expected " + std::to_string(dim) + " dimensions");
  return t;
}

void expect(const char* name, const Tensor& t, std::initializer_list<int64_t> shape, at::ScalarType dtype, at::Device device) {
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) refuse(std::string(name) + ": shape " + shape_text(t.sizes()) + ", expected " + shape_text(want));
  if (t.scalar_type() != dtype)
    refuse(std::string(name) + ": " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(dtype));
  if (t.device() != device) refuse(std::string(name) + ": on " + t.device().str() + ", expected " + device.str());
  if (!t.is_contiguous()) refuse(std::string(name) + ": must be contiguous");
}

const Tensor& expect(const char* name, PyObject* o, std::initializer_list<int64_t> shape, at::ScalarType dtype, at::Device device) {
  const Tensor& t = tensor(o, name);
  expect(name, t, shape, dtype, device);
  return t;
}

void on_cuda(const char* what, at::Device device) {
  if (!device.is_cuda()) refuse(std::string(what) + ": tensors must be on a CUDA device");
}

int count(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(std::string(name) + ": more than 2^31 - 1");
  return (int)n;
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

Tensor optional(const char* name, PyObject* o, std::initializer_list<int64_t> shape, at::ScalarType dtype, at::Device device) {
  return o == Py_None ? Tensor() : expect(name, o, shape, dtype, device);
}

Tensor output(const char* name, PyObject* o, std::initializer_list<int64_t> shape, at::ScalarType dtype, at::Device device) {
  if (o != Py_None) return expect(name, o, shape, dtype, device);
  return at::empty(at::IntArrayRef(shape.begin(), shape.size()), at::TensorOptions().dtype(dtype).device(device));
}

struct Workspace {
  Tensor t;
  size_t bytes = 0;
  Workspace(PyObject* o, size_t need, at::Device device) {
    if (o != Py_None) {
      t = tensor(o, "ws");
      if (t.device() != device || !t.is_contiguous()) refuse("ws: a contiguous tensor on the call's device");
    } else if (need > 0) {
      t = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(device));
    }
    if (t.defined()) bytes = t.nbytes();
  }
};

// Two objects of a list or tuple, or None twice for None.
struct Pair {
  PyObject* seq = nullptr;
  Pair(PyObject* o, const char* name) {
    if (o == Py_None) return;
    if ((!PyList_Check(o) && !PyTuple_Check(o)) || PySequence_Fast_GET_SIZE(o) != 2)
      refuse(std::string(name) + ": expected a pair of tensors");
    seq = o;
  }
  PyObject* first() const { return seq ? PySequence_Fast_GET_ITEM(seq, 0) : Py_None; }
  PyObject* second() const { return seq ? PySequence_Fast_GET_ITEM(seq, 1) : Py_None; }
};

sala_dtype dtype_code(const char* name, const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return SALA_BF16;
  if (t.scalar_type() == at::kFloat) return SALA_F32;
  refuse(std::string(name) + ": unsupported dtype " + c10::toString(t.scalar_type()));
}

float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused{};
  return (float)x;
}

PyObject* status(sala_status s) { return PyLong_FromLong(s); }

void* stream_of(at::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

constexpr at::ScalarType BF = at::kBFloat16, F32 = at::kFloat, I32 = at::kInt;

// q, k, wq, wk, positions, rope_base, rms_eps, outs
PyObject* qk_norm(PyObject* const* a) {
  const Tensor& q = ranked(a[0], "q", 3);
  const Tensor& k = ranked(a[1], "k", 3);
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k.size(1);
  const at::Device dev = q.device();
  expect("q", q, {T, Hq, D}, q.scalar_type(), dev);
  expect("k", k, {T, Hk, D}, q.scalar_type(), dev);
  const Tensor& wq = expect("wq", a[2], {D}, F32, dev);
  const Tensor& wk = expect("wk", a[3], {D}, F32, dev);
  const Tensor pos = optional("positions", a[4], {T}, I32, dev);
  const Pair outs(a[7], "outs");
  on_cuda("sala_qk_norm", dev);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor qn = output("q_norm", outs.first(), {T, Hq, D}, BF, dev), kn = output("k_norm", outs.second(), {T, Hk, D}, BF, dev);
  const sala_qk_norm_desc d = {count(T, "tokens"), count(Hq, "heads"), count(Hk, "heads"), count(D, "head_dim"),
                               dtype_code("q", q), number(a[5]), number(a[6])};
  const sala_status s = sala_qk_norm(&d, ptr(q), ptr(k), (const float*)ptr(wq), (const float*)ptr(wk),
                                     (const int32_t*)ptr(pos), ptr(qn), ptr(kn), stream_of(dev));
  if (s != SALA_OK) return status(s);
  if (a[7] != Py_None) return Py_NewRef(a[7]);
  PyObject* x = THPVariable_Wrap(std::move(qn));
  PyObject* y = THPVariable_Wrap(std::move(kn));
  PyObject* pair = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return pair;
}

PyObject* returned(PyObject* given, Tensor&& out) {
  return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(std::move(out));
}

// q_norm, k_norm, v, gate, cu_seqlens, scale, out, ws
PyObject* dense_prefill(PyObject* const* a) {
  const Tensor& q = ranked(a[0], "q_norm", 3);
  const Tensor& k = ranked(a[1], "k_norm", 3);
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
  const at::Device dev = q.device();
  expect("q_norm", q, {T, Hq, D}, BF, dev);
  expect("k_norm", k, {T, Hkv, D}, BF, dev);
  const Tensor& v = expect("v", a[2], {T, Hkv, D}, BF, dev);
  const Tensor& gate = expect("gate", a[3], {T, Hq, D}, BF, dev);
  const Tensor& cu = ranked(a[4], "cu_seqlens", 1);
  expect("cu_seqlens", cu, {cu.size(0)}, I32, dev);
  on_cuda("sala_dense_prefill", dev);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out = output("out", a[6], {T, Hq, D}, BF, dev);
  const sala_dense_desc d = {count(T, "tokens"), count(cu.size(0) - 1, "sequences"), count(Hq, "heads"), count(Hkv, "heads"),
                             count(D, "head_dim"), SALA_BF16, number(a[5])};
  const Workspace ws(a[7], sala_dense_workspace_size(&d), dev);
  const sala_status s = sala_dense_prefill(&d, ptr(q), ptr(k), ptr(v), ptr(gate), (const int32_t*)ptr(cu), ptr(out),
                                           ptr(ws.t), ws.bytes, stream_of(dev));
  return s == SALA_OK ? returned(a[6], std::move(out)) : status(s);
}

// The tensors that both forms of linear attention take.
struct Linear {
  const Tensor &q, &k, &v, &gate, &lam;
  at::Device dev;
  int64_t T, H, D;
  Linear(PyObject* const* a)
      : q(ranked(a[0], "q_norm", 3)), k(tensor(a[1], "k_norm")), v(tensor(a[2], "v")), gate(tensor(a[3], "gate")),
        lam(tensor(a[4], "lam")), dev(q.device()), T(q.size(0)), H(q.size(1)), D(q.size(2)) {
    expect("q_norm", q, {T, H, D}, BF, dev);
    expect("k_norm", k, {T, H, D}, BF, dev);
    expect("v", v, {T, H, D}, v.scalar_type(), dev);
    expect("gate", gate, {T, H, D}, v.scalar_type(), dev);
    expect("lam", lam, {H}, F32, dev);
  }
  sala_packed_linear_desc desc(int64_t n, int64_t n_slots, PyObject* scale) const {
    return {count(T, "tokens"), count(n, "sequences"), count(n_slots, "slots"), count(H, "heads"), count(D, "head_dim"),
            dtype_code("v", v), number(scale)};
  }
};

// q_norm, k_norm, v, gate, lam, cu_seqlens, slots, state_in, state_out, scale, out, ws
PyObject* linear_packed_prefill(PyObject* const* a) {
  const Linear t(a);
  const Tensor& cu = ranked(a[5], "cu_seqlens", 1);
  expect("cu_seqlens", cu, {cu.size(0)}, I32, t.dev);
  const int64_t n = cu.size(0) - 1;
  const Tensor slots = optional("slots", a[6], {n}, I32, t.dev);
  int64_t n_slots = n;
  for (const int i : {8, 7})
    if (a[i] != Py_None) n_slots = ranked(a[i], "state", 4).size(0);
  const Tensor in = optional("state", a[7], {n_slots, t.H, t.D, t.D}, F32, t.dev);
  const Tensor fin = optional("state", a[8], {n_slots, t.H, t.D, t.D}, F32, t.dev);
  on_cuda("sala_linear_packed_prefill", t.dev);
  const c10::cuda::CUDAGuard guard(t.dev);
  Tensor out = output("out", a[10], {t.T, t.H, t.D}, t.v.scalar_type(), t.dev);
  const sala_packed_linear_desc d = t.desc(n, n_slots, a[9]);
  const Workspace ws(a[11], sala_linear_packed_workspace_size(&d), t.dev);
  const sala_status s = sala_linear_packed_prefill(
      &d, ptr(t.q), ptr(t.k), ptr(t.v), ptr(t.gate), (const float*)ptr(t.lam), (const int32_t*)ptr(cu),
      (const int32_t*)ptr(slots), (const float*)ptr(in), (float*)ptr(fin), ptr(out), ptr(ws.t), ws.bytes, stream_of(t.dev));
  return s == SALA_OK ? returned(a[10], std::move(out)) : status(s);
}

// q_norm, k_norm, v, gate, lam, state, slots, scale, out
PyObject* linear_packed_step(PyObject* const* a) {
  const Linear t(a);
  const Tensor& state = ranked(a[5], "state", 4);
  expect("state", state, {state.size(0), t.H, t.D, t.D}, F32, t.dev);
  const Tensor slots = optional("slots", a[6], {t.T}, I32, t.dev);
  on_cuda("sala_linear_packed_step", t.dev);
  const c10::cuda::CUDAGuard guard(t.dev);
  Tensor out = output("out", a[8], {t.T, t.H, t.D}, t.v.scalar_type(), t.dev);
  const sala_packed_linear_desc d = t.desc(t.T, state.size(0), a[7]);
  const sala_status s = sala_linear_packed_step(&d, ptr(t.q), ptr(t.k), ptr(t.v), ptr(t.gate), (const float*)ptr(t.lam),
                                                (const int32_t*)ptr(slots), (float*)ptr(state), ptr(out), stream_of(t.dev));
  return s == SALA_OK ? returned(a[8], std::move(out)) : status(s);
}

// q_norm, k_norm, v, gate, prefix_k, prefix_v, k_cache, v_cache, lens, slots, scale, out, ws
PyObject* prefix_decode(PyObject* const* a) {
  const Tensor& q = ranked(a[0], "q_norm", 3);
  const Tensor& k = ranked(a[1], "k_norm", 3);
  const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
  const at::Device dev = q.device();
  expect("q_norm", q, {B, Hq, D}, BF, dev);
  expect("k_norm", k, {B, Hkv, D}, BF, dev);
  const Tensor& v = expect("v", a[2], {B, Hkv, D}, BF, dev);
  const Tensor& gate = expect("gate", a[3], {B, Hq, D}, BF, dev);
  if ((a[4] == Py_None) != (a[5] == Py_None)) refuse("prefix_k and prefix_v: both or neither");
  const int64_t P = a[4] == Py_None ? 0 : ranked(a[4], "prefix_k", 3).size(0);
  const Tensor pk = optional("prefix_k", a[4], {P, Hkv, D}, BF, dev);
  const Tensor pv = optional("prefix_v", a[5], {P, Hkv, D}, BF, dev);
  const Tensor& kc = ranked(a[6], "k_cache", 4);
  const int64_t n_slots = kc.size(0), cap = kc.size(1);
  expect("k_cache", kc, {n_slots, cap, Hkv, D}, BF, dev);
  const Tensor& vc = expect("v_cache", a[7], {n_slots, cap, Hkv, D}, BF, dev);
  const Tensor& lens = expect("lens", a[8], {B}, I32, dev);
  const Tensor slots = optional("slots", a[9], {B}, I32, dev);
  on_cuda("sala_prefix_decode", dev);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out = output("out", a[11], {B, Hq, D}, BF, dev);
  const sala_prefix_desc d = {count(B, "requests"), count(P, "prefix"), count(n_slots, "slots"), count(Hq, "heads"),
                              count(Hkv, "heads"), count(D, "head_dim"), cap, SALA_BF16, number(a[10])};
  const Workspace ws(a[12], sala_prefix_workspace_size(&d), dev);
  const sala_status s = sala_prefix_decode(&d, ptr(q), ptr(k), ptr(v), ptr(gate), P ? ptr(pk) : nullptr,
                                           P ? ptr(pv) : nullptr, ptr(kc), ptr(vc), (const int32_t*)ptr(lens),
                                           (const int32_t*)ptr(slots), ptr(out), ptr(ws.t), ws.bytes, stream_of(dev));
  return s == SALA_OK ? returned(a[11], std::move(out)) : status(s);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define SALA_METHOD(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SALA_METHOD(qk_norm, 8), SALA_METHOD(dense_prefill, 8), SALA_METHOD(linear_packed_prefill, 12),
                         SALA_METHOD(linear_packed_step, 9), SALA_METHOD(prefix_decode, 13), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_packed", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__packed() { return PyModule_Create(&module); }
