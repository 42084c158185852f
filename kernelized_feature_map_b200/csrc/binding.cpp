// binding.cpp -- Python binding of linear attention with a per-head decay and
// of the 8-bit state cache (include/kata.h): argument checks and marshalling.
//
// These calls are made once per layer and token, where the arithmetic takes a
// few microseconds; a binding through ctypes, with its checks in Python, takes
// 17 to 24 us for one of them, this one 3 to 4.5.
//
// Token tensors are [T, H, width] with the last two dimensions dense; the
// stride between tokens is free (a multiple of 16 bytes), so the parts of a
// fused projection go in as they are.  Every tensor of a call is on one device,
// which need not be the current one.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kata.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* kata_error = nullptr;  // the package's KataError

// KataError(function, status), as a Python exception in flight
[[noreturn]] void fail(const char* fn, int status) {
  PyObject* args = Py_BuildValue("(si)", fn, status);
  if (args) {
    PyErr_SetObject(kata_error ? kata_error : PyExc_RuntimeError, args);
    Py_DECREF(args);
  }
  throw python_error();
}
void check(const char* fn, int status) {
  if (status != KATA_OK) fail(fn, status);
}

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), name, " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

constexpr int64_t kAny = -1;

// Pointer of a contiguous CUDA tensor of this type and shape.
void* dense(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, at::Device device) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.device() == device, name, " is on ", t.device(), ", the call's tensors are on ", device);
  bool same = t.dim() == (int64_t)shape.size();
  for (size_t i = 0; same && i < shape.size(); ++i) same = shape[i] == kAny || shape[i] == t.size(i);
  TORCH_CHECK_VALUE(same, name, " must have the shape ", shape, " (-1: any), got ", t.sizes());
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return t.data_ptr();
}
void* optional(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, at::Device device) {
  return o == Py_None ? nullptr : dense(o, name, type, shape, device);
}

// A [rows, H, width] tensor, dense within a row; its pointer and the elements from one row to the next.
struct Rows {
  void* ptr;
  int64_t stride;
};
Rows rows(const Tensor& t, const char* name, ScalarType type, int64_t n, int64_t H, int64_t w, at::Device device) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.device() == device, name, " is on ", t.device(), ", the call's tensors are on ", device);
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == n && t.size(1) == H && t.size(2) == w, name, " must have the shape [",
                    n, ", ", H, ", ", w, "], got ", t.sizes());
  TORCH_CHECK_VALUE(n * H * w == 0 || ((w == 1 || t.stride(2) == 1) && (H == 1 || t.stride(1) == w)), name,
                    " must be dense within a token (its last two dimensions contiguous)");
  return {t.data_ptr(), n > 1 ? t.stride(0) : H * w};
}

int narrow(int64_t x, const char* what) {
  TORCH_CHECK_VALUE(x <= INT_MAX, what, " is ", x, ", more than the library counts");
  return (int)x;
}

// What the leading tensors q and v say about a call.
struct Lead {
  const Tensor &q, &v;
  at::Device device;
  ScalarType type;
  kata_dtype_t code;
  int64_t n, H, d, dv;
};
Lead lead(PyObject* qo, PyObject* vo, const char* what) {
  const Tensor &q = tensor(qo, "q"), &v = tensor(vo, "v");
  for (const Tensor* t : {&q, &v})
    TORCH_CHECK_VALUE(t->dim() == 3, t == &q ? "q" : "v", " must be [", what, ", H, width], got ", t->sizes());
  const ScalarType type = q.scalar_type();
  TORCH_CHECK_TYPE(type == at::kBFloat16 || type == at::kFloat,
                   "q, k, v must be torch.bfloat16 or torch.float32, got ", type);
  narrow(q.size(0), what);
  narrow(q.size(1), "H");
  narrow(q.size(2), "the width of q");
  narrow(v.size(2), "the width of v");
  return {q, v, q.device(), type, type == at::kBFloat16 ? KATA_BF16 : KATA_F32, q.size(0), q.size(1), q.size(2),
          v.size(2)};
}

Tensor empty(at::IntArrayRef shape, ScalarType type, at::Device device) {
  return Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

// Tensors of the caller that a call has written: torch's version counter says so to autograd, which refuses a backward
// pass whose saved tensors were written since.  (Inference tensors have none.)
void written(std::initializer_list<PyObject*> tensors) {
  for (PyObject* o : tensors) {
    if (o == Py_None) continue;
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
}

// The stream of a call: the one that was given, or the device's current one.
c10::cuda::CUDAStream stream_of(PyObject* o, at::Device device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device.index());
  PyObject* p = PyObject_GetAttrString(o, "cuda_stream");
  if (!p) throw python_error();
  void* ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  if (!ptr && PyErr_Occurred()) throw python_error();
  return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(ptr), device.index());
}

// A call's device, and its stream as the current one, so that what the call
// allocates belongs to that stream: from another stream's pool it could still be
// read there, by work that was queued before its owner let it go.
struct CallGuard {
  c10::cuda::CUDAGuard device;
  c10::cuda::CUDAStream stream;
  c10::cuda::OptionalCUDAStreamGuard current;
  CallGuard(c10::Device d, PyObject* stream_arg) : device(d), stream(stream_of(stream_arg, d)) {
    if (stream_arg != Py_None) current.reset_stream(stream);
  }
};

// The caller's workspace, or one that the allocator keeps until the stream is past the call.
struct Workspace {
  Tensor held;
  void* ptr = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, size_t need, at::Device device) {
    if (o != Py_None) {
      const Tensor& t = tensor(o, "workspace");
      TORCH_CHECK_VALUE(t.device() == device && t.is_contiguous(), "workspace must be a contiguous CUDA tensor on ",
                        device);
      ptr = t.data_ptr();
      bytes = t.nbytes();
    } else if (need) {
      held = empty({(int64_t)need}, at::kByte, device);
      ptr = held.data_ptr();
      bytes = need;
    }
  }
};

const int* sequences(PyObject* o, at::Device device, int& N) {
  if (o == Py_None) {
    N = 1;
    return nullptr;
  }
  const Tensor& t = tensor(o, "cu_seqlens");
  TORCH_CHECK_VALUE(t.dim() == 1 && t.numel() >= 1, "cu_seqlens must be [N + 1]");
  N = narrow(t.numel() - 1, "N");
  return static_cast<const int*>(dense(o, "cu_seqlens", at::kInt, {kAny}, device));
}

float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x != 0;
}
void count(Py_ssize_t have, Py_ssize_t want) {
  TORCH_CHECK_TYPE(have == want, "expected ", want, " arguments, got ", have);
}

// q, k, v, log_decay, cu_seqlens, scale, S0, S_out, slots, resume, return_state, zero_outside, o, workspace, stream
PyObject* fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const Lead c = lead(a[0], a[2], "T");
  const Rows q = rows(c.q, "q", c.type, c.n, c.H, c.d, c.device);
  const Rows k = rows(tensor(a[1], "k"), "k", c.type, c.n, c.H, c.d, c.device);
  const Rows v = rows(c.v, "v", c.type, c.n, c.H, c.dv, c.device);
  int N;
  const int* cu = sequences(a[4], c.device, N);
  const bool return_state = truth(a[10]);
  PyObject* pool = a[6] != Py_None ? a[6] : a[7];
  Tensor held_state;
  if (return_state && a[7] == Py_None)
    TORCH_CHECK_VALUE(a[8] == Py_None, "with slots, give the pool S_out that the final states go to");
  int64_t n_slots = 0;
  if (pool != Py_None) {
    const Tensor& t = tensor(pool, "S0 and S_out");
    n_slots = t.dim() ? t.size(0) : 0;
  } else if (return_state) {
    n_slots = N;
  }
  const int64_t state[4] = {n_slots, c.H, c.d, c.dv};
  const CallGuard guard(c.device, a[14]);
  float* S0 = static_cast<float*>(optional(a[6], "S0", at::kFloat, state, c.device));
  float* S_out = static_cast<float*>(optional(a[7], "S_out", at::kFloat, state, c.device));
  const int64_t fresh[4] = {N, c.H, c.d, c.dv};
  if (return_state && !S_out && a[7] == Py_None) {
    held_state = empty(fresh, at::kFloat, c.device);
    S_out = static_cast<float*>(held_state.data_ptr());
    TORCH_CHECK_VALUE(n_slots >= N, "S0 has ", n_slots, " states for ", N, " sequences");
  }
  Tensor held_o;
  if (a[12] == Py_None) held_o = empty({c.n, c.H, c.dv}, c.type, c.device);
  const Tensor& ot = a[12] == Py_None ? held_o : tensor(a[12], "o");
  const Rows o = rows(ot, "o", c.type, c.n, c.H, c.dv, c.device);
  const bool zero_outside = a[11] == Py_None ? a[12] == Py_None : truth(a[11]);
  const float* decay = static_cast<const float*>(dense(a[3], "log_decay", at::kFloat, {c.H}, c.device));
  const int* slots = static_cast<const int*>(optional(a[8], "slots", at::kInt, {N}, c.device));
  const unsigned char* resume = static_cast<const unsigned char*>(optional(a[9], "resume", at::kByte, {N}, c.device));
  const float scale = number(a[5]);
  // a state pool that is allocated here has a row for each sequence, S0 may have more: without slots only the
  // first N rows of either are the call's
  const Workspace ws(a[13], kata_fwd_linear_decay_workspace_size(c.n, c.H, c.d, c.dv, N), c.device);
  check("kata_fwd_linear_decay",
        kata_fwd_linear_decay(q.ptr, k.ptr, v.ptr, o.ptr, c.n, c.H, c.d, c.dv, q.stride, k.stride, v.stride, o.stride,
                              decay, scale, cu, N, S0, S_out, slots, narrow(n_slots, "n_slots"), resume, zero_outside,
                              c.code, ws.ptr, ws.bytes, guard.stream.stream()));
  written({a[7], a[12]});
  PyObject* out;
  if (a[12] == Py_None) {
    out = THPVariable_Wrap(std::move(held_o));
  } else {
    out = a[12];
    Py_INCREF(out);
  }
  if (!return_state) return out;
  PyObject* S;
  if (a[7] == Py_None) {
    S = THPVariable_Wrap(std::move(held_state));
  } else {
    S = a[7];
    Py_INCREF(S);
  }
  PyObject* both = PyTuple_Pack(2, out, S);
  Py_DECREF(out);
  Py_DECREF(S);
  return both;
  END_HANDLE_TH_ERRORS
}

// q, k, v, dO, log_decay, cu_seqlens, scale, S0, dS_out, return_dS0, workspace, stream
PyObject* bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Lead c = lead(a[0], a[2], "T");
  const Rows q = rows(c.q, "q", c.type, c.n, c.H, c.d, c.device);
  const Rows k = rows(tensor(a[1], "k"), "k", c.type, c.n, c.H, c.d, c.device);
  const Rows v = rows(c.v, "v", c.type, c.n, c.H, c.dv, c.device);
  const void* dO = dense(a[3], "dO", c.type, {c.n, c.H, c.dv}, c.device);
  int N;
  const int* cu = sequences(a[5], c.device, N);
  const int64_t state[4] = {N, c.H, c.d, c.dv};
  const float* decay = static_cast<const float*>(dense(a[4], "log_decay", at::kFloat, {c.H}, c.device));
  const float* S0 = static_cast<const float*>(optional(a[7], "S0", at::kFloat, state, c.device));
  const float* dS = static_cast<const float*>(optional(a[8], "dS_out", at::kFloat, state, c.device));
  const bool return_dS0 = truth(a[9]);
  const float scale = number(a[6]);
  const CallGuard guard(c.device, a[11]);
  Tensor dq = empty({c.n, c.H, c.d}, c.type, c.device), dk = empty({c.n, c.H, c.d}, c.type, c.device);
  Tensor dv = empty({c.n, c.H, c.dv}, c.type, c.device), dS0;
  if (return_dS0) dS0 = empty(state, at::kFloat, c.device);
  const Workspace ws(a[10], kata_bwd_linear_decay_workspace_size(c.n, c.H, c.d, c.dv, N), c.device);
  check("kata_bwd_linear_decay",
        kata_bwd_linear_decay(q.ptr, k.ptr, v.ptr, dO, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), c.n, c.H, c.d, c.dv,
                              q.stride, k.stride, v.stride, decay, scale, cu, N, S0, dS,
                              return_dS0 ? static_cast<float*>(dS0.data_ptr()) : nullptr, c.code, ws.ptr, ws.bytes,
                              guard.stream.stream()));
  PyObject* out = PyTuple_New(return_dS0 ? 4 : 3);
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(dq)));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(dk)));
  PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(std::move(dv)));
  if (return_dS0) PyTuple_SET_ITEM(out, 3, THPVariable_Wrap(std::move(dS0)));
  return out;
  END_HANDLE_TH_ERRORS
}

// q, k, v, S, log_decay, slots, scale, o, stream
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Lead c = lead(a[0], a[2], "n");
  const Rows q = rows(c.q, "q", c.type, c.n, c.H, c.d, c.device);
  const Rows k = rows(tensor(a[1], "k"), "k", c.type, c.n, c.H, c.d, c.device);
  const Rows v = rows(c.v, "v", c.type, c.n, c.H, c.dv, c.device);
  float* S = static_cast<float*>(dense(a[3], "S", at::kFloat, {kAny, c.H, c.d, c.dv}, c.device));
  const int n_slots = narrow(THPVariable_Unpack(a[3]).size(0), "n_slots");
  const float* decay = static_cast<const float*>(dense(a[4], "log_decay", at::kFloat, {c.H}, c.device));
  const int* slots = static_cast<const int*>(optional(a[5], "slots", at::kInt, {c.n}, c.device));
  const float scale = number(a[6]);
  const CallGuard guard(c.device, a[8]);
  Tensor held;
  if (a[7] == Py_None) held = empty({c.n, c.H, c.dv}, c.type, c.device);
  const Tensor& ot = a[7] == Py_None ? held : tensor(a[7], "o");
  const Rows o = rows(ot, "o", c.type, c.n, c.H, c.dv, c.device);
  check("kata_decode_step_linear_decay",
        kata_decode_step_linear_decay(q.ptr, k.ptr, v.ptr, o.ptr, S, c.n, c.H, c.d, c.dv, q.stride, k.stride, v.stride,
                                      o.stride, decay, scale, slots, n_slots, c.code, guard.stream.stream()));
  written({a[3], a[7]});
  if (a[7] == Py_None) return THPVariable_Wrap(std::move(held));
  Py_INCREF(a[7]);
  return a[7];
  END_HANDLE_TH_ERRORS
}

// The pool of states and the cache of a store or a load.
struct Pools {
  float *S, *z, *scale, *z_cache;
  signed char* cache;
  const int *slots, *entries;
  int n_slots, n_entries, n, H, rows, dv;
  at::Device device;
};
Pools pools(PyObject* S, PyObject* cache, PyObject* scale, PyObject* slots, PyObject* entries, PyObject* z,
            PyObject* z_cache) {
  const Tensor& s = tensor(S, "S");
  TORCH_CHECK_VALUE(s.dim() == 4, "S must be [n_slots, H, rows, dv], got ", s.sizes());
  TORCH_CHECK_VALUE(THPVariable_Check(cache) && THPVariable_Unpack(cache).dim() == 4,
                    "cache must be an int8 tensor [n_entries, H, rows, dv]");
  TORCH_CHECK_VALUE((z == Py_None) == (z_cache == Py_None), "z and z_cache: both or neither");
  const at::Device device = s.device();
  const int64_t n_slots = s.size(0), n_entries = THPVariable_Unpack(cache).size(0);
  const int64_t H = s.size(1), r = s.size(2), dv = s.size(3);
  int64_t n = std::min(n_slots, n_entries);
  for (PyObject* o : {entries, slots})
    if (o != Py_None) n = tensor(o, o == slots ? "slots" : "entries").numel();
  return Pools{static_cast<float*>(dense(S, "S", at::kFloat, {n_slots, H, r, dv}, device)),
               static_cast<float*>(optional(z, "z", at::kFloat, {n_slots, H, r}, device)),
               static_cast<float*>(dense(scale, "scale", at::kFloat, {n_entries, H, r}, device)),
               static_cast<float*>(optional(z_cache, "z_cache", at::kFloat, {n_entries, H, r}, device)),
               static_cast<signed char*>(dense(cache, "cache", at::kChar, {n_entries, H, r, dv}, device)),
               static_cast<const int*>(optional(slots, "slots", at::kInt, {n}, device)),
               static_cast<const int*>(optional(entries, "entries", at::kInt, {n}, device)),
               narrow(n_slots, "n_slots"),
               narrow(n_entries, "n_entries"),
               narrow(n, "n"),
               narrow(H, "H"),
               narrow(r, "rows"),
               narrow(dv, "dv"),
               device};
}

// S, cache, scale, slots, entries, z, z_cache, stream
PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Pools p = pools(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
  const CallGuard guard(p.device, a[7]);
  check("kata_state_store_q8",
        kata_state_store_q8(p.S, p.z, p.n_slots, p.cache, p.scale, p.z_cache, p.n_entries, p.slots, p.entries, p.n, p.H,
                            p.rows, p.dv, guard.stream.stream()));
  written({a[1], a[2], a[6]});
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// cache, scale, S, entries, slots, z, z_cache, stream
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Pools p = pools(a[2], a[0], a[1], a[4], a[3], a[5], a[6]);
  const CallGuard guard(p.device, a[7]);
  check("kata_state_load_q8",
        kata_state_load_q8(p.cache, p.scale, p.z_cache, p.n_entries, p.S, p.z, p.n_slots, p.entries, p.slots, p.n, p.H,
                           p.rows, p.dv, guard.stream.stream()));
  written({a[2], a[5]});
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(kata_error, type);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"fwd", reinterpret_cast<PyCFunction>(fwd), METH_FASTCALL, nullptr},
    {"bwd", reinterpret_cast<PyCFunction>(bwd), METH_FASTCALL, nullptr},
    {"step", reinterpret_cast<PyCFunction>(step), METH_FASTCALL, nullptr},
    {"store", reinterpret_cast<PyCFunction>(store), METH_FASTCALL, nullptr},
    {"load", reinterpret_cast<PyCFunction>(load), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
