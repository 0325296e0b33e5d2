// Python face of the per-layer calls pa_rope_and_cache, pa_diff_attention and pa_move_blocks:
// torch tensors -> pa_tensor descriptors, the current stream, the status back.  Marshalling only
// (the C ABI itself knows no torch types).  A serving step makes these calls once per layer, and a
// small batch's kernel takes a few microseconds: describing eight tensors field by field through
// ctypes takes 20, here 0.3.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>

#include "pa.h"

namespace {

// The library's entry points: the addresses the binding found in the library it loaded.
struct Api {
  decltype(&pa_rope_and_cache) rope;
  decltype(&pa_diff_attention_workspace_size) diff_size;
  decltype(&pa_diff_attention) diff;
  decltype(&pa_move_plan_create) plan_create;
  decltype(&pa_move_plan_destroy) plan_destroy;
  decltype(&pa_move_blocks_workspace_size) move_size;
  decltype(&pa_move_blocks) move;
} api = {};

// A Python error is set; unwinds to the entry.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Raised();
}

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "expected a torch.Tensor");
  return THPVariable_Unpack(o);
}

int32_t code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kHalf: return PA_F16;
    case at::kBFloat16: return PA_BF16;
    case at::kFloat: return PA_F32;
    case at::kInt: return PA_I32;
    case at::kLong: return PA_I64;
    case at::kByte:
    case at::kFloat8_e4m3fn: return PA_F8E4M3;
    default: raise(PyExc_TypeError, "unsupported dtype");
  }
}

// Descriptors of a call's tensors, which all have to be on the current device.
struct Described {
  pa_tensor t[9];
  int n = 0;
  int device = -1;
  pa_tensor* add(const at::Tensor& x) {
    if (!x.is_cuda() || (device >= 0 && x.get_device() != device))
      raise(PyExc_ValueError, "every tensor must be on the current CUDA device");
    if (device < 0) {
      device = x.get_device();
      if (device != c10::cuda::current_device())
        raise(PyExc_ValueError, "every tensor must be on the current CUDA device");
    }
    if (x.dim() > PA_MAX_DIMS) raise(PyExc_ValueError, "rank above 5");
    pa_tensor& d = t[n++];
    d.data = x.numel() > 0 ? x.data_ptr() : nullptr;
    d.dtype = code(x);
    d.ndim = static_cast<int32_t>(x.dim());
    for (int i = 0; i < d.ndim; ++i) {
      d.shape[i] = x.size(i);
      d.stride[i] = x.stride(i);
    }
    return &d;
  }
  pa_tensor* add(PyObject* o) { return add(tensor(o)); }
};

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised();
  return x;
}

int32_t integer(PyObject* o) {
  int overflow = 0;
  const long x = PyLong_AsLongAndOverflow(o, &overflow);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  if (overflow || x < INT32_MIN || x > INT32_MAX) raise(PyExc_OverflowError, "int32 expected");
  return static_cast<int32_t>(x);
}

void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised();
  return p;
}

// A stream handle, or the current stream of the device for None.
void* stream_of(PyObject* o, int device) {
  return o == Py_None ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(device).stream())
                      : address(o);
}

// The caller's workspace, or one of `need` bytes (from torch's allocator, on the current stream).
struct Workspace {
  at::Tensor held;
  void* data = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, size_t need, int device) {
    if (o == Py_None) {
      if (need == 0) return;
      held = at::empty({static_cast<int64_t>(need)},
                       at::TensorOptions().dtype(at::kByte).device(at::kCUDA, device));
    } else {
      held = tensor(o);
      if (!held.is_cuda() || held.get_device() != device)
        raise(PyExc_ValueError, "every tensor must be on the current CUDA device");
      if (!held.is_contiguous()) raise(PyExc_ValueError, "the workspace must be contiguous");
    }
    data = held.data_ptr();
    bytes = held.nbytes();
  }
};

template <typename F>
int unlocked(F f) {  // the call may wait for room in the launch queue
  PyThreadState* s = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(s);
  return status;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
    if (!api.rope) raise(PyExc_RuntimeError, "the library is not loaded");
    return f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

const void* host_vector(PyObject* o, at::ScalarType type, int64_t n, const char* text) {
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != type || !t.device().is_cpu() || t.dim() != 1 || t.numel() != n ||
      !t.is_contiguous())
    raise(PyExc_ValueError, text);
  return t.data_ptr();
}

// q, k, v, positions, inv_freq, k_cache, v_cache, slot_mapping, q_out, axes, adjacent, factor,
// stream, k_scale, v_scale -> status
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const int64_t pairs = tensor(a[4]).numel();
    pa_rope r{};
    r.num_pairs = static_cast<int32_t>(pairs);
    r.inv_freq = static_cast<const double*>(host_vector(
        a[4], at::kDouble, pairs, "inv_freq must be a contiguous host float64 vector"));
    if (a[9] != Py_None)
      r.axis_of_pair = static_cast<const int32_t*>(host_vector(
          a[9], at::kInt, pairs, "axes must be a contiguous host int32 vector, one entry per pair"));
    r.adjacent = PyObject_IsTrue(a[10]) == 1;
    r.factor = static_cast<float>(number(a[11]));
    Described d;
    pa_tensor *q = d.add(a[0]), *k = d.add(a[1]), *v = d.add(a[2]);
    at::Tensor positions = tensor(a[3]);
    if (positions.dim() == 1) positions = positions.unsqueeze(0);
    pa_tensor *p = d.add(positions), *kc = d.add(a[5]), *vc = d.add(a[6]);
    pa_tensor *slots = d.add(a[7]), *qo = d.add(a[8]);
    pa_kv_scales sc{};
    const bool fp8 = kc->dtype == PA_F8E4M3;
    if (fp8) {
      sc.k_scale = static_cast<float>(number(a[13]));
      sc.v_scale = static_cast<float>(number(a[14]));
    }
    void* st = stream_of(a[12], d.device);
    return PyLong_FromLong(unlocked([&] {
      return api.rope(q, k, v, p, &r, kc, vc, slots, qo, fp8 ? &sc : nullptr, st);
    }));
  });
}

// q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, lam, out, max_query_len,
// max_seq_len, norm_weight, eps, out_scale, workspace, stream, num_prefill_seqs -> status
PyObject* diff(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    Described d;
    pa_tensor *q = d.add(a[0]), *kc = d.add(a[1]), *vc = d.add(a[2]), *bt = d.add(a[3]);
    pa_tensor *sl = d.add(a[4]), *qsl = d.add(a[5]), *lam = d.add(a[7]), *out = d.add(a[8]);
    pa_diff p{};
    p.lambda = lam;
    p.norm_weight = a[11] != Py_None ? d.add(a[11]) : nullptr;
    p.eps = static_cast<float>(number(a[12]));
    p.out_scale = static_cast<float>(number(a[13]));
    const float scale = static_cast<float>(number(a[6]));
    const pa_batch_hint hint{integer(a[9]), integer(a[10]), integer(a[16]), 0};
    const size_t need = a[14] == Py_None && q->ndim == 3 && kc->ndim == 4 && sl->ndim == 1
                            ? api.diff_size(q->shape[0], sl->shape[0], q->shape[1], kc->shape[1],
                                            q->shape[2], &hint)
                            : 0;
    Workspace ws(a[14], need, d.device);
    void* st = stream_of(a[15], d.device);
    return PyLong_FromLong(unlocked([&] {
      return api.diff(q, kc, vc, bt, sl, qsl, scale, &p, out, &hint, ws.data, ws.bytes, st);
    }));
  });
}

// plan (handle, or host int32 [n, 2] pairs), k_cache, v_cache, block_tables, workspace, stream -> status, or -1 when the pairs make no plan
PyObject* move(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    Described d;
    pa_tensor *kc = d.add(a[1]), *vc = d.add(a[2]);
    pa_tensor* bt = a[3] != Py_None ? d.add(a[3]) : nullptr;
    struct Plan {
      pa_move_plan* p = nullptr;
      bool own = false;
      ~Plan() {
        if (own) api.plan_destroy(p);
      }
    } plan;
    if (PyLong_Check(a[0])) {
      plan.p = static_cast<pa_move_plan*>(address(a[0]));
    } else {
      const at::Tensor& t = tensor(a[0]);
      if (t.scalar_type() != at::kInt || !t.device().is_cpu() || t.dim() != 2 || t.size(1) != 2 ||
          !t.is_contiguous())
        raise(PyExc_ValueError, "pairs must be a contiguous host int32 [n, 2] tensor");
      plan.p = api.plan_create(static_cast<const int32_t*>(t.data_ptr()), t.size(0),
                               kc->ndim >= 4 ? kc->shape[kc->ndim - 4] : 0);
      plan.own = true;
      if (!plan.p) return PyLong_FromLong(-1);
    }
    size_t need = 0;
    if (a[4] == Py_None && (need = api.move_size(plan.p, kc, 1, bt != nullptr)) > 0) {
      // room to stage several layers per launch, up to 256 MB
      const size_t layer = api.move_size(plan.p, kc, 2, bt != nullptr) - need;
      const int64_t layers = kc->ndim == 5 ? kc->shape[0] : 1;
      if (layer > 0)
        need += layer * (std::min<int64_t>(layers, std::max<int64_t>(1, (256 << 20) / layer)) - 1);
    }
    Workspace ws(a[4], need, d.device);
    void* st = stream_of(a[5], d.device);
    return PyLong_FromLong(
        unlocked([&] { return api.move(plan.p, kc, vc, bt, ws.data, ws.bytes, st); }));
  });
}

// Addresses in the order of Api.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "seven addresses expected");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "address is NULL");
      return nullptr;
    }
  api.rope = reinterpret_cast<decltype(api.rope)>(p[0]);
  api.diff_size = reinterpret_cast<decltype(api.diff_size)>(p[1]);
  api.diff = reinterpret_cast<decltype(api.diff)>(p[2]);
  api.plan_create = reinterpret_cast<decltype(api.plan_create)>(p[3]);
  api.plan_destroy = reinterpret_cast<decltype(api.plan_destroy)>(p[4]);
  api.move_size = reinterpret_cast<decltype(api.move_size)>(p[5]);
  api.move = reinterpret_cast<decltype(api.move)>(p[6]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, "Set the library's entry points."},
                         {"rope", fast(rope), METH_FASTCALL, "pa_rope_and_cache"},
                         {"diff", fast(diff), METH_FASTCALL, "pa_diff_attention"},
                         {"move", fast(move), METH_FASTCALL, "pa_move_blocks"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_pa_torch", "Tensor marshalling.", -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_torch(void) { return PyModule_Create(&module_def); }
