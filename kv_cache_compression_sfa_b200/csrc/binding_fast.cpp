// binding_fast.cpp — the per-step calls of the paged cache from Python without
// ctypes: the checks of the binding and the C call in one step.
//
// Every function returns the C call's status, or None if an argument is not
// exactly what the call takes (then nothing has been enqueued, and the caller's
// Python checks say what is wrong).  A call of five tensors costs about 1 us
// here and 8 us through attribute checks and ctypes, which is as long as the
// small kernels that it launches.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <new>

#include "sfa.h"

namespace {

using PlanFn = decltype(&sfa_tree_plan);
using AppendFn = decltype(&sfa_kv_append);
using AttendFn = decltype(&sfa_kv_attend);
using AcceptFn = decltype(&sfa_kv_accept);
using BytesFn = decltype(&sfa_kv_attend_workspace_bytes);

// What the calls of one cache share.
struct Spec {
  AppendFn append;
  AttendFn attend;
  AcceptFn accept;
  BytesFn attend_bytes;
  const sfa_kv_cache* cache;  // owned by the Python object that keeps this spec
  int device;
  at::ScalarType dtype;
  int64_t batch, nq, nkv, d;
};

const char kName[] = "sfa_spec";

Spec* spec_of(PyObject* o) { return static_cast<Spec*>(PyCapsule_GetPointer(o, kName)); }

void free_spec(PyObject* o) { delete spec_of(o); }

// A contiguous tensor on the device with this dtype and shape; its pointer into
// *out.  None gives null where it is allowed.
bool take(PyObject* o, at::ScalarType dtype, int device, std::initializer_list<int64_t> shape, bool optional, void** out) {
  if (o == Py_None) {
    *out = nullptr;
    return optional;
  }
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != dtype || !t.device().is_cuda() || t.device().index() != device || !t.is_contiguous()) return false;
  const auto s = t.sizes();
  if (s.size() != shape.size()) return false;
  size_t i = 0;
  for (int64_t v : shape)
    if (s[i++] != v) return false;
  *out = t.data_ptr();
  return true;
}

bool dims(PyObject* o, size_t n, const at::Tensor** t) {
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return (*t)->sizes().size() == n && (*t)->device().is_cuda();
}

// The stream's handle: None is the device's current one, else an integer.
bool stream_of(PyObject* o, int device, void** out) {
  if (c10::cuda::current_device() != device) return false;
  if (o == Py_None) {
    *out = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    return true;
  }
  *out = PyLong_AsVoidPtr(o);
  return !PyErr_Occurred();
}

const sfa_handle* handle_of(PyObject* o) {
  return o == Py_None ? nullptr : static_cast<const sfa_handle*>(PyLong_AsVoidPtr(o));
}

PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

#define CALL(expr)              \
  int rc;                       \
  Py_BEGIN_ALLOW_THREADS        \
  rc = (expr);                  \
  Py_END_ALLOW_THREADS          \
  return PyLong_FromLong(rc);

// spec(append, attend, accept, attend_bytes, cache, device, is_bf16, batch, nq, nkv, d)
PyObject* make_spec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) return none();
  Spec* s = new (std::nothrow) Spec;
  if (!s) return PyErr_NoMemory();
  s->append = reinterpret_cast<AppendFn>(PyLong_AsVoidPtr(a[0]));
  s->attend = reinterpret_cast<AttendFn>(PyLong_AsVoidPtr(a[1]));
  s->accept = reinterpret_cast<AcceptFn>(PyLong_AsVoidPtr(a[2]));
  s->attend_bytes = reinterpret_cast<BytesFn>(PyLong_AsVoidPtr(a[3]));
  s->cache = static_cast<const sfa_kv_cache*>(PyLong_AsVoidPtr(a[4]));
  s->device = static_cast<int>(PyLong_AsLong(a[5]));
  s->dtype = PyObject_IsTrue(a[6]) ? at::kBFloat16 : at::kFloat;
  s->batch = PyLong_AsLongLong(a[7]);
  s->nq = PyLong_AsLongLong(a[8]);
  s->nkv = PyLong_AsLongLong(a[9]);
  s->d = PyLong_AsLongLong(a[10]);
  if (PyErr_Occurred()) {
    delete s;
    return nullptr;
  }
  return PyCapsule_New(s, kName, free_spec);
}

// plan(fn, handle, parents, ctx, lens, positions, mask, stream)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor* par;
  if (n != 8 || !dims(a[2], 2, &par)) return none();
  const int dev = par->device().index();
  const int64_t B = par->size(0), m = par->size(1);
  if (m > INT32_MAX || B > INT32_MAX) return none();
  void *pp, *cp, *lp, *op, *mp, *st;
  if (!take(a[2], at::kInt, dev, {B, m}, false, &pp) || !take(a[3], at::kInt, dev, {B}, false, &cp) ||
      !take(a[4], at::kInt, dev, {B}, true, &lp) || !take(a[5], at::kInt, dev, {B, m}, false, &op) ||
      !take(a[6], at::kInt, dev, {B, m, (m + 31) / 32}, false, &mp) || !stream_of(a[7], dev, &st))
    return none();
  const PlanFn fn = reinterpret_cast<PlanFn>(PyLong_AsVoidPtr(a[0]));
  const sfa_handle* h = handle_of(a[1]);
  if (PyErr_Occurred() || !fn) return none();
  CALL(fn(h, static_cast<const int*>(pp), static_cast<int>(m), static_cast<const int*>(lp), static_cast<const int*>(cp),
          static_cast<int>(B), static_cast<int*>(op), static_cast<uint32_t*>(mp), st))
}

// append(spec, handle, layer_begin, q, k, v, ctx, lens, positions, rope, q_out, k_out, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor* k;
  if (n != 13 || !dims(a[4], 5, &k)) return none();
  const Spec* s = spec_of(a[0]);
  if (!s) return none();
  const int64_t L = k->size(0), B = s->batch, m = k->size(2);
  if (L > INT32_MAX || m > INT32_MAX) return none();
  void *qp, *kp, *vp, *cp, *lp, *pp, *qo, *ko, *st;
  const auto dt = s->dtype;
  const int dev = s->device;
  if (!take(a[3], dt, dev, {L, B, m, s->nq, s->d}, true, &qp) || !take(a[4], dt, dev, {L, B, m, s->nkv, s->d}, false, &kp) ||
      !take(a[5], dt, dev, {L, B, m, s->nkv, s->d}, false, &vp) || !take(a[6], at::kInt, dev, {B}, false, &cp) ||
      !take(a[7], at::kInt, dev, {B}, true, &lp) || !take(a[8], at::kInt, dev, {B, m}, true, &pp) ||
      !take(a[10], dt, dev, {L, B, m, s->nq, s->d}, true, &qo) || !take(a[11], dt, dev, {L, B, m, s->nkv, s->d}, true, &ko) ||
      (qp == nullptr) != (qo == nullptr) || !stream_of(a[12], dev, &st))
    return none();
  const sfa_handle* h = handle_of(a[1]);
  const long l0 = PyLong_AsLong(a[2]);
  const sfa_rope* rope = a[9] == Py_None ? nullptr : static_cast<const sfa_rope*>(PyLong_AsVoidPtr(a[9]));
  if (PyErr_Occurred() || l0 < INT32_MIN || l0 > INT32_MAX) return none();
  CALL(s->append(h, s->cache, static_cast<int>(l0), static_cast<int>(L), qp, kp, vp, static_cast<int>(m),
                 static_cast<const int*>(lp), static_cast<const int*>(cp), static_cast<const int*>(pp), rope,
                 static_cast<int>(B), qo, ko, st))
}

// A workspace for the length of one call, from the pool of the call's stream: what
// is enqueued there later may have the memory again, and a capture there takes it
// from the graph's pool.
struct Scratch {
  void* p = nullptr;
  ~Scratch() {
    if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
};

// attend(spec, handle, layer_begin, q, ctx, lens, mask, out, workspace or None, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor *q, *w = nullptr;
  if (n != 10 || !dims(a[3], 5, &q) || (a[8] != Py_None && !dims(a[8], 1, &w))) return none();
  const Spec* s = spec_of(a[0]);
  if (!s) return none();
  const int64_t L = q->size(0), B = s->batch, m = q->size(2);
  if (L > INT32_MAX || m > INT32_MAX) return none();
  void *qp, *cp, *lp, *mp, *op, *wp = nullptr, *st;
  const auto dt = s->dtype;
  const int dev = s->device;
  if (!take(a[3], dt, dev, {L, B, m, s->nq, s->d}, false, &qp) || !take(a[4], at::kInt, dev, {B}, false, &cp) ||
      !take(a[5], at::kInt, dev, {B}, true, &lp) || !take(a[6], at::kInt, dev, {B, m, (m + 31) / 32}, true, &mp) ||
      !take(a[7], dt, dev, {L, B, m, s->nq * s->d}, false, &op) ||
      (w && !take(a[8], at::kByte, dev, {w->size(0)}, false, &wp)) || !stream_of(a[9], dev, &st))
    return none();
  const sfa_handle* h = handle_of(a[1]);
  const long l0 = PyLong_AsLong(a[2]);
  if (PyErr_Occurred() || l0 < INT32_MIN || l0 > INT32_MAX) return none();
  Scratch own;
  size_t bytes = w ? static_cast<size_t>(w->size(0)) : s->attend_bytes(h, static_cast<int>(m));
  if (!w && bytes > 0) {
    try {
      own.p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, static_cast<cudaStream_t>(st));
    } catch (const std::exception&) {
      return none();  // the caller's own way raises torch's error
    }
    wp = own.p;
  }
  CALL(s->attend(h, s->cache, static_cast<int>(l0), static_cast<int>(L), qp, static_cast<int>(m),
                 static_cast<const int*>(lp), static_cast<const int*>(cp), static_cast<const uint32_t*>(mp),
                 static_cast<int>(B), op, wp, bytes, st))
}

// accept(spec, handle, layer_begin, layer_count, path, n_accept, ctx, stream)
PyObject* accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor* path;
  if (n != 8 || !dims(a[4], 2, &path)) return none();
  const Spec* s = spec_of(a[0]);
  if (!s) return none();
  const int64_t B = s->batch, m = path->size(1);
  if (m > INT32_MAX) return none();
  void *pp, *np, *cp, *st;
  const int dev = s->device;
  if (!take(a[4], at::kInt, dev, {B, m}, false, &pp) || !take(a[5], at::kInt, dev, {B}, false, &np) ||
      !take(a[6], at::kInt, dev, {B}, false, &cp) || !stream_of(a[7], dev, &st))
    return none();
  const sfa_handle* h = handle_of(a[1]);
  const long l0 = PyLong_AsLong(a[2]), lc = PyLong_AsLong(a[3]);
  if (PyErr_Occurred() || l0 < INT32_MIN || l0 > INT32_MAX || lc < INT32_MIN || lc > INT32_MAX) return none();
  CALL(s->accept(h, s->cache, static_cast<int>(l0), static_cast<int>(lc), static_cast<const int*>(pp), static_cast<int>(m),
                 static_cast<const int*>(np), static_cast<const int*>(cp), static_cast<int>(B), st))
}

// Runs a call; no C++ exception leaves the module.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<fn>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD("spec", make_spec), METHOD("plan", plan), METHOD("append", append),
                          METHOD("attend", attend), METHOD("accept", accept), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "built_for", SFA_BUILT_FOR) < 0) {  // torch and Python, by the build
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
