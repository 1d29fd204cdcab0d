// tail_binding.cpp -- Python calls of include/strata_tail.h on PyTorch tensors.
//
// Checks what the C ABI cannot see (types, shapes, devices of tensors), allocates the outputs that the
// caller left out, and makes the C call on the tensors' addresses without holding the interpreter's lock.
// It is compiled because the smallest calls' kernels take 2 to 5 us: the same steps in Python took 20 us
// a call on a Grace core, most of it in cold attribute look-ups.  A C error code is returned as an int,
// which the Python side turns into StrataError.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/strata_tail.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A refusal on the way: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* name, const char* what) {
  PyErr_Format(type, "%s %s", name, what);
  throw Refused();
}

const Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, "must be a tensor");
  return &THPVariable_Unpack(o);
}

const Tensor& needed(PyObject* o, const char* name) {
  const Tensor* t = tensor(o, name);
  if (t == nullptr) refuse(PyExc_TypeError, name, "must be a tensor");
  return *t;
}

struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};

void check(const Tensor& t, const char* name, ScalarType type, int device) {
  if (t.scalar_type() != type) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    throw Refused();
  }
  if (!t.is_cuda() || t.get_device() != device) refuse(PyExc_ValueError, name, "must be a CUDA tensor on the call's device");
}

// A [rows, width] tensor whose rows are contiguous, any distance apart.
Rows rows(const Tensor* t, const char* name, int64_t n, int64_t width, ScalarType type, int device) {
  if (t == nullptr) return {};
  check(*t, name, type, device);
  if (t->dim() != 2 || t->size(0) != n || t->size(1) != width) {
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld]", name, static_cast<long long>(n), static_cast<long long>(width));
    throw Refused();
  }
  if (width > 1 && t->stride(1) != 1) refuse(PyExc_ValueError, name, "must have contiguous rows");
  return {t->data_ptr(), n > 1 ? t->stride(0) : width};  // the stride of one row means nothing
}

// A packed tensor of that shape.
void* dense(const Tensor* t, const char* name, std::initializer_list<int64_t> shape, ScalarType type, int device) {
  if (t == nullptr) return nullptr;
  check(*t, name, type, device);
  if (t->sizes() != at::IntArrayRef(shape)) refuse(PyExc_ValueError, name, "has another shape than the call's");
  if (!t->is_contiguous()) refuse(PyExc_ValueError, name, "must be contiguous");
  return t->data_ptr();
}

int call_device(const Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(PyExc_ValueError, name, "must be [rows, width]");
  if (!t.is_cuda()) refuse(PyExc_ValueError, name, "must be a CUDA tensor");
  const int device = t.get_device();
  if (device != c10::cuda::current_device()) refuse(PyExc_ValueError, name, "must be on the current device");
  return device;
}

int narrow(int64_t v, const char* name) {
  if (v < 0 || v > INT32_MAX) refuse(PyExc_ValueError, name, "is out of range");
  return static_cast<int>(v);
}

void* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  void* s = PyLong_AsVoidPtr(o);
  if (s == nullptr && PyErr_Occurred()) throw Refused();
  return s;
}

Tensor fresh(at::IntArrayRef shape, ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

PyObject* done(int rc, PyObject* result) {
  if (rc == STRATA_OK) return result;
  Py_XDECREF(result);
  return PyLong_FromLong(rc);
}

void put(PyObject* dict, const char* key, const Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  const int bad = o == nullptr || PyDict_SetItemString(dict, key, o) != 0;
  Py_XDECREF(o);
  if (bad) throw Refused();
}

void arguments(Py_ssize_t got, Py_ssize_t wanted) {
  if (got == wanted) return;
  PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", wanted, got);
  throw Refused();
}

#define TAIL_CALL(name)                                                    \
  PyObject* name##_body(PyObject* const* a, Py_ssize_t n);                 \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {            \
    HANDLE_TH_ERRORS                                                       \
    try {                                                                  \
      return name##_body(a, n);                                            \
    } catch (const Refused&) {                                             \
      return nullptr;                                                      \
    }                                                                      \
    END_HANDLE_TH_ERRORS                                                   \
  }                                                                        \
  PyObject* name##_body(PyObject* const* a, Py_ssize_t n)

// (x, weight, residual, eps, want residual, want y, want 8 bits, out, stream) -> out, a dict
TAIL_CALL(norm) {
  arguments(n, 9);
  const Tensor &x = needed(a[0], "x"), &weight = needed(a[1], "weight");
  const Tensor* residual = tensor(a[2], "residual");
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Refused();
  const ScalarType type = x.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) refuse(PyExc_TypeError, "x", "must be float32 or bfloat16");
  const int device = call_device(x, "x");
  const int64_t T = x.size(0), H = x.size(1);
  PyObject* out = a[7];
  if (!PyDict_Check(out)) refuse(PyExc_TypeError, "out", "must be a dict");
  auto output = [&](const char* key, bool wanted, at::IntArrayRef shape, ScalarType t) -> Tensor {
    PyObject* given = PyDict_GetItemString(out, key);
    if (given != nullptr && given != Py_None) return needed(given, key);
    if (!wanted) return Tensor();
    Tensor made = fresh(shape, t, x);
    put(out, key, made);
    return made;
  };
  const bool f8 = a[6] == Py_True;
  const Tensor ro = output("residual", a[4] == Py_True, {T, H}, type), y = output("y", a[5] == Py_True, {T, H}, type),
               q = output("q", f8, {T, H}, at::kFloat8_e4m3fn), scale = output("scale", f8, {T}, at::kFloat);
  auto given = [](const Tensor& t) { return t.defined() ? &t : nullptr; };
  const Rows rx = rows(&x, "x", T, H, type, device), rr = rows(residual, "residual", T, H, type, device),
             rro = rows(given(ro), "residual", T, H, type, device), ry = rows(given(y), "y", T, H, type, device),
             rq = rows(given(q), "q", T, H, at::kFloat8_e4m3fn, device);
  void *pw = dense(&weight, "weight", {H}, type, device), *ps = dense(given(scale), "scale", {T}, at::kFloat, device);
  void* stream = stream_of(a[8], device);
  const int t32 = narrow(T, "T"), h32 = narrow(H, "H");
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = strata_norm_rows(rx.p, rx.ld, rr.p, rr.ld, pw, type == at::kFloat ? STRATA_DTYPE_F32 : STRATA_DTYPE_BF16, t32, h32,
                        static_cast<float>(eps), rro.p, rro.ld, ry.p, ry.ld, rq.p, rq.ld, static_cast<float*>(ps), stream);
  Py_END_ALLOW_THREADS
  Py_INCREF(out);
  return done(rc, out);
}

// (x, w, x_scale, w_scale, a, b, row_adapter, adapter_scale, y or None, workspace, allocate it, stream) -> y
TAIL_CALL(project) {
  arguments(n, 12);
  const Tensor &x = needed(a[0], "x"), &w = needed(a[1], "w");
  const Tensor *x_scale = tensor(a[2], "x_scale"), *w_scale = tensor(a[3], "w_scale"), *pa = tensor(a[4], "a"),
               *pb = tensor(a[5], "b"), *of = tensor(a[6], "row_adapter"), *by = tensor(a[7], "adapter_scale"),
               *y_given = tensor(a[8], "y"), *ws_given = tensor(a[9], "workspace");
  const ScalarType type = x.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat8_e4m3fn) refuse(PyExc_TypeError, "x", "must be bfloat16 or float8_e4m3fn");
  const int device = call_device(x, "x");
  if (w.dim() != 2) refuse(PyExc_ValueError, "w", "must be [outputs, width]");
  const int64_t T = x.size(0), K = x.size(1), N = w.size(0);
  const Rows rx = rows(&x, "x", T, K, type, device), rw = rows(&w, "w", N, K, type, device);
  float *sx = static_cast<float*>(dense(x_scale, "x_scale", {T}, at::kFloat, device)),
        *sw = static_cast<float*>(dense(w_scale, "w_scale", {N}, at::kFloat, device));
  int64_t S = 0, R = 0, bytes = 0;
  void *va = nullptr, *vb = nullptr, *vof = nullptr, *vby = nullptr, *vws = nullptr;
  Tensor ws;
  if (pa != nullptr || pb != nullptr) {
    if (pa == nullptr || pb == nullptr || of == nullptr || by == nullptr)
      refuse(PyExc_ValueError, "a, b, row_adapter and adapter_scale", "go together");
    if (pa->dim() != 3) refuse(PyExc_ValueError, "a", "must be [adapters, rank, width]");
    S = pa->size(0);
    R = pa->size(1);
    va = dense(pa, "a", {S, R, K}, at::kBFloat16, device);
    vb = dense(pb, "b", {S, N, R}, at::kBFloat16, device);
    vof = dense(of, "row_adapter", {T}, at::kInt, device);
    vby = dense(by, "adapter_scale", {S}, at::kFloat, device);
    if (ws_given != nullptr) {
      bytes = ws_given->numel();
      vws = dense(ws_given, "workspace", {bytes}, at::kByte, device);
    } else if (a[10] == Py_True) {
      bytes = strata_project_workspace(narrow(T, "T"), narrow(S, "S"), narrow(R, "R"));
      if (bytes > 0) {
        ws = fresh({bytes}, at::kByte, x);
        vws = ws.data_ptr();
      }
    }
  }
  // rows start on 16 bytes, as draw_rows and the sampler want them (narrow() would take a microsecond and more)
  const int64_t ld = (N + 7) / 8 * 8;
  const Tensor y = y_given != nullptr ? *y_given : fresh({T, ld}, at::kBFloat16, x);
  if (y_given == nullptr && ld != N) y.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef({T, N}), at::IntArrayRef({ld, int64_t{1}}));
  const Rows ry = rows(&y, "y", T, N, at::kBFloat16, device);
  void* stream = stream_of(a[11], device);
  const int t32 = narrow(T, "T"), n32 = narrow(N, "N"), k32 = narrow(K, "K"), s32 = narrow(S, "S"), r32 = narrow(R, "R");
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = strata_project_rows(rx.p, rx.ld, sx, rw.p, rw.ld, sw, type == at::kBFloat16 ? STRATA_DTYPE_BF16 : STRATA_DTYPE_F8, t32,
                           n32, k32, va, vb, s32, r32, static_cast<int32_t*>(vof), static_cast<float*>(vby), ry.p, ry.ld, vws,
                           bytes, stream);
  Py_END_ALLOW_THREADS
  return done(rc, rc == STRATA_OK ? THPVariable_Wrap(y) : nullptr);
}

// (logits, u, temperature, top_k, top_p, min_p, V or None, want ids, want lps, out, stream) -> out, a dict
TAIL_CALL(draw) {
  arguments(n, 11);
  const Tensor &logits = needed(a[0], "logits"), &u = needed(a[1], "u");
  const Tensor *t = tensor(a[2], "temperature"), *k = tensor(a[3], "top_k"), *p = tensor(a[4], "top_p"), *m = tensor(a[5], "min_p");
  const ScalarType type = logits.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) refuse(PyExc_TypeError, "logits", "must be float32 or bfloat16");
  const int device = call_device(logits, "logits");
  const int64_t B = logits.size(0), width = logits.size(1);
  int64_t V = width;
  if (a[6] != Py_None) {
    V = PyLong_AsLongLong(a[6]);
    if (V == -1 && PyErr_Occurred()) throw Refused();
    // the C call can only compare V with the stride, which may reach past the tensor
    if (V < 1 || V > width) refuse(PyExc_ValueError, "V", "must be 1 to the logits' width");
  }
  Rows rl = rows(&logits, "logits", B, width, type, device);
  if (B <= 1) rl.ld = (rl.ld + 7) / 8 * 8;
  PyObject* out = a[9];
  if (!PyDict_Check(out)) refuse(PyExc_TypeError, "out", "must be a dict");
  auto output = [&](const char* key, bool wanted, ScalarType type) -> Tensor {
    PyObject* given = PyDict_GetItemString(out, key);
    if (given != nullptr && given != Py_None) return needed(given, key);
    if (!wanted) return Tensor();
    Tensor made = fresh({B}, type, logits);
    put(out, key, made);
    return made;
  };
  const Tensor ids = output("ids", a[7] == Py_True, at::kInt), lps = output("lps", a[8] == Py_True, at::kFloat);
  auto given = [](const Tensor& v) { return v.defined() ? &v : nullptr; };
  auto vector = [&](const Tensor* v, const char* name, ScalarType type) { return dense(v, name, {B}, type, device); };
  float *vu = static_cast<float*>(vector(&u, "u", at::kFloat)), *vt = static_cast<float*>(vector(t, "temperature", at::kFloat)),
        *vp = static_cast<float*>(vector(p, "top_p", at::kFloat)), *vm = static_cast<float*>(vector(m, "min_p", at::kFloat)),
        *vlps = static_cast<float*>(vector(given(lps), "lps", at::kFloat));
  int32_t *vk = static_cast<int32_t*>(vector(k, "top_k", at::kInt)), *vids = static_cast<int32_t*>(vector(given(ids), "ids", at::kInt));
  void* stream = stream_of(a[10], device);
  const int b32 = narrow(B, "B"), v32 = narrow(V, "V");
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = strata_draw_rows(rl.p, type == at::kFloat ? STRATA_DTYPE_F32 : STRATA_DTYPE_BF16, b32, v32, rl.ld, vu, vt, vk, vp, vm,
                        vids, vlps, stream);
  Py_END_ALLOW_THREADS
  Py_INCREF(out);
  return done(rc, out);
}

PyMethodDef methods[] = {
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm)), METH_FASTCALL, nullptr},
    {"project", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(project)), METH_FASTCALL, nullptr},
    {"draw", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(draw)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_strata_tail", "Calls of strata_tail.h on PyTorch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__strata_tail() { return PyModule_Create(&module); }
