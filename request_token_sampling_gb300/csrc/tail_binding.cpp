// tail_binding.cpp -- Python calls of include/strata_tail.h and include/strata_train.h on PyTorch tensors.
//
// Checks what the C ABI cannot see (types, shapes, devices of tensors), allocates the outputs that the
// caller left out, and makes the C call on the tensors' addresses without holding the interpreter's lock.
// It is compiled because the smallest calls' kernels take 2 to 5 us: the same steps in Python took 20 us
// a call on a Grace core, most of it in cold attribute look-ups.  A C error code is returned as an int,
// which the Python side turns into StrataError.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>


#include "../../include/strata_tail.h"
#include "../../include/strata_train.h"

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

const Tensor* given(const Tensor& t) { return t.defined() ? &t : nullptr; }

// The outputs and the workspace of a call: the caller's from `out`, or new ones (which are put there), or none.  New outputs of up
// to 32 KB share an allocation, since each takes more than half a microsecond and the smallest calls three on the GPU.  The
// workspace has its own, which ends with the call: an output that is kept keeps no more than its neighbours.
class Made {
 public:
  Made(PyObject* out, const Tensor& like) : out_(out), like_(like) {
    if (!PyDict_Check(out)) refuse(PyExc_TypeError, "out", "must be a dict");
  }
  void want(const char* key, PyObject* wanted, at::IntArrayRef shape, ScalarType type) {
    Item& i = items_[n_++];
    i.key = key;
    PyObject* had = PyDict_GET_SIZE(out_) > 0 ? PyDict_GetItemString(out_, key) : nullptr;
    if (had != nullptr && had != Py_None) {
      i.t = needed(had, key);
      return;
    }
    if (wanted != Py_True) return;
    size(i, shape, type);
  }
  void want_workspace(int64_t bytes) {
    Item& i = items_[n_++];
    if (bytes > 0) size(i, at::IntArrayRef(&bytes, 1), at::kByte);
  }
  void make() {
    int64_t shared = 0, small = 0;
    for (int k = 0; k < n_; ++k) {
      if (!shares(items_[k])) continue;
      shared += (items_[k].bytes + 255) / 256 * 256;
      ++small;
    }
    Tensor whole;
    int64_t at = 0;
    for (int k = 0; k < n_; ++k) {
      Item& i = items_[k];
      if (i.bytes < 0) continue;
      const at::IntArrayRef shape(i.shape, i.dims);
      if (!shares(i) || small == 1) {
        i.t = fresh(shape, i.type, like_);
      } else {
        if (!whole.defined()) whole = fresh({shared}, at::kByte, like_);
        i.t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(whole.storage()), whole.key_set(), c10::scalarTypeToTypeMeta(i.type));
        const int64_t strides[2] = {i.dims == 2 ? i.shape[1] : 1, 1};
        i.t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(i.type)));
        i.t.unsafeGetTensorImpl()->set_sizes_and_strides(shape, at::IntArrayRef(strides, i.dims));
        at += (i.bytes + 255) / 256 * 256;
      }
      if (i.key != nullptr) put(out_, i.key, i.t);
    }
  }
  const Tensor* operator[](int k) const { return given(items_[k].t); }

 private:
  static constexpr int64_t SMALL = 32768;
  struct Item {
    const char* key = nullptr;
    int64_t shape[2] = {}, bytes = -1;  // -1: nothing to make
    int dims = 0;
    ScalarType type = at::kByte;
    Tensor t;
  };
  static bool shares(const Item& i) { return i.key != nullptr && i.bytes > 0 && i.bytes <= SMALL; }
  static void size(Item& i, at::IntArrayRef shape, ScalarType type) {
    i.type = type;
    i.bytes = static_cast<int64_t>(c10::elementSize(type));
    for (const int64_t s : shape) {
      i.shape[i.dims++] = s;
      i.bytes *= s;
    }
  }
  PyObject* out_;
  const Tensor& like_;
  Item items_[5];
  int n_ = 0;
};

// The caller's workspace, or (`allocate`) the bytes to make.
int64_t workspace_bytes(const Tensor* had, PyObject* allocate, int64_t need) { return had == nullptr && allocate == Py_True ? need : 0; }
void* workspace_at(const Tensor* had, const Tensor* made, int device, int64_t& bytes) {
  const Tensor* t = had != nullptr ? had : made;
  bytes = t != nullptr ? t->numel() : 0;
  return dense(t, "workspace", {bytes}, at::kByte, device);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

// Automatic differentiation passes these calls by.  One that it would have to record says so, or a model would train without
// it; the warning is the caller's line's, once for each.
void unrecorded(std::initializer_list<const Tensor*> inputs, const char* by) {
  if (!c10::GradMode::is_enabled()) return;
  for (const Tensor* t : inputs) {
    if (t == nullptr || !t->requires_grad()) continue;
    if (PyErr_WarnFormat(PyExc_UserWarning, 2,
                         "an input requires a gradient, and this call is not recorded: %s computes its gradients. "
                         "Call it under torch.no_grad(), or with detached tensors", by) != 0)
      throw Refused();
    return;
  }
}

// (x, weight, bias, residual, eps, want residual, want y, want mean and rstd, out, stream) -> out, a dict
TAIL_CALL(layer_norm) {
  arguments(n, 10);
  const Tensor &x = needed(a[0], "x"), &weight = needed(a[1], "weight");
  const Tensor *bias = tensor(a[2], "bias"), *residual = tensor(a[3], "residual");
  const double eps = number(a[4]);
  const ScalarType type = x.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) refuse(PyExc_TypeError, "x", "must be float32 or bfloat16");
  const int device = call_device(x, "x");
  const int64_t T = x.size(0), H = x.size(1);
  PyObject* out = a[8];
  Made made(out, x);
  made.want("residual", a[5], {T, H}, type);
  made.want("y", a[6], {T, H}, type);
  made.want("mean", a[7], {T}, at::kFloat);
  made.want("rstd", a[7], {T}, at::kFloat);
  made.make();
  const Rows rx = rows(&x, "x", T, H, type, device), rr = rows(residual, "residual", T, H, type, device),
             rro = rows(made[0], "residual", T, H, type, device), ry = rows(made[1], "y", T, H, type, device);
  void *pw = dense(&weight, "weight", {H}, type, device), *pb = dense(bias, "bias", {H}, type, device),
       *pm = dense(made[2], "mean", {T}, at::kFloat, device), *ps = dense(made[3], "rstd", {T}, at::kFloat, device);
  void* stream = stream_of(a[9], device);
  const int t32 = narrow(T, "T"), h32 = narrow(H, "H");
  unrecorded({&x, &weight, bias, residual}, "layer_norm_grad");
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = strata_layer_norm_rows(rx.p, rx.ld, rr.p, rr.ld, pw, pb, type == at::kFloat ? STRATA_DTYPE_F32 : STRATA_DTYPE_BF16, t32, h32,
                              static_cast<float>(eps), rro.p, rro.ld, ry.p, ry.ld, static_cast<float*>(pm), static_cast<float*>(ps),
                              stream);
  Py_END_ALLOW_THREADS
  Py_INCREF(out);
  return done(rc, out);
}

// (dy, x, weight, mean, rstd, dresidual, want dx, want dweight, want dbias, out, workspace, allocate it, stream) -> out, a dict
TAIL_CALL(layer_norm_grad) {
  arguments(n, 13);
  const Tensor &dy = needed(a[0], "dy"), &x = needed(a[1], "x"), &weight = needed(a[2], "weight"), &mean = needed(a[3], "mean"),
               &rstd = needed(a[4], "rstd");
  const Tensor* dresidual = tensor(a[5], "dresidual");
  const ScalarType type = x.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) refuse(PyExc_TypeError, "x", "must be float32 or bfloat16");
  const int device = call_device(x, "x");
  const int64_t T = x.size(0), H = x.size(1);
  PyObject* out = a[9];
  const int t32 = narrow(T, "T"), h32 = narrow(H, "H");
  const Tensor* ws_given = tensor(a[10], "workspace");
  Made made(out, x);
  made.want("dx", a[6], {T, H}, type);
  made.want("dweight", a[7], {H}, type);
  made.want("dbias", a[8], {H}, type);
  const bool sums = a[7] == Py_True || a[8] == Py_True || made[1] != nullptr || made[2] != nullptr;
  made.want_workspace(sums ? workspace_bytes(ws_given, a[11], strata_layer_norm_workspace(t32, h32)) : 0);
  made.make();
  const Rows rdy = rows(&dy, "dy", T, H, type, device), rx = rows(&x, "x", T, H, type, device),
             rdr = rows(dresidual, "dresidual", T, H, type, device), rdx = rows(made[0], "dx", T, H, type, device);
  void *pw = dense(&weight, "weight", {H}, type, device), *pm = dense(&mean, "mean", {T}, at::kFloat, device),
       *ps = dense(&rstd, "rstd", {T}, at::kFloat, device), *pdw = dense(made[1], "dweight", {H}, type, device),
       *pdb = dense(made[2], "dbias", {H}, type, device);
  int64_t bytes = 0;
  void* ws = workspace_at(ws_given, made[3], device, bytes);
  void* stream = stream_of(a[12], device);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = strata_layer_norm_grad(rdy.p, rdy.ld, rx.p, rx.ld, pw, static_cast<float*>(pm), static_cast<float*>(ps), rdr.p, rdr.ld,
                              type == at::kFloat ? STRATA_DTYPE_F32 : STRATA_DTYPE_BF16, t32, h32, rdx.p, rdx.ld, pdw, pdb, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  Py_INCREF(out);
  return done(rc, out);
}

// The rows, the head and the tokens of a loss.
struct LossOperands {
  Rows x, w;
  int T = 0, V = 0, H = 0, K = 0;
  int32_t* ids = nullptr;
  float* teacher = nullptr;
};
LossOperands loss_operands(const Tensor& x, const Tensor& w, const Tensor& ids, const Tensor* teacher, int& device) {
  device = call_device(x, "x");
  if (w.dim() != 2) refuse(PyExc_ValueError, "w", "must be [ids, width]");
  const int64_t T = x.size(0), H = x.size(1), V = w.size(0);
  LossOperands o;
  o.x = rows(&x, "x", T, H, at::kBFloat16, device);
  o.w = rows(&w, "w", V, H, at::kBFloat16, device);
  if (T == 1) o.x.ld = (H + 7) / 8 * 8;  // the stride of one row means nothing
  if (V == 1) o.w.ld = (H + 7) / 8 * 8;
  if (teacher != nullptr) {
    if (teacher->dim() != 2) refuse(PyExc_ValueError, "teacher", "must be [rows, tokens]");
    const int64_t K = teacher->size(1);
    o.K = narrow(K, "K");
    o.teacher = static_cast<float*>(dense(teacher, "teacher", {T, K}, at::kFloat, device));
    o.ids = static_cast<int32_t*>(dense(&ids, "ids", {T, K}, at::kInt, device));
  } else {
    o.ids = static_cast<int32_t*>(dense(&ids, "ids", {T}, at::kInt, device));
  }
  o.T = narrow(T, "T");
  o.V = narrow(V, "V");
  o.H = narrow(H, "H");
  return o;
}

// (x, w, ids, teacher or None, temperature, want loss and lse, out, workspace, allocate it, stream) -> out, a dict
TAIL_CALL(loss) {
  arguments(n, 10);
  const Tensor &x = needed(a[0], "x"), &w = needed(a[1], "w"), &ids = needed(a[2], "ids");
  const Tensor* teacher = tensor(a[3], "teacher");
  const float temperature = static_cast<float>(number(a[4]));
  if (x.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "x", "must be bfloat16");
  int device;
  const LossOperands o = loss_operands(x, w, ids, teacher, device);
  PyObject* out = a[6];
  const Tensor* ws_given = tensor(a[7], "workspace");
  Made made(out, x);
  made.want("loss", a[5], {o.T}, at::kFloat);
  made.want("lse", a[5], {o.T}, at::kFloat);
  made.want_workspace(workspace_bytes(ws_given, a[8], strata_loss_workspace(o.T, o.V, o.H, o.K, 0)));
  made.make();
  float *pl = static_cast<float*>(dense(made[0], "loss", {o.T}, at::kFloat, device)),
        *pe = static_cast<float*>(dense(made[1], "lse", {o.T}, at::kFloat, device));
  int64_t bytes = 0;
  void* ws = workspace_at(ws_given, made[2], device, bytes);
  void* stream = stream_of(a[9], device);
  unrecorded({&x, &w, teacher}, teacher != nullptr ? "distill_grad" : "cross_entropy_grad");
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = teacher != nullptr ? strata_distill_rows(o.x.p, o.x.ld, o.w.p, o.w.ld, o.T, o.V, o.H, o.K, o.ids, o.teacher, temperature, pl, pe, ws, bytes, stream)
                          : strata_cross_entropy_rows(o.x.p, o.x.ld, o.w.p, o.w.ld, o.T, o.V, o.H, o.ids, pl, pe, ws, bytes, stream);
  Py_END_ALLOW_THREADS
  Py_INCREF(out);
  return done(rc, out);
}

// (x, w, ids, teacher or None, temperature, lse, g, want dx, want dw, out, workspace, allocate it, stream) -> out, a dict
TAIL_CALL(loss_grad) {
  arguments(n, 13);
  const Tensor &x = needed(a[0], "x"), &w = needed(a[1], "w"), &ids = needed(a[2], "ids"), &lse = needed(a[5], "lse"), &g = needed(a[6], "g");
  const Tensor* teacher = tensor(a[3], "teacher");
  const float temperature = static_cast<float>(number(a[4]));
  if (x.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "x", "must be bfloat16");
  int device;
  const LossOperands o = loss_operands(x, w, ids, teacher, device);
  float *pe = static_cast<float*>(dense(&lse, "lse", {o.T}, at::kFloat, device)), *pg = static_cast<float*>(dense(&g, "g", {o.T}, at::kFloat, device));
  PyObject* out = a[9];
  const Tensor* ws_given = tensor(a[10], "workspace");
  Made made(out, x);
  made.want("dx", a[7], {o.T, o.H}, at::kBFloat16);
  made.want("dw", a[8], {o.V, o.H}, at::kBFloat16);
  made.want_workspace(workspace_bytes(ws_given, a[11], strata_loss_workspace(o.T, o.V, o.H, o.K, 1)));
  made.make();
  Rows rdx = rows(made[0], "dx", o.T, o.H, at::kBFloat16, device), rdw = rows(made[1], "dw", o.V, o.H, at::kBFloat16, device);
  if (o.T == 1) rdx.ld = o.x.ld;
  if (o.V == 1) rdw.ld = o.w.ld;
  int64_t bytes = 0;
  void* ws = workspace_at(ws_given, made[2], device, bytes);
  void* stream = stream_of(a[12], device);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = teacher != nullptr ? strata_distill_grad(o.x.p, o.x.ld, o.w.p, o.w.ld, o.T, o.V, o.H, o.K, o.ids, o.teacher, temperature, pe, pg, rdx.p, rdx.ld,
                                                rdw.p, rdw.ld, ws, bytes, stream)
                          : strata_cross_entropy_grad(o.x.p, o.x.ld, o.w.p, o.w.ld, o.T, o.V, o.H, o.ids, pe, pg, rdx.p, rdx.ld, rdw.p, rdw.ld, ws,
                                                      bytes, stream);
  Py_END_ALLOW_THREADS
  Py_INCREF(out);
  return done(rc, out);
}

PyMethodDef methods[] = {
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm)), METH_FASTCALL, nullptr},
    {"project", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(project)), METH_FASTCALL, nullptr},
    {"draw", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(draw)), METH_FASTCALL, nullptr},
    {"layer_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(layer_norm)), METH_FASTCALL, nullptr},
    {"layer_norm_grad", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(layer_norm_grad)), METH_FASTCALL, nullptr},
    {"loss", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(loss)), METH_FASTCALL, nullptr},
    {"loss_grad", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(loss_grad)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_strata_tail", "Calls of strata_tail.h and strata_train.h on PyTorch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__strata_tail() { return PyModule_Create(&module); }
