// Argument checks and marshalling of the vocabulary-head operators for Python
// (head.py): tensors in, one call of the C ABI, tensors out.  Nothing is computed
// here.  It is native because the smallest calls are host bound: reading a
// tensor's type, strides and pointer costs 0.1 to 0.2 us an attribute from
// Python, so that the checks of a step over 24 tensors took 45 us beside 4 us on the
// GPU and those of one 8-bit product of one token 12 us beside 9; here the whole
// checks take less than 1 us a call and 0.05 us a tensor.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <utility>
#include <vector>

#include "os2.h"

namespace {

using at::Tensor;
constexpr int64_t kBlock = 256;  // elements that share a scale of an 8-bit moment

// the library that the binding has loaded, and its exception
struct {
  decltype(&os2_quantize_rows) quantize_rows;
  decltype(&os2_i8gemm_workspace_size) i8_workspace;
  decltype(&os2_i8gemm) i8gemm;
  decltype(&os2_i8linear) i8linear;
  decltype(&os2_xent_workspace_size) xent_workspace;
  decltype(&os2_xent) xent;
  decltype(&os2_xent_backward) xent_backward;
  decltype(&os2_adamw) adamw;
  decltype(&os2_adamw_moments) adamw_moments;
  decltype(&os2_rmsnorm) rmsnorm;
  decltype(&os2_rmsnorm_quantize) rmsnorm_quantize;
  decltype(&os2_rmsnorm_workspace_size) rmsnorm_workspace;
  decltype(&os2_rmsnorm_backward) rmsnorm_backward;
  decltype(&os2_sample) sample;
  decltype(&os2_linear_workspace_size) linear_workspace;
  decltype(&os2_linear) linear;
  decltype(&os2_linear_backward_workspace_size) linear_backward_workspace;
  decltype(&os2_linear_backward) linear_backward;
} lib;
PyObject *g_error;

const Tensor &tensor(PyObject *o, const char *name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

int code(at::ScalarType t) {  // os2_dtype, or -1
  return t == at::kFloat ? OS2_F32 : t == at::kHalf ? OS2_F16 : t == at::kBFloat16 ? OS2_BF16 : -1;
}

int as_int(int64_t x, const char *name) {
  TORCH_CHECK_VALUE(x <= INT32_MAX, name, " is too long: ", x);
  return int(x);
}

// A 2-D CUDA tensor with contiguous rows that do not overlap.
struct Rows {
  int m, k, ld;
  void *p;
};

Rows rows(const Tensor &x, const char *name, bool type_ok, const char *types) {
  TORCH_CHECK_VALUE(x.dim() == 2 && type_ok, name, " must be a 2-D CUDA tensor of ", types);
  const int64_t m = x.size(0), k = x.size(1), ld = x.stride(0);
  TORCH_CHECK_VALUE(k <= 1 || x.stride(1) == 1, name, " must have contiguous rows");
  // (an expanded tensor's rows do; the stride of a single row means nothing)
  TORCH_CHECK_VALUE(m <= 1 || ld >= k, name, " must have rows that do not overlap: row stride ", ld, " of ", k, " entries");
  TORCH_CHECK_VALUE(x.is_cuda(), name, " must be a 2-D CUDA tensor of ", types);
  return {as_int(m, name), as_int(k, name), as_int(std::max<int64_t>(m > 1 ? ld : k, 1), name), x.data_ptr()};
}

Tensor vec(PyObject *o, const char *name, int64_t n, at::ScalarType t, c10::Device dev) {
  const Tensor &x = tensor(o, name);
  TORCH_CHECK_VALUE(x.scalar_type() == t && x.dim() == 1 && x.size(0) == n && x.device() == dev, name, " must be ", n, " ",
                    t, " values on ", dev);
  return x.is_contiguous() ? x : x.contiguous();
}

// Whether someone looks on in the dispatcher: a dispatch mode (by its key), a profiler, or the filling of new
// memory that deterministic algorithms ask for.  Asked once a call, and by calls with new outputs only.
struct Seen {
  int known = -1;
  explicit operator bool() {
    if (known < 0)
      known = c10::impl::tls_local_dispatch_key_set().included_.has(c10::DispatchKey::Python) || at::hasCallbacks() ||
              (at::globalContext().deterministicAlgorithms() && at::globalContext().deterministicFillUninitializedMemory());
    return known;
  }
};

// A new output: past the dispatcher, which takes 0.4 us (a norm with a residual of one row 5.4 and
// 4.4 us a call), unless it is seen there.
Tensor fresh(Seen &seen, at::IntArrayRef shape, at::ScalarType t, c10::Device dev) {
  if (seen) return at::empty(shape, at::TensorOptions().dtype(t).device(dev));
  return at::detail::empty_cuda(shape, t, dev, std::nullopt);
}

// The output, the caller's or a new one, and its leading dimension.
Tensor out_rows(Seen &seen, PyObject *o, const char *name, int64_t m, int64_t n, at::ScalarType t, c10::Device dev, int &ld) {
  ld = as_int(std::max<int64_t>(n, 1), name);
  if (o == Py_None) return fresh(seen, {m, n}, t, dev);
  const Tensor &x = tensor(o, name);
  TORCH_CHECK_VALUE(x.dim() == 2 && x.size(0) == m && x.size(1) == n && x.scalar_type() == t && x.device() == dev, name,
                    " must be (", m, ", ", n, ") ", t, " on ", dev);
  TORCH_CHECK_VALUE(n <= 1 || x.stride(1) == 1, name, " must have contiguous rows");
  TORCH_CHECK_VALUE(m <= 1 || x.stride(0) >= n, name, " must not overlap itself");
  if (m > 1) ld = as_int(std::max<int64_t>(x.stride(0), ld), name);
  return x;
}

// Where a matrix (or a vector, as one row) lies: m rows of `row` bytes, `pitch` apart.
struct Area {
  intptr_t p;
  int64_t m, row, pitch;
  Area(const Rows &x, size_t elem) : p((intptr_t)x.p), m(x.m), row(x.k * (int64_t)elem), pitch(x.ld * (int64_t)elem) {}
  Area(const Tensor &x, int ld) : Area(Rows{int(x.size(0)), int(x.size(1)), ld, x.data_ptr()}, x.element_size()) {}
  explicit Area(const Tensor &v) : p(v.defined() ? (intptr_t)v.data_ptr() : 0), m(1), row(p ? int64_t(v.nbytes()) : 0), pitch(row) {}
};

// Refuses an output of the caller's that shares memory with `in`; where they are the same entry
// on entry, it may (same).
void apart(const Area &out, const char *name, const Area &in, const char *other, bool same = false) {
  if (!out.p || !in.p || !out.m || !in.m || !out.row || !in.row) return;
  if (out.p + (out.m - 1) * out.pitch + out.row <= in.p || in.p + (in.m - 1) * in.pitch + in.row <= out.p) return;
  // (one row has any pitch)
  const int64_t pitch = out.m > 1 ? out.pitch : in.pitch;
  if (out.m == 1 || in.m == 1 || out.pitch == in.pitch) {
    if (same && out.p == in.p && out.m == in.m && out.row == in.row) return;
    // side by side in rows of one length
    const int64_t off = ((in.p - out.p) % pitch + pitch) % pitch;
    if (off >= out.row && off + in.row <= pitch) return;
  }
  TORCH_CHECK_VALUE(false, name, " must not overlap ", other);
}

Tensor out_vec(Seen &seen, PyObject *o, const char *name, int64_t n, at::ScalarType t, c10::Device dev) {
  if (o == Py_None) return fresh(seen, {n}, t, dev);
  const Tensor &x = tensor(o, name);
  TORCH_CHECK_VALUE(x.dim() == 1 && x.size(0) == n && x.scalar_type() == t && x.device() == dev && x.is_contiguous(), name,
                    " must be ", n, " contiguous ", t, " values on ", dev);
  return x;
}

// Small workspaces are kept, one for each thread, device and stream (calls that
// share one are ordered by the stream): an allocation between two launches costs
// as much host time as a launch.  A captured call gets its own.
constexpr size_t kKeep = size_t(32) << 20;

struct Kept : std::map<std::pair<int, cudaStream_t>, Tensor> {
  ~Kept() {  // a process that ends leaves them to the driver
    if (!Py_IsInitialized())
      for (auto &e : *this) (void)e.second.unsafeReleaseTensorImpl();
  }
};

Tensor workspace(PyObject *o, size_t need, c10::Device dev, cudaStream_t stream) {
  if (o != Py_None) {
    const Tensor &x = tensor(o, "workspace");
    TORCH_CHECK_VALUE(x.device() == dev && x.is_contiguous(), "workspace must be contiguous and on ", dev);
    return x;
  }
  // (nobody's but the kernels': a mode that makes stand-ins of new tensors would have one kept)
  auto scratch = [&](size_t bytes) { return at::detail::empty_cuda({int64_t(bytes)}, at::kByte, dev, std::nullopt); };
  if (need > kKeep || c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    return scratch(need);
  static thread_local Kept kept;
  Tensor &ws = kept[{dev.index(), stream}];
  if (!ws.defined() || size_t(ws.numel()) < need)
    ws = scratch(std::min(kKeep, std::max(size_t(1) << 20, 2 * need)));
  return ws;
}

// A tensor of the caller's was written in place: autograd then refuses to go back
// through what had saved it before.  (Inference tensors have no such count.)
void written(c10::TensorImpl *x) {
  if (!x->is_inference()) x->bump_version();
}
void written(PyObject *o) {  // a caller's output, or None
  if (o != Py_None) written(THPVariable_Unpack(o).unsafeGetTensorImpl());
}

void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// The call itself, without the interpreter's lock; its status as an exception.
template <class F, class... A>
bool call(const char *where, F f, A... a) {
  os2_status st;
  Py_BEGIN_ALLOW_THREADS st = f(a...);
  Py_END_ALLOW_THREADS if (st == OS2_OK) return true;
  if (PyObject *e = PyObject_CallFunction(g_error, "is", int(st), where)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return false;
}

PyObject *pair(const Tensor &a, const Tensor &b) {  // None for one that is not there
  PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
  PyObject *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

#define OS2_ARGS(count)                                                              \
  HANDLE_TH_ERRORS                                                                   \
  if (nargs != (count)) {                                                            \
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %d", nargs, int(count)); \
    return nullptr;                                                                  \
  }                                                                                  \
  [[maybe_unused]] Seen seen;

constexpr const char *kFloats = "float32, float16 or bfloat16", *kHalves = "bfloat16 or float16, one type for H and W";

// quantize_rows(X, out, scale)
PyObject *py_quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(3)
  const Tensor &X = tensor(a[0], "X");
  const Rows x = rows(X, "X", code(X.scalar_type()) >= 0, kFloats);
  const c10::Device dev = X.device();
  c10::cuda::CUDAGuard on(dev);
  int ldq;
  const Tensor q = out_rows(seen, a[1], "out", x.m, x.k, at::kChar, dev, ldq), scale = out_vec(seen, a[2], "scale", x.m, at::kFloat, dev);
  if (!call("os2_quantize_rows", lib.quantize_rows, x.m, x.k, code(X.scalar_type()), (const void *)x.p, x.ld,
            (int8_t *)ptr(q), ldq, (float *)ptr(scale), (void *)c10::cuda::getCurrentCUDAStream(dev.index()).stream()))
    return nullptr;
  written(a[1]), written(a[2]);
  return pair(q, scale);
  END_HANDLE_TH_ERRORS
}

// i8(X, a_scale, Bt, b_scale, bias, out_dtype, out, workspace, linear): i8linear, or i8gemm with a_scale
PyObject *py_i8(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(9)
  const bool linear = a[8] == Py_True;
  const Tensor &X = tensor(a[0], linear ? "X" : "A"), &B = tensor(a[2], "Bt");
  const at::ScalarType xt = X.scalar_type();
  const Rows x = linear ? rows(X, "X", code(xt) >= 0, kFloats) : rows(X, "A", xt == at::kChar, "int8");
  const Rows b = rows(B, "Bt", B.scalar_type() == at::kChar, "int8");
  const c10::Device dev = X.device();
  TORCH_CHECK_VALUE(B.device() == dev, "Bt must be on ", dev);
  TORCH_CHECK_VALUE(b.k == x.k, "inner dimensions differ");
  const int m = x.m, n = b.m, k = x.k;
  at::ScalarType ct = linear ? xt : at::kBFloat16;
  if (a[5] != Py_None) {
    TORCH_CHECK_VALUE(THPDtype_Check(a[5]), "out_dtype must be a torch.dtype");
    ct = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
  } else if (a[6] != Py_None) {
    ct = tensor(a[6], "out").scalar_type();
  }
  TORCH_CHECK_VALUE(code(ct) >= 0, "out_dtype must be ", kFloats);
  c10::cuda::CUDAGuard on(dev);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index());
  const Tensor sa = linear ? Tensor() : vec(a[1], "a_scale", m, at::kFloat, dev), sb = vec(a[3], "b_scale", n, at::kFloat, dev);
  const Tensor bias = a[4] == Py_None ? Tensor() : vec(a[4], "bias", n, at::kFloat, dev);
  int ldc;
  const Tensor C = out_rows(seen, a[6], "out", m, n, ct, dev, ldc);
  const Tensor ws = workspace(a[7], lib.i8_workspace(m, n, k, b.p, b.ld), dev, stream);
  const bool ok =
      linear ? call("os2_i8linear", lib.i8linear, m, n, k, code(xt), (const void *)x.p, x.ld, (const int8_t *)b.p, b.ld,
                    (const float *)ptr(sb), (const float *)ptr(bias), ptr(C), ldc, code(ct), ptr(ws), size_t(ws.nbytes()),
                    (void *)stream)
             : call("os2_i8gemm", lib.i8gemm, m, n, k, (const int8_t *)x.p, x.ld, (const float *)ptr(sa), (const int8_t *)b.p,
                    b.ld, (const float *)ptr(sb), (const float *)ptr(bias), ptr(C), ldc, code(ct), ptr(ws),
                    size_t(ws.nbytes()), (void *)stream);
  if (!ok) return nullptr;
  written(a[6]);
  return THPVariable_Wrap(C);
  END_HANDLE_TH_ERRORS
}

struct Head {
  Rows h, w;
  int dtype;
  c10::Device dev;
};

Head head(PyObject *ho, PyObject *wo) {
  const Tensor &H = tensor(ho, "H"), &W = tensor(wo, "W");
  const at::ScalarType t = H.scalar_type();
  const Rows h = rows(H, "H", t == at::kHalf || t == at::kBFloat16, kHalves), w = rows(W, "W", W.scalar_type() == t, kHalves);
  TORCH_CHECK_VALUE(W.device() == H.device(), "W must be on ", H.device());
  TORCH_CHECK_VALUE(h.k == w.k, "inner dimensions differ");
  return {h, w, code(t), H.device()};
}

// A Python integer as it is, or raises.
long long integer(PyObject *o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}

double real(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}

// xent(H, W, labels, ignore_index, workspace)
PyObject *py_xent(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(5)
  const Head t = head(a[0], a[1]);
  const int n = t.h.m, k = t.h.k, v = t.w.m;
  c10::cuda::CUDAGuard on(t.dev);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(t.dev.index());
  const Tensor y = vec(a[2], "labels", n, at::kLong, t.dev), loss = fresh(seen, {n}, at::kFloat, t.dev),
               lse = fresh(seen, {n}, at::kFloat, t.dev);
  const Tensor ws = workspace(a[4], lib.xent_workspace(n, k, v, t.w.p, t.w.ld, 0), t.dev, stream);
  if (!call("os2_xent", lib.xent, n, k, v, t.dtype, (const void *)t.h.p, t.h.ld, (const void *)t.w.p, t.w.ld,
            (const long long *)ptr(y), integer(a[3]), (float *)ptr(loss), (float *)ptr(lse), ptr(ws), size_t(ws.nbytes()),
            (void *)stream))
    return nullptr;
  return pair(loss, lse);
  END_HANDLE_TH_ERRORS
}

// xent_backward(H, W, labels, lse, grad, ignore_index, need_dh, need_dw, workspace)
PyObject *py_xent_backward(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(9)
  const Head t = head(a[0], a[1]);
  const int n = t.h.m, k = t.h.k, v = t.w.m, need_dh = PyObject_IsTrue(a[6]), need_dw = PyObject_IsTrue(a[7]);
  if (need_dh < 0 || need_dw < 0) return nullptr;
  const at::ScalarType dt = THPVariable_Unpack(a[0]).scalar_type();
  c10::cuda::CUDAGuard on(t.dev);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(t.dev.index());
  const Tensor y = vec(a[2], "labels", n, at::kLong, t.dev), lse = vec(a[3], "lse", n, at::kFloat, t.dev),
               grad = vec(a[4], "grad", n, at::kFloat, t.dev);
  const Tensor dh = need_dh ? fresh(seen, {n, k}, dt, t.dev) : Tensor(), dw = need_dw ? fresh(seen, {v, k}, dt, t.dev) : Tensor();
  const Tensor ws = workspace(a[8], lib.xent_workspace(n, k, v, t.w.p, t.w.ld, t.dtype == OS2_BF16 ? OS2_XENT_BACKWARD_BF16 : 1), t.dev, stream);
  if (!call("os2_xent_backward", lib.xent_backward, n, k, v, t.dtype, (const void *)t.h.p, t.h.ld, (const void *)t.w.p,
            t.w.ld, (const long long *)ptr(y), integer(a[5]), (const float *)ptr(lse), (const float *)ptr(grad), ptr(dh), k,
            ptr(dw), k, ptr(ws), size_t(ws.nbytes()), (void *)stream))
    return nullptr;
  return pair(dh, dw);
  END_HANDLE_TH_ERRORS
}

// A list of contiguous tensors, one for each parameter, and its pointers.
struct List {
  THPObjectPtr seq;
  std::vector<void *> p;
  std::vector<c10::TensorImpl *> impl;  // held by seq
  at::ScalarType type = at::kFloat;

  const Tensor &at(size_t i, const char *name) const { return tensor(PyTuple_GET_ITEM(seq.get(), i), name); }
  void open(PyObject *o, const char *name) {
    // (a tuple of its own: another thread may change the caller's list during the call)
    seq = PySequence_Tuple(o);
    if (!seq) throw python_error();
    p.reserve(PyTuple_GET_SIZE(seq.get()));
    impl.reserve(p.capacity());
    if (p.capacity()) type = at(0, name).scalar_type();
  }
  // sized: as large as ref's tensors, or with a value for each block of them
  void take(const List &ref, const char *name, c10::Device dev, bool type_ok, const char *types, bool blocks) {
    const size_t count = PyTuple_GET_SIZE(ref.seq.get());
    TORCH_CHECK_VALUE(size_t(PyTuple_GET_SIZE(seq.get())) == count, name, ": ",
                      PyTuple_GET_SIZE(seq.get()), " tensors for ", count, " parameters");
    TORCH_CHECK_VALUE(type_ok, name, " must be all ", types);
    for (size_t i = 0; i < count; i++) {
      const Tensor &x = at(i, name), &r = ref.at(i, "params");
      TORCH_CHECK_VALUE(x.scalar_type() == type, name, " must be all ", types);
      TORCH_CHECK_VALUE(x.device() == dev && x.is_contiguous() &&
                            (blocks ? x.numel() == (r.numel() + kBlock - 1) / kBlock : x.sizes().equals(r.sizes())),
                        name, " must be contiguous, on one CUDA device, and ",
                        blocks ? "one value for each block of elements" : "of the parameters' shapes");
      p.push_back(x.data_ptr());
      impl.push_back(x.unsafeGetTensorImpl());
    }
  }
  void written() const {
    for (c10::TensorImpl *x : impl) ::written(x);
  }
};

// adamw(params, grads, exp_avg, exp_avg_sq, exp_avg_scales, exp_avg_sq_scales, step, lr, beta1, beta2, eps, weight_decay)
PyObject *py_adamw(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(12)
  List p, g, m, v, ms, vs;
  p.open(a[0], "params");
  const size_t count = PyTuple_GET_SIZE(p.seq.get());
  if (!count) Py_RETURN_NONE;
  as_int(int64_t(count), "params");
  const c10::Device dev = p.at(0, "params").device();
  TORCH_CHECK_VALUE(dev.is_cuda(), "params must be on one CUDA device");
  const bool q8 = a[4] != Py_None || a[5] != Py_None;
  g.open(a[1], "grads"), m.open(a[2], "exp_avg"), v.open(a[3], "exp_avg_sq");
  p.take(p, "params", dev, code(p.type) >= 0, kFloats, false);
  g.take(p, "grads", dev, code(g.type) >= 0, kFloats, false);
  m.take(p, "exp_avg", dev, m.type == (q8 ? at::kChar : at::kFloat), q8 ? "int8" : "float32", false);
  v.take(p, "exp_avg_sq", dev, v.type == (q8 ? at::kByte : at::kFloat), q8 ? "uint8" : "float32", false);
  if (q8) {
    TORCH_CHECK_VALUE(a[4] != Py_None && a[5] != Py_None, "8-bit moments need exp_avg_scales and exp_avg_sq_scales");
    ms.open(a[4], "exp_avg_scales"), vs.open(a[5], "exp_avg_sq_scales");
    ms.take(p, "exp_avg_scales", dev, ms.type == at::kFloat, "float32", true);
    vs.take(p, "exp_avg_sq_scales", dev, vs.type == at::kFloat, "float32", true);
  }
  std::vector<long long> sizes(count);
  for (size_t i = 0; i < count; i++) sizes[i] = p.at(i, "params").numel();
  const long long step = integer(a[6]);
  const double lr = real(a[7]), b1 = real(a[8]), b2 = real(a[9]), eps = real(a[10]), wd = real(a[11]);
  c10::cuda::CUDAGuard on(dev);
  if (!call("os2_adamw", lib.adamw, int(count), (const long long *)sizes.data(), (void *const *)p.p.data(),
            (const void *const *)g.p.data(), (void *const *)m.p.data(), (void *const *)v.p.data(),
            q8 ? (float *const *)ms.p.data() : nullptr, q8 ? (float *const *)vs.p.data() : nullptr, code(p.type),
            code(g.type), q8 ? 8 : 32, lr, b1, b2, eps, wd, step,
            (void *)c10::cuda::getCurrentCUDAStream(dev.index()).stream()))
    return nullptr;
  p.written(), m.written(), v.written(), ms.written(), vs.written();
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// adamw_moments(exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale)
PyObject *py_adamw_moments(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(4)
  const Tensor &c = tensor(a[0], "exp_avg");
  const int64_t n = c.numel();
  const c10::Device dev = c.device();
  auto check = [&](PyObject *o, const char *name, at::ScalarType t, int64_t size) {
    const Tensor &x = tensor(o, name);
    TORCH_CHECK_VALUE(x.is_cuda() && x.device() == dev && x.scalar_type() == t && x.numel() == size && x.is_contiguous(), name,
                      " must be ", size, " contiguous ", t, " values on one CUDA device");
    return x.data_ptr();
  };
  const int64_t blocks = (n + kBlock - 1) / kBlock;
  const void *cm = check(a[0], "exp_avg", at::kChar, n), *sm = check(a[1], "exp_avg_scale", at::kFloat, blocks),
             *cv = check(a[2], "exp_avg_sq", at::kByte, n), *sv = check(a[3], "exp_avg_sq_scale", at::kFloat, blocks);
  c10::cuda::CUDAGuard on(dev);
  const Tensor m = fresh(seen, c.sizes(), at::kFloat, dev), v = fresh(seen, c.sizes(), at::kFloat, dev);
  if (!call("os2_adamw_moments", lib.adamw_moments, (long long)n, (const int8_t *)cm, (const float *)sm, (const uint8_t *)cv,
            (const float *)sv, (float *)ptr(m), (float *)ptr(v),
            (void *)c10::cuda::getCurrentCUDAStream(dev.index()).stream()))
    return nullptr;
  return pair(m, v);
  END_HANDLE_TH_ERRORS
}

// The weights of the norm: FP32, or of the rows' type.
Tensor norm_weight(PyObject *o, int64_t d, at::ScalarType t, c10::Device dev) {
  const Tensor &w = tensor(o, "weight");
  TORCH_CHECK_VALUE((w.scalar_type() == at::kFloat || w.scalar_type() == t) && w.dim() == 1 && w.size(0) == d && w.device() == dev,
                    "weight must be ", d, " values of float32 or of X's type on ", dev);
  return w.is_contiguous() ? w : w.contiguous();
}

// A matrix of the same shape, type and device as the first, or None.
Rows like(PyObject *o, const char *name, const Rows &x, at::ScalarType t, c10::Device dev) {
  if (o == Py_None) return {x.m, x.k, std::max(x.k, 1), nullptr};
  const Tensor &r = tensor(o, name);
  const Rows y = rows(r, name, r.scalar_type() == t, "one type and shape");
  TORCH_CHECK_VALUE(r.device() == dev && y.m == x.m && y.k == x.k, name, " must be (", x.m, ", ", x.k, ") ", t, " on ", dev);
  return y;
}

// rmsnorm(X, weight, residual, eps, out, out_h, scale, quantize): (y, h), or (q, scale, h)
PyObject *py_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(8)
  const bool q8 = a[7] == Py_True;
  const Tensor &X = tensor(a[0], "X");
  const at::ScalarType t = X.scalar_type();
  const Rows x = rows(X, "X", code(t) >= 0, kFloats);
  const c10::Device dev = X.device();
  const Rows r = like(a[2], "residual", x, t, dev);
  TORCH_CHECK_VALUE(a[2] != Py_None || a[5] == Py_None, "out_h needs a residual");
  c10::cuda::CUDAGuard on(dev);
  const Tensor w = norm_weight(a[1], x.k, t, dev);
  const double eps = real(a[3]);
  int ldy, ldh = std::max(x.k, 1);
  const Tensor y = out_rows(seen, a[4], "out", x.m, x.k, q8 ? at::kChar : t, dev, ldy);
  const Tensor h = a[2] == Py_None ? Tensor() : out_rows(seen, a[5], "out_h", x.m, x.k, t, dev, ldh);
  const Tensor scale = q8 ? out_vec(seen, a[6], "scale", x.m, at::kFloat, dev) : Tensor();
  const size_t e = X.element_size();
  const bool own_y = a[4] != Py_None, own_h = h.defined() && a[5] != Py_None, own_s = q8 && a[6] != Py_None;
  if (own_y || own_h || own_s) {
    const Area ax(x, e), ar(r, e), aw(w), as(own_s ? scale : Tensor()), ah = own_h ? Area(h, ldh) : Area(Tensor());
    if (own_y) {
      const Area ay(y, ldy);
      apart(ay, "out", ax, "X", !q8);
      apart(ay, "out", ar, "residual", !q8);
      apart(ay, "out", aw, "weight");
      apart(ay, "out", ah, "out_h");
      apart(as, "scale", ay, "out");
    }
    apart(ah, "out_h", ax, "X", true);
    apart(ah, "out_h", ar, "residual", true);
    apart(ah, "out_h", aw, "weight");
    apart(as, "scale", ax, "X");
    apart(as, "scale", ar, "residual");
    apart(as, "scale", aw, "weight");
    apart(as, "scale", ah, "out_h");
  }
  void *const stream = (void *)c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  const bool ok =
      q8 ? call("os2_rmsnorm_quantize", lib.rmsnorm_quantize, x.m, x.k, code(t), (const void *)x.p, x.ld, (const void *)r.p,
                r.ld, ptr(h), ldh, (const void *)ptr(w), code(w.scalar_type()), eps, (int8_t *)ptr(y), ldy,
                (float *)ptr(scale), stream)
         : call("os2_rmsnorm", lib.rmsnorm, x.m, x.k, code(t), (const void *)x.p, x.ld, (const void *)r.p, r.ld, ptr(h), ldh,
                (const void *)ptr(w), code(w.scalar_type()), eps, ptr(y), ldy, stream);
  if (!ok) return nullptr;
  written(a[4]), written(a[5]), written(a[6]);
  if (!q8) return h.defined() ? pair(y, h) : THPVariable_Wrap(y);
  if (!h.defined()) return pair(y, scale);
  THPObjectPtr py(THPVariable_Wrap(y)), ps(THPVariable_Wrap(scale)), ph(THPVariable_Wrap(h));
  return py && ps && ph ? PyTuple_Pack(3, py.get(), ps.get(), ph.get()) : nullptr;
  END_HANDLE_TH_ERRORS
}

// rmsnorm_backward(H, weight, dY, dH, eps, need_dx, need_dw, workspace): (dX, dW)
PyObject *py_rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(8)
  const Tensor &H = tensor(a[0], "H");
  const at::ScalarType t = H.scalar_type();
  const Rows h = rows(H, "H", code(t) >= 0, kFloats);
  const c10::Device dev = H.device();
  TORCH_CHECK_VALUE(a[2] != Py_None, "dY must be a tensor");
  const Rows dy = like(a[2], "dY", h, t, dev), dh = like(a[3], "dH", h, t, dev);
  const int need_dx = PyObject_IsTrue(a[5]), need_dw = PyObject_IsTrue(a[6]);
  if (need_dx < 0 || need_dw < 0) return nullptr;
  const double eps = real(a[4]);
  c10::cuda::CUDAGuard on(dev);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index());
  const Tensor w = norm_weight(a[1], h.k, t, dev);
  const Tensor dx = need_dx ? fresh(seen, {h.m, h.k}, t, dev) : Tensor(), dw = need_dw ? fresh(seen, {h.k}, w.scalar_type(), dev) : Tensor();
  const Tensor ws = workspace(a[7], need_dw ? lib.rmsnorm_workspace(h.m, h.k) : 0, dev, stream);
  if (!call("os2_rmsnorm_backward", lib.rmsnorm_backward, h.m, h.k, code(t), (const void *)h.p, h.ld, (const void *)ptr(w),
            code(w.scalar_type()), (const void *)dy.p, dy.ld, (const void *)dh.p, dh.ld, eps, ptr(dx), std::max(h.k, 1),
            ptr(dw), ptr(ws), size_t(ws.nbytes()), (void *)stream))
    return nullptr;
  return pair(dx, dw);
  END_HANDLE_TH_ERRORS
}

// A setting of each row: a tensor of n values, or a number for all.
template <class T>
Tensor setting(PyObject *o, const char *name, int64_t n, at::ScalarType t, c10::Device dev, T &all) {
  if (THPVariable_Check(o)) return vec(o, name, n, t, dev);
  if (std::is_same<T, int>::value) {
    const long long x = integer(o);
    all = T(std::min<long long>(std::max<long long>(x, 0), INT32_MAX));  // (below 1: no filter)
  } else {
    all = T(real(o));
  }
  return Tensor();
}

// sample(logits, u, temperature, top_k, top_p, min_p): (token, logprob)
PyObject *py_sample(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(6)
  const Tensor &Z = tensor(a[0], "logits");
  const Rows z = rows(Z, "logits", code(Z.scalar_type()) >= 0, kFloats);
  const c10::Device dev = Z.device();
  float t0 = 1, p0 = 1, m0 = 0;
  int k0 = 0;
  c10::cuda::CUDAGuard on(dev);
  const Tensor u = vec(a[1], "u", z.m, at::kFloat, dev), t = setting(a[2], "temperature", z.m, at::kFloat, dev, t0),
               k = setting(a[3], "top_k", z.m, at::kInt, dev, k0), p = setting(a[4], "top_p", z.m, at::kFloat, dev, p0),
               m = setting(a[5], "min_p", z.m, at::kFloat, dev, m0);
  const Tensor token = fresh(seen, {z.m}, at::kLong, dev), logprob = fresh(seen, {z.m}, at::kFloat, dev);
  if (!call("os2_sample", lib.sample, z.m, z.k, code(Z.scalar_type()), (const void *)z.p, z.ld, (const float *)ptr(u),
            (const float *)ptr(t), t0, (const int *)ptr(k), k0, (const float *)ptr(p), p0, (const float *)ptr(m), m0,
            (long long *)ptr(token), (float *)ptr(logprob), (void *)c10::cuda::getCurrentCUDAStream(dev.index()).stream()))
    return nullptr;
  return pair(token, logprob);
  END_HANDLE_TH_ERRORS
}

constexpr const char *kOneType = "bfloat16 or float16, one type for X and W";

// linear(X, W, bias, residual, activation, return_pre, out, workspace): Y, or (Y, pre)
PyObject *py_linear(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(8)
  const Tensor &X = tensor(a[0], "X"), &W = tensor(a[1], "W");
  const at::ScalarType t = X.scalar_type();
  const Rows x = rows(X, "X", t == at::kHalf || t == at::kBFloat16, kOneType), w = rows(W, "W", W.scalar_type() == t, kOneType);
  const c10::Device dev = X.device();
  TORCH_CHECK_VALUE(W.device() == dev, "W must be on ", dev);
  TORCH_CHECK_VALUE(w.k == x.k, "inner dimensions differ");
  const int m = x.m, n = w.m, k = x.k, act = int(integer(a[4]));
  c10::cuda::CUDAGuard on(dev);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index());
  const Tensor bias = a[2] == Py_None ? Tensor()
                                      : vec(a[2], "bias", n, tensor(a[2], "bias").scalar_type() == t ? t : at::kFloat, dev);
  const Rows r = like(a[3], "residual", Rows{m, n, 0, nullptr}, t, dev);
  int ldy;
  const Tensor Y = out_rows(seen, a[6], "out", m, n, t, dev, ldy), pre = a[5] == Py_True ? fresh(seen, {m, n}, t, dev) : Tensor();
  if (a[6] != Py_None) {
    const Area y(Y, ldy);
    apart(y, "out", Area(x, 2), "X");
    apart(y, "out", Area(w, 2), "W");
    apart(y, "out", Area(r, 2), "residual", true);
    apart(y, "out", Area(bias), "bias");
  }
  const Tensor ws = workspace(a[7], lib.linear_workspace(m, n, k, x.p, x.ld, w.p, w.ld), dev, stream);
  if (!call("os2_linear", lib.linear, m, n, k, code(t), (const void *)x.p, x.ld, (const void *)w.p, w.ld, (const void *)ptr(bias),
            bias.defined() ? code(bias.scalar_type()) : int(OS2_F32), act, (const void *)r.p, r.ld, ptr(Y), ldy, ptr(pre),
            std::max(n, 1), ptr(ws), size_t(ws.nbytes()), (void *)stream))
    return nullptr;
  written(a[6]);
  return pre.defined() ? pair(Y, pre) : THPVariable_Wrap(Y);
  END_HANDLE_TH_ERRORS
}

// linear_backward(X, W, dY, pre, activation, need_dx, need_dw, need_db, db_dtype, workspace): (dX, dW, db)
PyObject *py_linear_backward(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(10)
  const Tensor &X = tensor(a[0], "X"), &W = tensor(a[1], "W");
  const at::ScalarType t = X.scalar_type();
  const Rows x = rows(X, "X", t == at::kHalf || t == at::kBFloat16, kOneType), w = rows(W, "W", W.scalar_type() == t, kOneType);
  const c10::Device dev = X.device();
  TORCH_CHECK_VALUE(W.device() == dev, "W must be on ", dev);
  TORCH_CHECK_VALUE(w.k == x.k, "inner dimensions differ");
  const int m = x.m, n = w.m, k = x.k, act = int(integer(a[4]));
  TORCH_CHECK_VALUE(a[2] != Py_None, "dY must be a tensor");
  TORCH_CHECK_VALUE(act == OS2_ACT_NONE || a[3] != Py_None, "an activation's gradient needs pre (return_pre=True)");
  const Rows shape{m, n, 0, nullptr}, dy = like(a[2], "dY", shape, t, dev), pre = like(a[3], "pre", shape, t, dev);
  const int need_dx = PyObject_IsTrue(a[5]), need_dw = PyObject_IsTrue(a[6]), need_db = PyObject_IsTrue(a[7]);
  if (need_dx < 0 || need_dw < 0 || need_db < 0) return nullptr;
  at::ScalarType bt = t;
  if (a[8] != Py_None) {
    TORCH_CHECK_VALUE(THPDtype_Check(a[8]), "db_dtype must be a torch.dtype");
    bt = reinterpret_cast<THPDtype *>(a[8])->scalar_type;
    TORCH_CHECK_VALUE(bt == t || bt == at::kFloat, "db_dtype must be float32 or X's type");
  }
  c10::cuda::CUDAGuard on(dev);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index());
  const Tensor dx = need_dx ? fresh(seen, {m, k}, t, dev) : Tensor(), dw = need_dw ? fresh(seen, {n, k}, t, dev) : Tensor(),
               db = need_db ? fresh(seen, {n}, bt, dev) : Tensor();
  const Tensor ws = workspace(a[9], lib.linear_backward_workspace(m, n, k, x.p, x.ld, w.p, w.ld, dy.p, dy.ld, act), dev, stream);
  if (!call("os2_linear_backward", lib.linear_backward, m, n, k, code(t), (const void *)x.p, x.ld, (const void *)w.p, w.ld,
            (const void *)dy.p, dy.ld, (const void *)pre.p, pre.ld, act, ptr(dx), std::max(k, 1), ptr(dw), std::max(k, 1), ptr(db),
            code(bt), ptr(ws), size_t(ws.nbytes()), (void *)stream))
    return nullptr;
  THPObjectPtr px(THPVariable_Wrap(dx)), pw(THPVariable_Wrap(dw)), pb(THPVariable_Wrap(db));
  return px && pw && pb ? PyTuple_Pack(3, px.get(), pw.get(), pb.get()) : nullptr;
  END_HANDLE_TH_ERRORS
}

// bind(error, address of each function in the order of `lib`)
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(19)
  auto at = [&](int i) { return (void *)(uintptr_t)integer(a[i]); };
  lib.quantize_rows = (decltype(lib.quantize_rows))at(1);
  lib.i8_workspace = (decltype(lib.i8_workspace))at(2);
  lib.i8gemm = (decltype(lib.i8gemm))at(3);
  lib.i8linear = (decltype(lib.i8linear))at(4);
  lib.xent_workspace = (decltype(lib.xent_workspace))at(5);
  lib.xent = (decltype(lib.xent))at(6);
  lib.xent_backward = (decltype(lib.xent_backward))at(7);
  lib.adamw = (decltype(lib.adamw))at(8);
  lib.adamw_moments = (decltype(lib.adamw_moments))at(9);
  lib.rmsnorm = (decltype(lib.rmsnorm))at(10);
  lib.rmsnorm_quantize = (decltype(lib.rmsnorm_quantize))at(11);
  lib.rmsnorm_workspace = (decltype(lib.rmsnorm_workspace))at(12);
  lib.rmsnorm_backward = (decltype(lib.rmsnorm_backward))at(13);
  lib.sample = (decltype(lib.sample))at(14);
  lib.linear_workspace = (decltype(lib.linear_workspace))at(15);
  lib.linear = (decltype(lib.linear))at(16);
  lib.linear_backward_workspace = (decltype(lib.linear_backward_workspace))at(17);
  lib.linear_backward = (decltype(lib.linear_backward))at(18);
  Py_INCREF(a[0]);
  g_error = a[0];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define OS2_METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {OS2_METHOD(bind),  OS2_METHOD(quantize_rows), OS2_METHOD(i8),
                         OS2_METHOD(xent),  OS2_METHOD(xent_backward), OS2_METHOD(adamw),
                         OS2_METHOD(adamw_moments), OS2_METHOD(rmsnorm), OS2_METHOD(rmsnorm_backward),
                         OS2_METHOD(sample),    OS2_METHOD(linear),  OS2_METHOD(linear_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "os2_head", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_os2_head(void) { return PyModule_Create(&module); }
