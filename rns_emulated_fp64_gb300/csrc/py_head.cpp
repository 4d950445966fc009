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

#include <ATen/ops/empty.h>
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

Tensor fresh(at::IntArrayRef shape, at::ScalarType t, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(t).device(dev));
}

// The output, the caller's or a new one, and its leading dimension.
Tensor out_rows(PyObject *o, const char *name, int64_t m, int64_t n, at::ScalarType t, c10::Device dev, int &ld) {
  ld = as_int(std::max<int64_t>(n, 1), name);
  if (o == Py_None) return fresh({m, n}, t, dev);
  const Tensor &x = tensor(o, name);
  TORCH_CHECK_VALUE(x.dim() == 2 && x.size(0) == m && x.size(1) == n && x.scalar_type() == t && x.device() == dev, name,
                    " must be (", m, ", ", n, ") ", t, " on ", dev);
  TORCH_CHECK_VALUE(n <= 1 || x.stride(1) == 1, name, " must have contiguous rows");
  TORCH_CHECK_VALUE(m <= 1 || x.stride(0) >= n, name, " must not overlap itself");
  if (m > 1) ld = as_int(std::max<int64_t>(x.stride(0), ld), name);
  return x;
}

Tensor out_vec(PyObject *o, const char *name, int64_t n, at::ScalarType t, c10::Device dev) {
  if (o == Py_None) return fresh({n}, t, dev);
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
  if (need > kKeep || c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    return fresh({int64_t(need)}, at::kByte, dev);
  static thread_local Kept kept;
  Tensor &ws = kept[{dev.index(), stream}];
  if (!ws.defined() || size_t(ws.numel()) < need)
    ws = fresh({int64_t(std::min(kKeep, std::max(size_t(1) << 20, 2 * need)))}, at::kByte, dev);
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
  }

constexpr const char *kFloats = "float32, float16 or bfloat16", *kHalves = "bfloat16 or float16, one type for H and W";

// quantize_rows(X, out, scale)
PyObject *py_quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(3)
  const Tensor &X = tensor(a[0], "X");
  const Rows x = rows(X, "X", code(X.scalar_type()) >= 0, kFloats);
  const c10::Device dev = X.device();
  c10::cuda::CUDAGuard on(dev);
  int ldq;
  const Tensor q = out_rows(a[1], "out", x.m, x.k, at::kChar, dev, ldq), scale = out_vec(a[2], "scale", x.m, at::kFloat, dev);
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
  const Tensor C = out_rows(a[6], "out", m, n, ct, dev, ldc);
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
  const Tensor y = vec(a[2], "labels", n, at::kLong, t.dev), loss = fresh({n}, at::kFloat, t.dev),
               lse = fresh({n}, at::kFloat, t.dev);
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
  const Tensor dh = need_dh ? fresh({n, k}, dt, t.dev) : Tensor(), dw = need_dw ? fresh({v, k}, dt, t.dev) : Tensor();
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
  const Tensor m = fresh(c.sizes(), at::kFloat, dev), v = fresh(c.sizes(), at::kFloat, dev);
  if (!call("os2_adamw_moments", lib.adamw_moments, (long long)n, (const int8_t *)cm, (const float *)sm, (const uint8_t *)cv,
            (const float *)sv, (float *)ptr(m), (float *)ptr(v),
            (void *)c10::cuda::getCurrentCUDAStream(dev.index()).stream()))
    return nullptr;
  return pair(m, v);
  END_HANDLE_TH_ERRORS
}

// bind(error, address of each function in the order of `lib`)
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
  OS2_ARGS(10)
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
  Py_INCREF(a[0]);
  g_error = a[0];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define OS2_METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {OS2_METHOD(bind),  OS2_METHOD(quantize_rows), OS2_METHOD(i8),
                         OS2_METHOD(xent),  OS2_METHOD(xent_backward), OS2_METHOD(adamw),
                         OS2_METHOD(adamw_moments), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "os2_head", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_os2_head(void) { return PyModule_Create(&module); }
