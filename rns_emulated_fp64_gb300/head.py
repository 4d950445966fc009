"""Operators of a language model's vocabulary head (include/os2.h).

Argument checks and marshalling only, as in ``binding``: the compute runs in
the CUDA kernels of libos2, on the current stream (or ``stream``), and nothing
synchronises.  Every tensor of a call lives on one CUDA device.

  i8linear, i8gemm, quantize_rows   the product in 8-bit integers with a scale
                                    for each token and each output channel
  xent, xent_backward, XentFunction softmax cross entropy of H W^T and its
                                    gradient, without the logits in memory
  adamw, adamw_moments              an AdamW step over many tensors, moments in
                                    32 or in 8 bits
"""
from __future__ import annotations

import array
import contextlib
import operator
import threading

import torch

from .binding import _check, load

F32, F16, BF16 = 0, 1, 2
_INT8, _HALVES = (torch.int8,), (torch.bfloat16, torch.float16)
_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
ADAMW_BLOCK = 256  # elements that share a scale of an 8-bit moment


_HERE = contextlib.nullcontext()


def _on(index, stream):
    """Device and stream of a call; what it allocates and copies belongs to them."""
    if stream is None:
        return _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    return torch.cuda.stream(stream)


# the current stream's handle, without a Stream object around it (3 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _rows(X, name, dtypes):
    """Checks a 2-D CUDA tensor with contiguous rows; returns (rows, columns,
    leading dimension)."""
    if X.dim() != 2 or X.dtype not in dtypes or not X.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of " + ", ".join(str(t) for t in dtypes))
    (m, k), (ld, inner) = X.shape, X.stride()
    if inner != 1 and k > 1:
        raise ValueError(f"{name} must have contiguous rows")
    # the stride of a single row means nothing
    return m, k, (ld if m > 1 and ld > k else k if k else 1)


def _vector(x, name, n, dtype, index):
    if x.dtype is not dtype or x.dim() != 1 or x.shape[0] != n or x.get_device() != index:
        raise ValueError(f"{name} must be {n} {dtype} values on cuda:{index}")
    return x if x.is_contiguous() else x.contiguous()


def _out(out, like, shape, dtype, name="out"):
    """The output and its leading dimension."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device), shape[-1] or 1
    if tuple(out.shape) != shape or out.dtype is not dtype or out.device != like.device:
        raise ValueError(f"{name} must be {shape} {dtype} on {like.device}")
    if len(shape) == 1:
        if not out.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return out, shape[0]
    if shape[1] > 1 and out.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if shape[0] > 1 and out.stride(0) < shape[1]:
        raise ValueError(f"{name} must not overlap itself")
    return out, max(out.stride(0) if shape[0] > 1 else 0, shape[1], 1)


_KEEP = 32 << 20           # bytes of a workspace that is kept for the next call
_kept = threading.local()  # of a thread: {(device, stream): workspace}


def _workspace(workspace, need, like, index):
    """The call's workspace: the caller's, or one of the binding's own.  Small ones
    are kept, one for each thread, device and stream (calls that share one are
    ordered by the stream), because an allocation between two launches costs as
    much host time as a launch; a captured call gets its own."""
    if workspace is not None:
        if workspace.device != like.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {like.device}")
        return workspace
    if need > _KEEP or torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    kept, key = _kept.__dict__, (index, _raw_stream(index))
    ws = kept.get(key)
    if ws is None or ws.numel() < need:
        size = min(_KEEP, max(1 << 20, 2 * need))
        ws = kept[key] = torch.empty(size, dtype=torch.uint8, device=like.device)
    return ws


def _nbytes(t):
    return t.numel() * t.element_size()


# ------------------------------------------------------------------- 8 bits
def quantize_rows(X: torch.Tensor, out=None, scale=None, stream=None):
    """8-bit integers of X (m x k, float32, float16 or bfloat16) with one scale
    a row: returns (q int8, scale float32), X ~ q * scale[:, None].  Weights are
    quantised by output channel the same way, as n x k."""
    m, k, ld = _rows(X, "X", _DTYPE)
    index = X.get_device()
    with _on(index, stream):
        q, ldq = _out(out, X, (m, k), torch.int8)
        scale, _ = _out(scale, X, (m,), torch.float32, "scale")
        _check(load().os2_quantize_rows(m, k, _DTYPE[X.dtype], X.data_ptr(), ld, q.data_ptr(), ldq,
                                        scale.data_ptr(), _raw_stream(index)), "os2_quantize_rows")
    return q, scale


def _i8(X, m, k, ldx, a_scale, Bt, b_scale, bias, out_dtype, out, workspace, stream):
    n, kb, ldb = _rows(Bt, "Bt", _INT8)
    index = X.get_device()
    if Bt.get_device() != index:
        raise ValueError(f"Bt must be on {X.device}")
    if kb != k:
        raise ValueError("inner dimensions differ")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be float32, float16 or bfloat16")
    L = load()
    with _on(index, stream):
        if a_scale is not None:
            a_scale = _vector(a_scale, "a_scale", m, torch.float32, index)
        b_scale = _vector(b_scale, "b_scale", n, torch.float32, index)
        if bias is not None:
            bias = _vector(bias, "bias", n, torch.float32, index)
        out, ldc = _out(out, X, (m, n), out_dtype)
        bp = Bt.data_ptr()
        ws = _workspace(workspace, L.os2_i8gemm_workspace_size(m, n, k, bp, ldb), X, index)
        rest = (bp, ldb, b_scale.data_ptr(), None if bias is None else bias.data_ptr(),
                out.data_ptr(), ldc, _DTYPE[out_dtype], ws.data_ptr(), _nbytes(ws),
                _raw_stream(index))
        if a_scale is not None:
            _check(L.os2_i8gemm(m, n, k, X.data_ptr(), ldx, a_scale.data_ptr(), *rest),
                   "os2_i8gemm")
        else:
            _check(L.os2_i8linear(m, n, k, _DTYPE[X.dtype], X.data_ptr(), ldx, *rest),
                   "os2_i8linear")
    return out


def i8gemm(A: torch.Tensor, a_scale: torch.Tensor, Bt: torch.Tensor, b_scale: torch.Tensor,
           bias=None, out_dtype=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """(A @ Bt.T) * a_scale[:, None] * b_scale + bias, the integer product exact.

    A: m x k int8 (tokens), Bt: n x k int8 (output channels), scales and bias
    float32.  out_dtype: float32, float16 or bfloat16 (the default)."""
    m, k, lda = _rows(A, "A", _INT8)
    if a_scale is None:
        raise ValueError("a_scale is missing")
    return _i8(A, m, k, lda, a_scale, Bt, b_scale, bias, out_dtype, out, workspace, stream)


def i8linear(X: torch.Tensor, Bt: torch.Tensor, b_scale: torch.Tensor, bias=None, out_dtype=None,
             out=None, workspace=None, stream=None) -> torch.Tensor:
    """A linear layer with 8-bit weights: X (m x k, float32, float16 or
    bfloat16) is quantised token by token (``quantize_rows``), then ``i8gemm``.
    out_dtype: X's by default."""
    m, k, ldx = _rows(X, "X", _DTYPE)
    if out_dtype is None and out is None:
        out_dtype = X.dtype
    return _i8(X, m, k, ldx, None, Bt, b_scale, bias, out_dtype, out, workspace, stream)


# ------------------------------------------------------------ cross entropy
def _head(H, W):
    n, k, ldh = _rows(H, "H", _HALVES)
    v, kw, ldw = _rows(W, "W", (H.dtype,))
    index = H.get_device()
    if W.get_device() != index:
        raise ValueError(f"W must be on {H.device}")
    if kw != k:
        raise ValueError("inner dimensions differ")
    return n, k, v, ldh, ldw, index


def xent(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100,
         workspace=None, stream=None):
    """Softmax cross entropy of the logits H @ W.T without the logits.

    H: n x k, W: v x k, bfloat16 or float16; labels: n int64.  Returns (loss,
    lse), float32, one value a row; 0 for rows labelled ignore_index.  A label
    out of range is reported by ``get_status`` (ERR_RANGE)."""
    n, k, v, ldh, ldw, index = _head(H, W)
    L = load()
    with _on(index, stream):
        labels = _vector(labels, "labels", n, torch.int64, index)
        dev = H.device
        loss = torch.empty(n, dtype=torch.float32, device=dev)
        lse = torch.empty(n, dtype=torch.float32, device=dev)
        wp = W.data_ptr()
        ws = _workspace(workspace, L.os2_xent_workspace_size(n, k, v, wp, ldw, 0), H, index)
        _check(L.os2_xent(n, k, v, _DTYPE[H.dtype], H.data_ptr(), ldh, wp, ldw, labels.data_ptr(),
                          int(ignore_index), loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                          _nbytes(ws), _raw_stream(index)), "os2_xent")
    return loss, lse


def xent_backward(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor,
                  grad: torch.Tensor, ignore_index: int = -100, need_dh: bool = True,
                  need_dw: bool = True, workspace=None, stream=None):
    """The gradient of ``xent``: (dH, dW) for grad = d/d loss (n float32 values),
    in H's type; None for the one not needed."""
    n, k, v, ldh, ldw, index = _head(H, W)
    L = load()
    with _on(index, stream):
        labels = _vector(labels, "labels", n, torch.int64, index)
        lse = _vector(lse, "lse", n, torch.float32, index)
        grad = _vector(grad, "grad", n, torch.float32, index)
        dt, dev = H.dtype, H.device
        dh = torch.empty((n, k), dtype=dt, device=dev) if need_dh else None
        dw = torch.empty((v, k), dtype=dt, device=dev) if need_dw else None
        wp = W.data_ptr()
        ws = _workspace(workspace, L.os2_xent_workspace_size(n, k, v, wp, ldw, 1), H, index)
        _check(L.os2_xent_backward(n, k, v, _DTYPE[H.dtype], H.data_ptr(), ldh, wp, ldw,
                                   labels.data_ptr(), int(ignore_index), lse.data_ptr(),
                                   grad.data_ptr(), None if dh is None else dh.data_ptr(), k,
                                   None if dw is None else dw.data_ptr(), k, ws.data_ptr(),
                                   _nbytes(ws), _raw_stream(index)), "os2_xent_backward")
    return dh, dw


class XentFunction(torch.autograd.Function):
    """``xent`` for autograd: XentFunction.apply(H, W, labels, ignore_index) gives
    the losses, row by row; their mean, sum or weights are ordinary operations."""

    @staticmethod
    def forward(ctx, H, W, labels, ignore_index=-100):
        loss, lse = xent(H, W, labels, ignore_index)
        ctx.save_for_backward(H, W, labels, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    def backward(ctx, grad):
        H, W, labels, lse = ctx.saved_tensors
        dh, dw = xent_backward(H, W, labels, lse, grad.float(), ctx.ignore_index,
                               ctx.needs_input_grad[0], ctx.needs_input_grad[1])
        return dh, dw, None, None


# -------------------------------------------------------------------- AdamW
_dtype_of, _shape_of = operator.attrgetter("dtype"), operator.attrgetter("shape")


def _pointers(ts):
    return array.array("Q", map(torch.Tensor.data_ptr, ts))


def _address(a):
    return None if a is None else a.buffer_info()[0]


def _list(ts, name, shapes, index, dtypes):
    """Checks a list of tensors, one for each parameter; returns their type."""
    if len(ts) != len(shapes):
        raise ValueError(f"{name}: {len(ts)} tensors for {len(shapes)} parameters")
    types = set(map(_dtype_of, ts))
    dtype = types.pop()
    if types or dtype not in dtypes:
        raise ValueError(f"{name} must be all " + " or all ".join(str(t) for t in dtypes))
    if (list(map(_shape_of, ts)) != shapes or set(map(torch.Tensor.get_device, ts)) != {index} or
            not all(map(torch.Tensor.is_contiguous, ts))):
        raise ValueError(f"{name} must be contiguous, on one CUDA device, and of the parameters' "
                         "shapes")
    return dtype


def adamw(params, grads, exp_avg, exp_avg_sq, *, step: int, lr: float, beta1: float = 0.9,
          beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
          exp_avg_scales=None, exp_avg_sq_scales=None, stream=None):
    """One AdamW step, number ``step`` (from 1), in place, over lists of
    contiguous CUDA tensors: params and grads float32, float16 or bfloat16 (one
    type each), moments float32, or 8-bit codes (exp_avg int8, exp_avg_sq uint8)
    with float32 scales, one for each ADAMW_BLOCK elements of a tensor.  Zero
    codes and scales are the initial state."""
    params = list(params)
    if not params:
        return
    index = params[0].get_device()
    if index < 0:
        raise ValueError("params must be on one CUDA device")
    shapes = list(map(_shape_of, params))
    pt = _list(params, "params", shapes, index, _DTYPE)
    gt = _list(grads, "grads", shapes, index, _DTYPE)
    q8 = exp_avg_scales is not None or exp_avg_sq_scales is not None
    _list(exp_avg, "exp_avg", shapes, index, _INT8 if q8 else (torch.float32,))
    _list(exp_avg_sq, "exp_avg_sq", shapes, index, (torch.uint8,) if q8 else (torch.float32,))
    sizes = list(map(torch.Tensor.numel, params))
    scales = (None, None)
    if q8:
        for ss, name in ((exp_avg_scales, "exp_avg_scales"), (exp_avg_sq_scales, "exp_avg_sq_scales")):
            if ss is None or len(ss) != len(params):
                raise ValueError(f"{name}: one tensor for each parameter")
            if (set(map(_dtype_of, ss)) != {torch.float32} or
                    set(map(torch.Tensor.get_device, ss)) != {index} or
                    not all(map(torch.Tensor.is_contiguous, ss)) or
                    list(map(torch.Tensor.numel, ss)) != [-(-n // ADAMW_BLOCK) for n in sizes]):
                raise ValueError(f"{name} must be contiguous float32, one value for each "
                                 f"{ADAMW_BLOCK} elements")
        scales = _pointers(exp_avg_scales), _pointers(exp_avg_sq_scales)
    with _on(index, stream):
        # host arrays, read before the call returns
        arrays = [array.array("q", sizes), *map(_pointers, (params, grads, exp_avg, exp_avg_sq)),
                  *scales]
        _check(load().os2_adamw(len(params), *map(_address, arrays), _DTYPE[pt], _DTYPE[gt],
                                8 if q8 else 32, lr, beta1, beta2, eps, weight_decay, int(step),
                                _raw_stream(index)), "os2_adamw")


def adamw_moments(exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, stream=None):
    """The float32 values (m, v) that 8-bit moments stand for: one tensor's
    codes and scales, or storage of several laid out on blocks of ADAMW_BLOCK."""
    n = exp_avg.numel()
    for t, name, dtype, size in ((exp_avg, "exp_avg", torch.int8, n),
                                 (exp_avg_sq, "exp_avg_sq", torch.uint8, n),
                                 (exp_avg_scale, "exp_avg_scale", torch.float32, -(-n // ADAMW_BLOCK)),
                                 (exp_avg_sq_scale, "exp_avg_sq_scale", torch.float32, -(-n // ADAMW_BLOCK))):
        if not t.is_cuda or t.device != exp_avg.device or t.dtype != dtype or t.numel() != size or not t.is_contiguous():
            raise ValueError(f"{name} must be {size} contiguous {dtype} values on one CUDA device")
    index = exp_avg.get_device()
    with _on(index, stream):
        m = torch.empty(exp_avg.shape, dtype=torch.float32, device=exp_avg.device)
        v = torch.empty_like(m)
        _check(load().os2_adamw_moments(n, exp_avg.data_ptr(), exp_avg_scale.data_ptr(),
                                        exp_avg_sq.data_ptr(), exp_avg_sq_scale.data_ptr(),
                                        m.data_ptr(), v.data_ptr(), _raw_stream(index)),
               "os2_adamw_moments")
    return m, v
