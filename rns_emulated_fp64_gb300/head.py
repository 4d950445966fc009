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

import contextlib
import ctypes as ct

import torch

from .binding import _check, _stream, alloc_workspace, load

F32, F16, BF16 = 0, 1, 2
_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
ADAMW_BLOCK = 256  # elements that share a scale of an 8-bit moment


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Device and stream of a call; what it allocates and copies belongs to them."""
    if stream is None:
        return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _rows(X, name, dtypes):
    """A 2-D CUDA tensor with contiguous rows; returns its leading dimension."""
    if not (X.is_cuda and X.dim() == 2 and X.dtype in dtypes):
        raise ValueError(f"{name} must be a 2-D CUDA tensor of " + ", ".join(str(t) for t in dtypes))
    if X.shape[1] > 1 and X.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return _ld(X)


def _ld(X):
    # the stride of a single row means nothing
    return max(X.stride(0) if X.shape[0] > 1 else 0, X.shape[1], 1)


def _vector(x, name, n, dtype, device):
    if x.dtype != dtype or x.device != device or x.dim() != 1 or x.shape[0] != n:
        raise ValueError(f"{name} must be {n} {dtype} values on {device}")
    return x if x.is_contiguous() else x.contiguous()


def _out(out, shape, dtype, device, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != device:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on {device}")
    if out.dim() == 2 and out.shape[1] > 1 and out.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if out.dim() == 2 and out.shape[0] > 1 and out.stride(0) < out.shape[1]:
        raise ValueError(f"{name} must not overlap itself")
    if out.dim() == 1 and not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return out


def _workspace(workspace, need, device):
    if workspace is None:
        return alloc_workspace(need, device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace


def _nbytes(t):
    return t.numel() * t.element_size()


# ------------------------------------------------------------------- 8 bits
def quantize_rows(X: torch.Tensor, out=None, scale=None, stream=None):
    """8-bit integers of X (m x k, float32, float16 or bfloat16) with one scale
    a row: returns (q int8, scale float32), X ~ q * scale[:, None].  Weights are
    quantised by output channel the same way, as n x k."""
    ld = _rows(X, "X", tuple(_DTYPE))
    m, k = X.shape
    with _on(X.device, stream):
        q = _out(out, (m, k), torch.int8, X.device)
        scale = _out(scale, (m,), torch.float32, X.device, "scale")
        _check(load().os2_quantize_rows(m, k, _DTYPE[X.dtype], X.data_ptr(), ld, q.data_ptr(),
                                        _ld(q), scale.data_ptr(), _stream(None)),
               "os2_quantize_rows")
    return q, scale


def _i8(X, ldx, a_scale, Bt, b_scale, bias, out_dtype, out, workspace, stream):
    ldb = _rows(Bt, "Bt", (torch.int8,))
    m, k = X.shape
    n = Bt.shape[0]
    dev = X.device
    if Bt.device != dev:
        raise ValueError(f"Bt must be on {dev}")
    if Bt.shape[1] != k:
        raise ValueError("inner dimensions differ")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be float32, float16 or bfloat16")
    L = load()
    with _on(dev, stream):
        if a_scale is not None:
            a_scale = _vector(a_scale, "a_scale", m, torch.float32, dev)
        b_scale = _vector(b_scale, "b_scale", n, torch.float32, dev)
        if bias is not None:
            bias = _vector(bias, "bias", n, torch.float32, dev)
        out = _out(out, (m, n), out_dtype, dev)
        ws = _workspace(workspace, L.os2_i8gemm_workspace_size(m, n, k, Bt.data_ptr(), ldb), dev)
        rest = (Bt.data_ptr(), ldb, b_scale.data_ptr(), None if bias is None else bias.data_ptr(),
                out.data_ptr(), _ld(out), _DTYPE[out_dtype], ws.data_ptr(), _nbytes(ws),
                _stream(None))
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
    lda = _rows(A, "A", (torch.int8,))
    return _i8(A, lda, a_scale, Bt, b_scale, bias, out_dtype, out, workspace, stream)


def i8linear(X: torch.Tensor, Bt: torch.Tensor, b_scale: torch.Tensor, bias=None, out_dtype=None,
             out=None, workspace=None, stream=None) -> torch.Tensor:
    """A linear layer with 8-bit weights: X (m x k, float32, float16 or
    bfloat16) is quantised token by token (``quantize_rows``), then ``i8gemm``.
    out_dtype: X's by default."""
    ldx = _rows(X, "X", tuple(_DTYPE))
    if out_dtype is None and out is None:
        out_dtype = X.dtype
    return _i8(X, ldx, None, Bt, b_scale, bias, out_dtype, out, workspace, stream)


# ------------------------------------------------------------ cross entropy
def _head(H, W):
    ldh, ldw = _rows(H, "H", (torch.bfloat16, torch.float16)), _rows(W, "W", (H.dtype,))
    if W.device != H.device:
        raise ValueError(f"W must be on {H.device}")
    if H.shape[1] != W.shape[1]:
        raise ValueError("inner dimensions differ")
    return ldh, ldw


def xent(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100,
         workspace=None, stream=None):
    """Softmax cross entropy of the logits H @ W.T without the logits.

    H: n x k, W: v x k, bfloat16 or float16; labels: n int64.  Returns (loss,
    lse), float32, one value a row; 0 for rows labelled ignore_index.  A label
    out of range is reported by ``get_status`` (ERR_RANGE)."""
    ldh, ldw = _head(H, W)
    (n, k), v, dev = H.shape, W.shape[0], H.device
    L = load()
    with _on(dev, stream):
        labels = _vector(labels, "labels", n, torch.int64, dev)
        loss = torch.empty(n, dtype=torch.float32, device=dev)
        lse = torch.empty(n, dtype=torch.float32, device=dev)
        ws = _workspace(workspace, L.os2_xent_workspace_size(n, k, v, W.data_ptr(), ldw, 0), dev)
        _check(L.os2_xent(n, k, v, _DTYPE[H.dtype], H.data_ptr(), ldh, W.data_ptr(), ldw,
                          labels.data_ptr(), int(ignore_index), loss.data_ptr(), lse.data_ptr(),
                          ws.data_ptr(), _nbytes(ws), _stream(None)), "os2_xent")
    return loss, lse


def xent_backward(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor,
                  grad: torch.Tensor, ignore_index: int = -100, need_dh: bool = True,
                  need_dw: bool = True, workspace=None, stream=None):
    """The gradient of ``xent``: (dH, dW) for grad = d/d loss (n float32 values),
    in H's type; None for the one not needed."""
    ldh, ldw = _head(H, W)
    (n, k), v, dev = H.shape, W.shape[0], H.device
    L = load()
    with _on(dev, stream):
        labels = _vector(labels, "labels", n, torch.int64, dev)
        lse = _vector(lse, "lse", n, torch.float32, dev)
        grad = _vector(grad, "grad", n, torch.float32, dev)
        dh = torch.empty((n, k), dtype=H.dtype, device=dev) if need_dh else None
        dw = torch.empty((v, k), dtype=H.dtype, device=dev) if need_dw else None
        ws = _workspace(workspace, L.os2_xent_workspace_size(n, k, v, W.data_ptr(), ldw, 1), dev)
        _check(L.os2_xent_backward(n, k, v, _DTYPE[H.dtype], H.data_ptr(), ldh, W.data_ptr(), ldw,
                                   labels.data_ptr(), int(ignore_index), lse.data_ptr(),
                                   grad.data_ptr(), None if dh is None else dh.data_ptr(), k,
                                   None if dw is None else dw.data_ptr(), k, ws.data_ptr(),
                                   _nbytes(ws), _stream(None)), "os2_xent_backward")
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
def _pointers(ts):
    return (ct.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def _list(ts, name, like, dtypes):
    if len(ts) != len(like):
        raise ValueError(f"{name}: {len(ts)} tensors for {len(like)} parameters")
    dtype = ts[0].dtype
    if dtype not in dtypes:
        raise ValueError(f"{name} must be " + " or ".join(str(t) for t in dtypes))
    for t, p in zip(ts, like):
        if t.dtype != dtype or t.device != p.device or t.shape != p.shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous, of one type, and match the parameters")


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
    dev = params[0].device
    if dev.type != "cuda" or any(p.device != dev for p in params):
        raise ValueError("params must be on one CUDA device")
    _list(params, "params", params, tuple(_DTYPE))
    _list(grads, "grads", params, tuple(_DTYPE))
    q8 = exp_avg_scales is not None or exp_avg_sq_scales is not None
    _list(exp_avg, "exp_avg", params, (torch.int8,) if q8 else (torch.float32,))
    _list(exp_avg_sq, "exp_avg_sq", params, (torch.uint8,) if q8 else (torch.float32,))
    sizes = [p.numel() for p in params]
    scales = (None, None)
    if q8:
        for ss, name in ((exp_avg_scales, "exp_avg_scales"), (exp_avg_sq_scales, "exp_avg_sq_scales")):
            if ss is None or len(ss) != len(params):
                raise ValueError(f"{name}: one tensor for each parameter")
            for s, n in zip(ss, sizes):
                if (s.dtype != torch.float32 or s.device != dev or not s.is_contiguous() or
                        s.numel() != -(-n // ADAMW_BLOCK)):
                    raise ValueError(f"{name} must be contiguous float32, one value for each "
                                     f"{ADAMW_BLOCK} elements")
        scales = _pointers(exp_avg_scales), _pointers(exp_avg_sq_scales)
    with _on(dev, stream):
        _check(load().os2_adamw(len(params), (ct.c_longlong * len(params))(*sizes),
                                _pointers(params), _pointers(grads), _pointers(exp_avg),
                                _pointers(exp_avg_sq), *scales, _DTYPE[params[0].dtype],
                                _DTYPE[grads[0].dtype], 8 if q8 else 32, lr, beta1, beta2, eps,
                                weight_decay, int(step), _stream(None)), "os2_adamw")


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
    with _on(exp_avg.device, stream):
        m = torch.empty(exp_avg.shape, dtype=torch.float32, device=exp_avg.device)
        v = torch.empty_like(m)
        _check(load().os2_adamw_moments(n, exp_avg.data_ptr(), exp_avg_scale.data_ptr(),
                                        exp_avg_sq.data_ptr(), exp_avg_sq_scale.data_ptr(),
                                        m.data_ptr(), v.data_ptr(), _stream(None)),
               "os2_adamw_moments")
    return m, v
