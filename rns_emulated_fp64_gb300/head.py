"""Operators of a language model's vocabulary head (include/os2.h).

Argument checks and marshalling only, as in ``binding``, and native
(csrc/py_head.cpp), because the smallest calls are host bound: the compute runs
in the CUDA kernels of libos2, on the current stream (or ``stream``), and nothing
synchronises.  Every tensor of a call lives on one CUDA device.  A call that is
given no workspace uses one that the binding keeps for the thread and stream, if
32 MB are enough.

  i8linear, i8gemm, quantize_rows   the product in 8-bit integers with a scale
                                    for each token and each output channel
  xent, xent_backward, XentFunction softmax cross entropy of H W^T and its
                                    gradient, without the logits in memory
  adamw, adamw_moments              an AdamW step over many tensors, moments in
                                    32 or in 8 bits
"""
from __future__ import annotations

import torch

from .binding import load_head

ADAMW_BLOCK = 256  # elements that share a scale of an 8-bit moment


def _run(f, stream, like, *args):
    """The call; what it allocates and copies belongs to its stream."""
    if stream is None or not hasattr(like, "get_device"):  # (no tensor: nothing to do, or f's error)
        return f(*args)
    index = like.get_device()
    if index < 0:
        raise ValueError("every tensor must be on one CUDA device")
    if not isinstance(stream, torch.cuda.Stream):
        # The default stream has the handles 0 and 1 (the legacy one), neither of which
        # ExternalStream takes for it.
        handle = int(stream)
        stream = (torch.cuda.default_stream(index) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=index))
    elif stream.device_index != index:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{index}")
    with torch.cuda.stream(stream):
        return f(*args)


# ------------------------------------------------------------------- 8 bits
def quantize_rows(X: torch.Tensor, out=None, scale=None, stream=None):
    """8-bit integers of X (m x k, float32, float16 or bfloat16) with one scale
    a row: returns (q int8, scale float32), X ~ q * scale[:, None].  Weights are
    quantised by output channel the same way, as n x k."""
    return _run(load_head().quantize_rows, stream, X, X, out, scale)


def i8gemm(A: torch.Tensor, a_scale: torch.Tensor, Bt: torch.Tensor, b_scale: torch.Tensor,
           bias=None, out_dtype=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """(A @ Bt.T) * a_scale[:, None] * b_scale + bias, the integer product exact.

    A: m x k int8 (tokens), Bt: n x k int8 (output channels), scales and bias
    float32.  out_dtype: float32, float16 or bfloat16 (the default)."""
    return _run(load_head().i8, stream, A, A, a_scale, Bt, b_scale, bias, out_dtype, out, workspace,
                False)


def i8linear(X: torch.Tensor, Bt: torch.Tensor, b_scale: torch.Tensor, bias=None, out_dtype=None,
             out=None, workspace=None, stream=None) -> torch.Tensor:
    """A linear layer with 8-bit weights: X (m x k, float32, float16 or
    bfloat16) is quantised token by token (``quantize_rows``), then ``i8gemm``.
    out_dtype: X's by default."""
    return _run(load_head().i8, stream, X, X, None, Bt, b_scale, bias, out_dtype, out, workspace,
                True)


# ------------------------------------------------------------ cross entropy
def xent(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100,
         workspace=None, stream=None):
    """Softmax cross entropy of the logits H @ W.T without the logits.

    H: n x k, W: v x k, bfloat16 or float16; labels: n int64.  Returns (loss,
    lse), float32, one value a row; 0 for rows labelled ignore_index.  A label
    out of range is reported by ``get_status`` (ERR_RANGE).  A width that is a
    multiple of 8 (rows of W on 16-byte boundaries) saves a copy of W in each call."""
    return _run(load_head().xent, stream, H, H, W, labels, ignore_index, workspace)


def xent_backward(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor,
                  grad: torch.Tensor, ignore_index: int = -100, need_dh: bool = True,
                  need_dw: bool = True, workspace=None, stream=None):
    """The gradient of ``xent``: (dH, dW) for grad = d/d loss (n float32 values),
    in H's type; None for the one not needed."""
    return _run(load_head().xent_backward, stream, H, H, W, labels, lse, grad, ignore_index, need_dh,
                need_dw, workspace)


class XentFunction(torch.autograd.Function):
    """``xent`` for autograd: XentFunction.apply(H, W, labels, ignore_index) gives
    the losses, row by row; their mean, sum or weights are ordinary operations.
    The gradient has no gradient of its own: to go back through it raises."""

    @staticmethod
    def forward(ctx, H, W, labels, ignore_index=-100):
        loss, lse = xent(H, W, labels, ignore_index)
        ctx.save_for_backward(H, W, labels, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    def backward(ctx, grad):
        H, W, labels, lse = ctx.saved_tensors
        # (with create_graph only is a gradient taken while autograd records)
        gradient = _XentGradient.apply if torch.is_grad_enabled() else xent_backward
        dh, dw = gradient(H, W, labels, lse, grad.float(), ctx.ignore_index,
                          ctx.needs_input_grad[0], ctx.needs_input_grad[1])
        return dh, dw, None, None


class _XentGradient(torch.autograd.Function):
    """``xent_backward`` where a graph of the gradient is asked for: a function of H, W
    and grad that raises when it is differentiated, instead of a constant."""

    @staticmethod
    def forward(ctx, H, W, labels, lse, grad, ignore_index, need_dh, need_dw):
        return xent_backward(H, W, labels, lse, grad, ignore_index, need_dh, need_dw)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("XentFunction: the gradient has no gradient of its own")


# -------------------------------------------------------------------- AdamW
def adamw(params, grads, exp_avg, exp_avg_sq, *, step: int, lr: float, beta1: float = 0.9,
          beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
          exp_avg_scales=None, exp_avg_sq_scales=None, stream=None):
    """One AdamW step, number ``step`` (from 1), in place, over lists of
    contiguous CUDA tensors: params and grads float32, float16 or bfloat16 (one
    type each), moments float32, or 8-bit codes (exp_avg int8, exp_avg_sq uint8)
    with float32 scales, one for each ADAMW_BLOCK elements of a tensor.  Zero
    codes and scales are the initial state."""
    if stream is not None:
        params = list(params)
    return _run(load_head().adamw, stream, params[0] if stream is not None and params else None,
                params, grads, exp_avg, exp_avg_sq, exp_avg_scales, exp_avg_sq_scales, step, lr,
                beta1, beta2, eps, weight_decay)


def adamw_moments(exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, stream=None):
    """The float32 values (m, v) that 8-bit moments stand for: one tensor's
    codes and scales, or storage of several laid out on blocks of ADAMW_BLOCK."""
    return _run(load_head().adamw_moments, stream, exp_avg, exp_avg, exp_avg_scale, exp_avg_sq,
                exp_avg_sq_scale)
