"""Operators of a language model's vocabulary head and of what stands around it
(include/os2.h).

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
  rmsnorm, rmsnorm_quantize,        root-mean-square norm with the residual's
  rmsnorm_backward, RMSNormFunction addition, its gradient, and in 8 bits as
                                    i8gemm takes its tokens
  linear, linear_backward,          a linear layer with bias, activation and residual,
  linear_ways, LinearFunction       and its gradient
  sample                            a token from each row of logits by temperature,
                                    top-k, top-p and min-p
"""
from __future__ import annotations

import ctypes as ct

import torch

from .binding import _check, load, load_head

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
    The gradient has no gradient of its own: to go back through it raises, and so do
    forward mode and vmap."""

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


# --------------------------------------------------------------------- norm
def rmsnorm(X: torch.Tensor, weight: torch.Tensor, residual=None, eps: float = 1e-6, out=None,
            out_h=None, stream=None):
    """The root-mean-square norm of X's rows (n x d, float32, float16 or bfloat16),
    Y = H * rsqrt(mean(H^2) + eps) * weight, where H is X, or X + residual rounded to
    their type: the residual stream.  Returns Y, or (Y, H) with a residual.  weight: d
    values of float32 or of X's type.  out may be X, out_h X or the residual (not all of them
    X); an output that overlaps an input in another way is refused."""
    return _run(load_head().rmsnorm, stream, X, X, weight, residual, eps, out, out_h, None, False)


def rmsnorm_quantize(X: torch.Tensor, weight: torch.Tensor, residual=None, eps: float = 1e-6,
                     out=None, scale=None, out_h=None, stream=None):
    """``rmsnorm`` in 8-bit integers with one scale a row, Y ~ q * scale[:, None], as
    ``i8gemm`` takes them: (q int8, scale float32), or (q, scale, H) with a residual."""
    return _run(load_head().rmsnorm, stream, X, X, weight, residual, eps, out, out_h, scale, True)


def rmsnorm_backward(H: torch.Tensor, weight: torch.Tensor, dY: torch.Tensor, dh=None,
                     eps: float = 1e-6, need_dx: bool = True, need_dw: bool = True, workspace=None,
                     stream=None):
    """The gradient of ``rmsnorm``: (dX, dW) for dY, H as returned (X without a residual)
    and dh, what comes back along the residual stream.  dX, the gradient of X and of the
    residual alike, is of H's type, dW of the weight's; None for the one not needed."""
    return _run(load_head().rmsnorm_backward, stream, H, H, weight, dY, dh, eps, need_dx, need_dw,
                workspace)


def _in_rows(x):
    """x, as rows that a call takes (a gradient may be an expanded scalar)."""
    return x if x is None or x.is_contiguous() else x.contiguous()


class RMSNormFunction(torch.autograd.Function):
    """``rmsnorm`` for autograd: RMSNormFunction.apply(X, weight, residual, eps) gives Y, or
    (Y, H) with a residual.  The gradient has no gradient of its own, and there is no
    forward mode and no vmap: they raise.  (As with any function
    of autograd: a backward pass is captured into a graph only while no graph of the same
    leaves lives that was recorded outside of the capture; what autograd keeps of a leaf
    belongs to the stream that it was made on.)"""

    @staticmethod
    def forward(ctx, X, weight, residual=None, eps=1e-6):
        ctx.set_materialize_grads(False)
        ctx.eps = eps
        if residual is None:
            ctx.save_for_backward(X, weight)
            return rmsnorm(X, weight, eps=eps)
        Y, H = rmsnorm(X, weight, residual, eps)
        ctx.save_for_backward(H, weight)
        return Y, H

    @staticmethod
    def backward(ctx, dY, dH=None):
        H, weight = ctx.saved_tensors
        need_x, need_w, need_r = (*ctx.needs_input_grad, False)[:3]  # (the residual may be left out)
        if dY is None:  # Y was not used: the stream's gradient passes
            dx, dw = dH, None
        else:
            dx, dw = _once(rmsnorm_backward, H, weight, _in_rows(dY), _in_rows(dH), ctx.eps,
                           need_x or need_r, need_w)
        return dx if need_x else None, dw, dx if need_r else None, None


def _once(gradient, *args):
    """A gradient's call; where a graph of it is asked for, one that raises when it is
    differentiated, instead of a constant."""
    # (with create_graph only is a gradient taken while autograd records)
    return _Once.apply(gradient, *args) if torch.is_grad_enabled() else gradient(*args)


class _Once(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gradient, *args):
        return gradient(*args)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("this gradient has no gradient of its own")


# ------------------------------------------------------------- linear layer
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}") from None


def linear(X: torch.Tensor, W: torch.Tensor, bias=None, residual=None, activation: str = "none",
           return_pre: bool = False, out=None, workspace=None, stream=None):
    """Y = residual + act(X @ W.T + bias), in one product's epilogue.

    X: m x k, W: n x k, residual: m x n, all bfloat16 or all float16; bias: n values of
    float32 or of X's type; activation: none, relu, gelu, gelu_tanh or silu.  With
    return_pre, (Y, pre): pre = X @ W.T + bias in X's type, what ``linear_backward`` goes by.
    out may be the residual, and overlaps no other input.  Widths that are multiples of 8 (rows on 16-byte boundaries) save
    a copy of X and W in each call."""
    return _run(load_head().linear, stream, X, X, W, bias, residual, _activation(activation),
                bool(return_pre), out, workspace)


def linear_backward(X: torch.Tensor, W: torch.Tensor, dY: torch.Tensor, pre=None,
                    activation: str = "none", need_dx: bool = True, need_dw: bool = True,
                    need_db: bool = False, db_dtype=None, workspace=None, stream=None):
    """The gradient of ``linear``: (dX, dW, db) for dY, which is the residual's gradient
    too; None for the one not needed.  pre: as ``linear`` returned it (not read without an
    activation).  db_dtype: float32 or X's type (the default)."""
    return _run(load_head().linear_backward, stream, X, X, W, dY, pre, _activation(activation),
                need_dx, need_dw, need_db, db_dtype, workspace)


def linear_ways(m: int, n: int, k: int, activation: str = "none", pre: bool = False, residual: bool = False,
                aligned: bool = True) -> dict:
    """Which kernels ``linear`` and ``linear_backward`` go through on the current device, by sizes
    alone (os2_linear_ways): way and dx_way are 0 for tiles of few tokens, 1 for tiles of 256 x 256, 2 for
    those with the terms cut into parts.  Nothing is launched."""
    names = ("way", "tokens", "cluster", "parts", "dx_way", "dx_tokens", "dx_cluster", "dx_parts", "dw_parts")
    out = (ct.c_int * len(names))()
    _check(load().os2_linear_ways(m, n, k, _activation(activation), bool(pre), bool(residual), bool(aligned), out),
           "os2_linear_ways")
    return dict(zip(names, out))


class LinearFunction(torch.autograd.Function):
    """``linear`` for autograd: LinearFunction.apply(X, W, bias, residual, activation).
    No gradient of the gradient, forward mode or vmap, and captured, as ``RMSNormFunction`` is."""

    @staticmethod
    def forward(ctx, X, W, bias=None, residual=None, activation="none"):
        ctx.activation, ctx.bias_dtype = activation, None if bias is None else bias.dtype
        pre = None
        if activation != "none" and any(ctx.needs_input_grad[:3]):
            Y, pre = linear(X, W, bias, residual, activation, return_pre=True)
        else:
            Y = linear(X, W, bias, residual, activation)
        ctx.save_for_backward(X, W, pre)
        return Y

    @staticmethod
    def backward(ctx, dY):
        X, W, pre = ctx.saved_tensors
        need_x, need_w, need_b, need_r = (*ctx.needs_input_grad, False, False)[:4]
        dx = dw = db = None
        if need_x or need_w or need_b:
            dx, dw, db = _once(linear_backward, X, W, _in_rows(dY), pre, ctx.activation, need_x,
                               need_w, need_b, ctx.bias_dtype)
        return dx, dw, db, dY if need_r else None, None


# ------------------------------------------------------------------- a token
def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           stream=None):
    """A token from each row of logits (n x v, float32, float16 or bfloat16) by the given
    random numbers u (n float32 values in [0, 1)): (token int64, logprob float32).

    The order is by falling logit, the lower index first.  Kept are the first top_k of it
    (0: all), of those the ones before which less than top_p of their mass lies, and of those the
    ones with at least min_p of the largest probability; the token is, by index, the first
    at which the mass kept so far exceeds u times the mass kept, logprob its logarithm of
    the mass kept.  temperature 0 takes the first of the order.  Each setting is a number or
    a tensor of n values (float32; top_k int32).  Sums are exact: the same inputs give the
    same token in any batch.  A row without a finite largest logit gives token -1; settings out of
    range in a tensor do too and are reported by ``get_status`` (ERR_RANGE)."""
    return _run(load_head().sample, stream, logits, logits, u, temperature, top_k, top_p, min_p)
