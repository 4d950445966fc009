"""The cross entropy's gradient where a pair of SMs works through many tiles of
dW.  Definitions, bounds and inputs as in test_gpu_head."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from test_gpu_head import DT, clean_status, close, xent_case, xent_want  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 8, 64, 300])
@pytest.mark.parametrize("k", [80, 96, 160, 224, 352, 480])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_dw_of_many_tiles(n, k, dt):
    """Widths whose last 128 columns are one or three blocks of 32, and so many
    columns of the vocabulary that every pair of SMs has several tiles: each row of dW
    is its own, and the same every time."""
    h, w, y, grad = xent_case(n, k, 60000, DT[dt], 0.0, n + k)
    loss, lse = os2.xent(h, w, y)
    dh, dw = os2.xent_backward(h, w, y, lse, grad)
    want, tol = xent_want(h, w, y, grad)
    for got, x, t in zip((loss, lse, dh, dw), want, tol):
        close(got, x, t)
    for _ in range(10):
        again = os2.xent_backward(h, w, y, lse, grad)
        assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_a_gradient_that_is_not_finite_stays_in_its_row(bad, dt):
    """One row's g is not finite, the others' are large: their rows of dH are what they
    are with a zero in its place."""
    h, w, y, grad = xent_case(60, 64, 900, DT[dt], 0.0, 21)
    grad = grad.sign() * 1000.0 * (1 + torch.arange(60, device="cuda"))
    grad[7] = 0
    loss, lse = os2.xent(h, w, y)
    want = os2.xent_backward(h, w, y, lse, grad)[0]
    assert torch.isfinite(want).all()
    grad[7] = bad
    dh, dw = os2.xent_backward(h, w, y, lse, grad)
    rest = torch.arange(60, device="cuda") != 7
    assert torch.equal(dh[rest], want[rest])
    assert not torch.isfinite(dh[7]).any() and not torch.isfinite(dw).any()


def spread_rows(n, k, v, dt, seed, least, most):
    """Rows whose g are powers of two times a number, from 2^least to 2^most; the rows of W have
    a part in common, so that a row of dH needs its whole softmax, not the label alone."""
    h, w, y, _ = xent_case(n, k, v, dt, 0.1, seed)
    w = (w.float() + 0.5 * w[0].float().sign()).to(dt)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    grad = 2.0 ** torch.linspace(least, most, n, device="cuda")[torch.randperm(n, generator=g, device="cuda")]
    grad *= torch.where(torch.rand(n, generator=g, device="cuda") < 0.3, -1.0, 1.0)
    grad[n // 2] = 0
    return h, w, y, grad


def row_bound(h, w, y, grad, dh):
    """The bound of dH's error, each row's by its own g (xent_want's, but for what D loses
    below its smallest numbers: 2^-24 a unit, held times 2^14, of the row's |g| or of one 2^6
    as large)."""
    h64, w64 = h.double(), w.double()
    k, v = h.shape[1], w.shape[0]
    valid = y != -100
    z = h64 @ w64.t()
    dz = (k / 16 + 1) * 2.0 ** -22 * (h64.abs() @ w64.abs().t()).amax(1)
    lse = torch.logsumexp(z, 1)
    g = torch.where(valid, grad.double().abs(), 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    d = p.clone()
    d.scatter_add_(1, torch.where(valid, y, 0)[:, None], torch.full_like(d[:, :1], -1.0))
    d = d.abs() * g
    ed = d * 2.0 ** -11 + p * g * (3 * dz + 2.0 ** -19 * (2 + lse.abs() + z.abs().amax(1)))[:, None] + g * 2.0 ** -33
    return ed @ w64.abs() + (v / 16 + 1) * 2.0 ** -22 * (d @ w64.abs()) + 2.0 ** -11 * dh.abs() * 1.01 + 2.0 ** -24


# dH out of one product, out of parts of one, and out of several pieces of the vocabulary
@pytest.mark.parametrize("n,k,v", [(2048, 2048, 4096), (100, 128, 50021), (333, 100, 3001), (66000, 64, 4100)])
@pytest.mark.parametrize("least,most", [(-14, 10), (-24, 0), (-5, 0)])
def test_dh_of_rows_far_apart_in_f16(n, k, v, least, most):
    """A row of dH is as near its own size as if it were alone, however large the
    others' g: 2^-24 of the largest here, where FP16 holds it well."""
    h, w, y, grad = spread_rows(n, k, v, torch.float16, n, least, most)
    loss, lse = os2.xent(h, w, y)
    dh, dw = os2.xent_backward(h, w, y, lse, grad)
    parts = torch.arange(n, device="cuda").split(16500)
    for r in parts:
        (_, _, want, want_w), (_, _, _, tol_w) = xent_want(h[r], w, y[r], grad[r])
        close(dh[r], want, row_bound(h[r], w, y[r], grad[r], want))
    if len(parts) == 1:
        close(dw, want_w, tol_w)
    only, none = os2.xent_backward(h, w, y, lse, grad, need_dw=False)
    none2, only_w = os2.xent_backward(h, w, y, lse, grad, need_dh=False)
    assert none is None and none2 is None and torch.equal(only, dh) and torch.equal(only_w, dw)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("k", [64, 1100])
def test_logits_that_are_infinite(n, k):
    """A logit of -Inf is a term of 0; one of +Inf makes its row's values NaN, and no other's."""
    h, w, y, _ = xent_case(n, k, 700, torch.bfloat16, 0.0, 41)
    h[:, 5] = 1.0
    y = y.clamp(min=10)
    w2 = w.clone()
    w2[7, 5] = -float("inf")
    loss, lse = os2.xent(h, w2, y)
    (want, want_lse, _, _), (tl, ts, _, _) = xent_want(h, torch.cat([w[:7], w[8:]]), y - 1, torch.ones(n, device="cuda"))
    close(loss, want, tl)
    close(lse, want_lse, ts)
    h[1, 5] = -1.0                                # a logit of +Inf for this row alone
    base = os2.xent(h, w2, y)
    for got, before in zip(base, (loss, lse)):
        rest = torch.arange(n, device="cuda") != 1
        assert torch.isnan(got[1]) and torch.equal(got[rest], before[rest])
