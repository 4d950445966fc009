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
