"""The linear layer at the ends of its range, and over more tiles than run at once."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from test_gpu_head import DT, clean_status, close, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_slopes_of_large_and_infinite_pre_activations(act, dt):
    """A slope's limits are 1 and 0: for the largest pre, and where it was rounded to infinity.  An FP32
    sigmoid or normal distribution there is off by a unit in the last place at most, 2^-23; D is
    rounded to the type, which holds dy itself."""
    t = DT[dt]
    ends = [1e4, 6e4, float("inf")] + ([1e15, 3e19, 1e20, 1e30, 3e38] if dt == "bf16" else [7e4])
    v = torch.tensor(ends + [-e for e in ends]).to(t).cuda()
    n, m, k = len(v), 5, 16
    g = gen(3)
    pre = v[None].repeat(m, 1)
    x, w, dy = randn(g, m, k).to(t), torch.eye(n, k, device="cuda").to(t), randn(g, m, n).to(t)
    dx, dw, db = os2.linear_backward(x, w, dy, pre=pre, activation=act, need_db=True, db_dtype=torch.float32)
    d = torch.where(v > 0, dy.double(), 0.0)
    close(dx[:, :n], d, 2.0 ** -22 * d.abs())             # W picks D's columns
    assert (dx[:, n:] == 0).all()
    close(db, d.sum(0), m * 2.0 ** -23 * d.abs().sum(0))
    size = d.abs().t() @ x.double().abs()
    close(dw, d.t() @ x.double(), (2.0 ** -21 + torch.finfo(t).eps / 2) * size)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_slope_of_nan_is_nan(act):
    """And does not reach another token's dx or another output's dW."""
    g = gen(4)
    m, n, k = 6, 24, 16
    x, w, dy = randn(g, m, k).bfloat16(), randn(g, n, k).bfloat16(), randn(g, m, n).bfloat16()
    pre = randn(g, m, n).bfloat16()
    want = os2.linear_backward(x, w, dy, pre=pre, activation=act, need_db=True)
    pre[2, 7] = float("nan")
    got = os2.linear_backward(x, w, dy, pre=pre, activation=act, need_db=True)
    for a, b, at in zip(got, want, (2, 7, 7)):
        others = torch.arange(len(a), device="cuda") != at
        assert a[at].isnan().all() and torch.equal(a[others], b[others])
