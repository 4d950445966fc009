"""The linear layer at the ends of its range, and over more tiles than run at once."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from test_gpu_head import DT, clean_status, close, gen, randn  # noqa: F401
from test_gpu_linear import SHAPES, case, check, close_product, grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_slopes_of_large_and_infinite_pre_activations(act, dt):
    """A slope's limits are 1 and 0: for the largest pre, and where it was rounded to infinity.  An FP32
    sigmoid or normal distribution there is off by a unit in the last place at most, 2^-23.  D is
    rounded to the type: BF16 holds dy itself, and so does FP16 for relu; elsewhere FP16 holds 7/8 of it
    to 2^-11, and 8/7 of that is rounded to 2^-11 again."""
    t = DT[dt]
    ends = [1e4, 6e4, float("inf")] + ([1e15, 3e19, 1e20, 1e30, 3e38] if dt == "bf16" else [7e4])
    v = torch.tensor(ends + [-e for e in ends]).to(t).cuda()
    n, m, k = len(v), 5, 16
    g = gen(3)
    pre = v[None].repeat(m, 1)
    x, w, dy = randn(g, m, k).to(t), torch.eye(n, k, device="cuda").to(t), randn(g, m, n).to(t)
    dx, dw, db = os2.linear_backward(x, w, dy, pre=pre, activation=act, need_db=True, db_dtype=torch.float32)
    d = torch.where(v > 0, dy.double(), 0.0)
    held = 0.0 if dt == "bf16" or act == "relu" else 2.0 ** -11
    close(dx[:, :n], d, (2.0 ** -22 + 2.01 * held) * d.abs() + (2.0 ** -23 if held else 0.0))  # W picks D's columns
    assert (dx[:, n:] == 0).all()
    close(db, d.sum(0), m * 2.0 ** -23 * d.abs().sum(0))
    size = d.abs().t() @ x.double().abs()
    close(dw, d.t() @ x.double(), (2.0 ** -21 + torch.finfo(t).eps / 2 + 1.01 * held) * size + (2.0 ** -23 if held else 0.0))


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


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 64), (5, 200, 72), (40, 129, 333), (300, 200, 136), (700, 2047, 264), (2100, 72, 64), (40, 12000, 64)])
def test_gradients_of_the_largest_fp16_numbers(act, m, n, k):
    """Where dy is FP16's largest and the slope is above 1, D is beyond FP16, and its products need not be."""
    g = gen(m + n + k)
    x, w = (randn(g, m, k) * 0.002).half(), (randn(g, n, k) * 0.002).half()
    dy = torch.where(randn(g, m, n) < 0, -65504.0, 65504.0).half()
    pre = torch.where(randn(g, m, n) < 0, 1.4, 2.4).half()
    dx, dw, db = os2.linear_backward(x, w, dy, pre=pre, activation=act, need_db=True, db_dtype=torch.float32)
    d, dd = grads(x, w, dy, pre, act)
    assert act in ("none", "relu") or d.abs().max() > 71000
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    close_product(dx, d, dd, w.double(), torch.float16)
    close_product(dw, d.t(), dd.t() if torch.is_tensor(dd) else dd, x.double(), torch.float16)
    size = d.abs().sum(0)
    close(db, d.sum(0), ((m // 4 + 72) * 2.0 ** -24 + 8e-6) * size)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradients_of_the_smallest_fp16_numbers(act):
    """D among FP16's subnormal numbers is off by at most half a step of them, 8/7 of it as it is held."""
    g = gen(7)
    m, n, k = 33, 48, 40
    x, w = randn(g, m, k).half(), randn(g, n, k).half()
    dy, pre = (randn(g, m, n) * 2.0 ** -19).half(), randn(g, m, n).half()
    dx, dw, _ = os2.linear_backward(x, w, dy, pre=pre, activation=act)
    d, dd = grads(x, w, dy, pre, act)                    # (a whole step of slack, TINY, is in dd)
    close_product(dx, d, dd, w.double(), torch.float16)
    close_product(dw, d.t(), dd.t(), x.double(), torch.float16)


# More tiles of 256 x 256 than an SM pair each: accumulators and store buffers go from tile to tile.
# Columns on 16-byte boundaries leave by TMA, the others by rows.
MANY_TILES = [(2600, 4104, 264), (2600, 4101, 264), (4200, 2568, 520), (4200, 2571, 520)]


@pytest.mark.parametrize("m,n,k", MANY_TILES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act,bias,residual,pre", [("none", None, False, False), ("silu", "f32", True, False), ("gelu", "same", True, True),
                                                   ("relu", None, False, True)])
def test_forward_over_many_tiles(m, n, k, dt, act, bias, residual, pre):
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    ways = os2.linear_ways(m, n, k, act, pre, residual, n % 8 == 0)
    assert ways["way"] == 1 and -(-m // 256) * -(-n // 256) > 2 * pairs
    _, x, w, b, r = case(m, n, k, dt)
    b = None if bias is None else b.to(DT[dt]) if bias == "same" else b
    got = os2.linear(x, w, bias=b, residual=r if residual else None, activation=act, return_pre=pre)
    y, z = got if pre else (got, None)
    check(x, w, b, r if residual else None, act, y, z)


@pytest.mark.parametrize("m,n,k", [(5000, 264, 4104), (5000, 267, 4101), (600, 4104, 4104), (600, 4104, 4101)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_gradient_over_many_tiles(m, n, k, dt, act):
    """dX (5000 x 4104) or dW (4104 x 4104) of more tiles than SM pairs, of three to five stages each."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    ways = os2.linear_ways(m, n, k, act)
    rows, parts = (m, ways["dx_parts"]) if m > n else (n, ways["dw_parts"])
    assert parts == 1 and -(-rows // 256) * -(-k // 256) > 2 * pairs and (m < n or ways["dx_way"] == 1)
    g, x, w, _, _ = case(m, n, k, dt)
    dy, pre = randn(g, m, n).to(DT[dt]), (randn(g, m, n) * 1.5).to(DT[dt])
    dx, dw, _ = os2.linear_backward(x, w, dy, pre=pre, activation=act)
    d, dd = grads(x, w, dy, pre, act)
    close_product(dx, d, dd, w.double(), DT[dt])
    close_product(dw, d.t(), dd.t() if torch.is_tensor(dd) else dd, x.double(), DT[dt])


# dX with its terms cut into 24, 6, 5, 3 and 2 parts, by clusters of two, and dW's into eight
GRADIENT_PARTS = [(40, 12000, 64), (400, 8200, 1003), (800, 8200, 520), (600, 4100, 2000), (600, 5000, 2571), (800, 1000, 520), (2048, 8, 64)]


@pytest.mark.parametrize("m,n,k", GRADIENT_PARTS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradient_in_parts(m, n, k, dt, act):
    g, x, w, _, _ = case(m, n, k, dt)
    dy, pre = randn(g, m, n).to(DT[dt]), (randn(g, m, n) * 1.5).to(DT[dt])
    dx, dw, db = os2.linear_backward(x, w, dy, pre=pre, activation=act, need_db=True, db_dtype=torch.float32)
    d, dd = grads(x, w, dy, pre, act)
    close_product(dx, d, dd, w.double(), DT[dt])
    close_product(dw, d.t(), dd.t() if torch.is_tensor(dd) else dd, x.double(), DT[dt])
    off = 2e-6 * (dy.double().abs() * (1 + pre.double().abs())).sum(0)
    close(db, d.sum(0), (m // 4 + 72) * 2.0 ** -24 * (d.abs().sum(0) + off) + off)
    assert torch.equal(os2.linear_backward(x, w, dy, pre=pre, activation=act, need_dw=False)[0], dx)
    assert torch.equal(os2.linear_backward(x, w, dy, pre=pre, activation=act, need_dx=False)[1], dw)


def test_the_tested_shapes_go_every_way():
    """The shapes compared with 64 bits here and beside reach every kernel of the linear layer, each
    cluster size and both ways to store."""
    seen = set()
    for m, n, k in SHAPES + MANY_TILES + GRADIENT_PARTS + [(600, 2000, 5000), (600, 2003, 5001)]:
        y = os2.linear_ways(m, n, k, aligned=n % 8 == 0)
        seen.add(("way", y["way"], n % 8 == 0 if y["way"] == 1 else None))
        seen.add(("dx", y["dx_way"], k % 8 == 0 if y["dx_way"] == 1 else None))
        seen.add(("dw", min(y["dw_parts"], 2), k % 8 == 0 if y["dw_parts"] == 1 else None))
        if y["way"] == 0:
            seen |= {("cluster", y["cluster"]), ("tokens", y["tokens"])}
        if y["dx_way"] == 0:
            seen.add(("dx_cluster", y["dx_cluster"]))
    wanted = {("way", 0, None), ("way", 1, True), ("way", 1, False), ("way", 2, None), ("dx", 0, None), ("dx", 1, True), ("dx", 1, False),
              ("dx", 2, None), ("dw", 1, True), ("dw", 1, False), ("dw", 2, None), ("tokens", 16), ("tokens", 128)}
    wanted |= {(name, c) for name in ("cluster", "dx_cluster") for c in (1, 2, 4, 8)}
    assert wanted <= seen, sorted(wanted - seen, key=str)


def test_no_vmap_and_no_forward_mode():
    """They raise, as the second gradient does, and leave no wrong tangent behind."""
    import torch.autograd.forward_ad as fwad
    x, w, g = torch.ones(4, 8, device="cuda").half(), torch.ones(16, 8, device="cuda").half(), torch.ones(8, device="cuda")
    for f in (lambda x: os2.LinearFunction.apply(x, w), lambda x: os2.RMSNormFunction.apply(x, g),
              lambda x: os2.XentFunction.apply(x, w, torch.zeros(4, dtype=torch.long, device="cuda"))):
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.func.vmap(f)(x[None].repeat(2, 1, 1))
        with pytest.raises((RuntimeError, NotImplementedError)):
            with fwad.dual_level():
                f(fwad.make_dual(x, torch.ones_like(x)))
