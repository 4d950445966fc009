"""The vocabulary-head operators against their definitions in 64 bits.

Tolerances follow from the arithmetic.  U[t] is the unit roundoff of type t.  A
tensor-core sum of k products adds k / 16 groups to an FP32 accumulator, each
with a relative error of at most 2^-22 of what has been summed in magnitude:
dz = (k / 16 + 1) 2^-22 sum |a b|.  Exponentials, logarithms and their
arguments in FP32 add 2^-20 (1 + |argument|)."""
import math

import numpy as np
import pytest
import torch

import rns_emulated_fp64_gb300 as os2

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def close(got, want, tol):
    got = got.double()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= tol) & ~(torch.isnan(got) & torch.isnan(want)) & ~(got == want)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.fixture(autouse=True)
def clean_status():
    yield
    assert os2.get_status() == 0


# ------------------------------------------------------------------- 8 bits
def quantized(x):
    """The definition in FP32, operation by operation."""
    x = x.float().cpu().numpy()
    with np.errstate(all="ignore"):
        s = np.abs(x).max(1) / np.float32(127) if x.shape[1] else np.zeros(len(x), np.float32)
        q = np.where(s[:, None] > 0, np.clip(np.rint(x / np.where(s > 0, s, 1)[:, None]), -127, 127), 0)
        ok = np.isfinite(x).all(1)
    return np.where(ok[:, None], np.nan_to_num(q), 0).astype(np.int8), np.where(ok, s, np.nan).astype(np.float32)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (5, 64), (2, 4096), (33, 1777), (1, 8200)])
def test_quantize_rows(dt, m, k):
    x = (randn(gen(m * k), m, k) * torch.exp(3 * randn(gen(1), m, 1))).to(DT[dt])
    q, s = os2.quantize_rows(x)
    qr, sr = quantized(x)
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)


def test_quantize_rows_edges():
    x = randn(gen(7), 9, 50)
    x[0] = 0
    x[1, 3] = math.inf
    x[2, 4] = math.nan
    x[3] *= 1e-44 / x[3].abs().max()           # subnormal: the scale has few bits, or is 0
    x[4] *= 3e38 / x[4].abs().max()
    x[5] = 127 * torch.sign(x[5])              # every entry at the end of the range
    x[6] = 0
    x[6, 49] = -5.0
    x[7] = torch.arange(50, device="cuda") + 0.5   # ties
    x[7, 0] = 127.0
    q, s = os2.quantize_rows(x)
    qr, sr = quantized(x)
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr, equal_nan=True)
    wide = torch.zeros(9, 64, device="cuda")
    wide[:, 3:53] = x                          # a view off the alignment
    out = torch.full((9, 61), 99, dtype=torch.int8, device="cuda")
    q2, _ = os2.quantize_rows(wide[:, 3:53], out=out[:, 5:55])
    assert torch.equal(q2, q) and (out[:, :5] == 99).all() and (out[:, 55:] == 99).all()


def i8_want(q, sa, w, sb, bias):
    s = q.double() @ w.double().t()
    y = s * sa.double()[:, None] * sb.double()
    return (y if bias is None else y + bias.double()), s


def i8_tol(want, bias, dt):
    # the sum to FP32, two scales, the bias: four roundings; then the output's
    b = 0 if bias is None else bias.double().abs()
    return (want.abs() + 2 * b) * (4 * U[torch.float32] * (1 + U[dt]) + (U[dt] if dt != torch.float32 else 0)) + TINY[dt]


I8_SHAPES = [(1, 1, 1), (1, 33, 64), (1, 4096, 4096), (2, 50, 100), (3, 129, 1777), (4, 257, 512), (5, 64, 2000),
             (8, 1000, 640), (9, 130, 128), (16, 300, 1024), (17, 255, 96), (31, 4000, 130), (33, 128, 1025),
             (64, 500, 2048), (77, 513, 999), (128, 256, 1152), (129, 384, 4096), (205, 1003, 1777), (300, 77, 3000),
             (513, 1200, 896), (1030, 2050, 1300)]


@pytest.mark.parametrize("m,n,k", I8_SHAPES)
@pytest.mark.parametrize("out,bias", [("f32", True), ("bf16", False), ("f16", True)])
def test_i8gemm(m, n, k, out, bias):
    g = gen(m + n + k)
    q = torch.randint(-128, 128, (m, k), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda").to(torch.int8)
    sa, sb = torch.rand(m, generator=g, device="cuda") * 1e-3, torch.rand(n, generator=g, device="cuda") * 1e-2
    b = randn(g, n) if bias else None
    y = os2.i8gemm(q, sa, w, sb, bias=b, out_dtype=DT[out])
    want, _ = i8_want(q, sa, w, sb, b)
    close(y, want, i8_tol(want, b, DT[out]))


@pytest.mark.parametrize("m", [1, 7, 40, 300])
@pytest.mark.parametrize("k", [1024, 1025, 4096, 20000])
def test_i8gemm_sums_are_exact(m, k):
    """All products at the end of the range: sums far above 2^24, with unit
    scales and integers that FP32 holds, have to come out exactly."""
    n = 260
    for a, b in ((-128, -128), (127, -128), (127, 127)):
        q = torch.full((m, k), a, dtype=torch.int8, device="cuda")
        w = torch.full((n, k), b, dtype=torch.int8, device="cuda")
        w[3] = 0
        w[4, : k // 2] *= -1 if b != -128 else 0
        one = torch.ones(max(m, n), device="cuda")
        y = os2.i8gemm(q, one[:m], w, one[:n], out_dtype=torch.float32)
        want = (q.double() @ w.double().t()).float()
        assert torch.equal(y, want)
    # odd sums that differ in their last bit from row to row
    g = gen(k)
    q = torch.randint(100, 128, (m, k), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(100, 128, (n, k), generator=g, device="cuda").to(torch.int8)
    y = os2.i8gemm(q, one[:m], w, one[:n], out_dtype=torch.float32)
    assert torch.equal(y, (q.double() @ w.double().t()).float())


@pytest.mark.parametrize("m", [1, 3, 8, 30, 200])
@pytest.mark.parametrize("off,pad", [(0, 16), (1, 15), (5, 27), (8, 8), (0, 1)])
def test_i8gemm_strides(m, off, pad):
    """Rows that start anywhere: views into wider matrices, outputs too."""
    n, k = 150, 333
    g = gen(m + off)
    Q = torch.randint(-128, 128, (m, off + k + pad), generator=g, device="cuda").to(torch.int8)
    Wf = torch.randint(-128, 128, (n, off + k + pad), generator=g, device="cuda").to(torch.int8)
    q, w = Q[:, off:off + k], Wf[:, off:off + k]
    sa, sb = torch.rand(m, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        big = torch.full((m, n + 11), 7.0, dtype=dt, device="cuda")
        y = os2.i8gemm(q, sa, w, sb, out=big[:, 3:3 + n])
        want, _ = i8_want(q, sa, w, sb, None)
        close(y, want, i8_tol(want, None, dt))
        assert (big[:, :3] == 7).all() and (big[:, 3 + n:] == 7).all()


@pytest.mark.parametrize("m", [1, 6, 20, 140])
def test_i8linear_matches_its_parts(m):
    g = gen(m)
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        x = (randn(g, m, 700) * torch.exp(randn(g, m, 1))).to(dt)
        if m > 2:
            x[1] = 0
            x[2, 5] = math.nan
        w, sb = os2.quantize_rows(randn(g, 333, 700))
        b = randn(g, 333)
        q, sa = os2.quantize_rows(x)
        for od in (torch.float32, dt):
            y, z = os2.i8linear(x, w, sb, bias=b, out_dtype=od), os2.i8gemm(q, sa, w, sb, bias=b, out_dtype=od)
            assert torch.equal(torch.isnan(y), torch.isnan(z)) and torch.equal(y.nan_to_num(), z.nan_to_num())
        if m > 2:
            assert torch.isnan(y[2]).all() and not torch.isnan(y[[0, 1] + list(range(3, m))]).any()
            close(y[1], b.double().to(dt).double(), 0)


def test_i8_empty():
    dev = "cuda"
    z = lambda *s, dt=torch.int8: torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
    f = torch.float32
    assert os2.i8gemm(z(0, 8), z(0, dt=f), z(5, 8), z(5, dt=f)).shape == (0, 5)
    assert os2.i8gemm(z(3, 8), z(3, dt=f), z(0, 8), z(0, dt=f)).shape == (3, 0)
    bias = torch.arange(5, device=dev, dtype=f)
    for m in (3, 40):
        y = os2.i8gemm(z(m, 0), z(m, dt=f) + 1, z(5, 0), z(5, dt=f) + 1, bias=bias, out_dtype=f)
        assert torch.equal(y, bias.expand(m, 5))
    assert os2.quantize_rows(z(0, 8, dt=f))[0].shape == (0, 8)
    q, s = os2.quantize_rows(z(4, 0, dt=f))
    assert q.shape == (4, 0) and (s == 0).all()


def test_i8_refuses_what_does_not_match():
    q, w = torch.zeros(3, 8, dtype=torch.int8, device="cuda"), torch.zeros(5, 8, dtype=torch.int8, device="cuda")
    s3, s5 = torch.ones(3, device="cuda"), torch.ones(5, device="cuda")
    for f in (lambda: os2.i8gemm(q, s5, w, s5), lambda: os2.i8gemm(q, s3, w, s3), lambda: os2.i8gemm(q, s3, w[:, :7], s5),
              lambda: os2.i8gemm(q, s3, w.t(), s5), lambda: os2.i8gemm(q, s3, w, s5, bias=s3),
              lambda: os2.i8gemm(q, s3, w, s5, out_dtype=torch.float64), lambda: os2.i8gemm(q, s3.double(), w, s5),
              lambda: os2.i8gemm(q, s3, w, s5, out=torch.empty(3, 4, device="cuda")),
              lambda: os2.i8gemm(q, s3, w, s5, out=torch.empty(1, 5, device="cuda").expand(3, 5)),
              lambda: os2.i8linear(q, w, s5)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(os2.Os2Error):
        os2.i8gemm(q, s3, w, s5, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------ cross entropy
def xent_want(h, w, y, g, ignore=-100):
    """loss, lse, dh, dw and the bounds of their errors, in 64 bits."""
    h64, w64 = h.double(), w.double()
    (n, k), v = h.shape, w.shape[0]
    valid = (y != ignore)
    h64 = torch.where(valid[:, None], h64, 0.0)
    z = h64 @ w64.t()
    dz = (k / 16 + 1) * 2.0 ** -22 * (h64.abs() @ w64.abs().t()).amax(1)
    lse = torch.logsumexp(z, 1)
    at = torch.where(valid, y, 0)[:, None]
    zy = z.gather(1, at)[:, 0]
    tl = 2 * dz + 2.0 ** -20 * (1 + lse.abs() + zy.abs())
    loss = torch.where(valid, lse - zy, 0.0)
    p = torch.exp(z - lse[:, None])
    g64 = torch.where(valid, g.double(), 0.0)[:, None]
    d = p.clone()
    d.scatter_add_(1, at, torch.full_like(d[:, :1], -1.0))
    d = d * g64
    u = U[h.dtype]
    # an entry of D: rounded to the type; its exponential is off by dz and FP32's own error
    ed = d.abs() * u + p * g64.abs() * (3 * dz + 2.0 ** -19 * (2 + lse.abs() + z.abs().amax(1)))[:, None]
    if h.dtype == torch.float16 and n:
        ed += g64.abs().max() * 2.0 ** -38
    dh, dw = d @ w64, d.t() @ h64
    th = ed @ w64.abs() + (v / 16 + 1) * 2.0 ** -22 * (d.abs() @ w64.abs()) + u * dh.abs() * 1.01 + TINY[h.dtype]
    tw = ed.t() @ h64.abs() + (n / 16 + 1) * 2.0 ** -22 * (d.t().abs() @ h64.abs()) + u * dw.abs() * 1.01 + TINY[h.dtype]
    return (loss, torch.where(valid, lse, 0.0), dh, dw), (tl, tl, th, tw)


def xent_case(n, k, v, dt, masked, seed):
    g = gen(seed)
    h = randn(g, n, k).to(dt)
    w = (randn(g, v, k) * (2 / math.sqrt(k))).to(dt)
    y = torch.randint(0, v, (n,), generator=g, device="cuda")
    y[torch.rand(n, generator=g, device="cuda") < masked] = -100
    grad = torch.rand(n, generator=g, device="cuda") / n * (torch.rand(n, generator=g, device="cuda") - 0.3).sign()
    return h, w, y, grad


def xent_check(h, w, y, grad):
    loss, lse = os2.xent(h, w, y)
    dh, dw = os2.xent_backward(h, w, y, lse, grad)
    assert dh.dtype == h.dtype and dw.dtype == w.dtype
    want, tol = xent_want(h, w, y, grad)
    for got, x, t in zip((loss, lse, dh, dw), want, tol):
        close(got, x, t)
    return loss, lse, dh, dw


XENT_SHAPES = [(1, 1, 1), (1, 64, 2), (2, 8, 300), (1, 1024, 32000), (7, 33, 129), (31, 100, 1000), (64, 256, 511),
               (130, 72, 257), (128, 128, 256), (256, 512, 1024), (257, 520, 700), (300, 1000, 5021), (513, 640, 2049)]


@pytest.mark.parametrize("n,k,v", XENT_SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_xent(n, k, v, dt):
    xent_check(*xent_case(n, k, v, DT[dt], 0.0, n + k + v))


@pytest.mark.parametrize("n,masked", [(1, 1.0), (5, 0.5), (300, 0.4), (700, 0.9), (400, 1.0), (1500, 0.3)])
def test_xent_masked_rows(n, masked):
    for dt in (torch.bfloat16, torch.float16):
        h, w, y, grad = xent_case(n, 200, 900, dt, masked, n)
        loss, lse, dh, dw = xent_check(h, w, y, grad)
        out = y == -100
        assert (loss[out] == 0).all() and (lse[out] == 0).all() and (dh[out] == 0).all()
        # what ignored rows hold reaches nothing
        h2, g2 = h.clone(), grad.clone()
        h2[out] = math.nan
        g2[out] = math.inf
        l2, s2 = os2.xent(h2, w, y)
        dh2, dw2 = os2.xent_backward(h2, w, y, s2, g2)
        assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(dh2, dh) and torch.equal(dw2, dw)
        if masked == 1.0:
            assert (dw == 0).all()


def test_xent_strides_and_alignment():
    h, w, y, grad = xent_case(150, 136, 700, torch.bfloat16, 0.2, 3)
    want = xent_check(h, w, y, grad)
    for off, pad in ((0, 8), (1, 7), (3, 2), (8, 0)):
        H = torch.full((150, 136 + off + pad), 9.0, dtype=h.dtype, device="cuda")
        W = torch.full((700, 136 + off + pad), 9.0, dtype=h.dtype, device="cuda")
        H[:, off:off + 136], W[:, off:off + 136] = h, w
        hv, wv = H[:, off:off + 136], W[:, off:off + 136]
        loss, lse = os2.xent(hv, wv, y)
        dh, dw = os2.xent_backward(hv, wv, y, lse, grad)
        for a, b in zip((loss, lse, dh, dw), want):
            assert torch.equal(a, b)
    y2 = torch.stack([y, y], 1)[:, 0]          # strided labels and gradients
    g2 = torch.stack([grad, grad], 1)[:, 0]
    loss, lse = os2.xent(h, w, y2)
    dh, dw = os2.xent_backward(h, w, y2, lse, g2)
    assert torch.equal(loss, want[0]) and torch.equal(dh, want[2]) and torch.equal(dw, want[3])
    only = os2.xent_backward(h, w, y, want[1], grad, need_dw=False)
    assert torch.equal(only[0], want[2]) and only[1] is None
    only = os2.xent_backward(h, w, y, want[1], grad, need_dh=False)
    assert only[0] is None and torch.equal(only[1], want[3])


@pytest.mark.parametrize("scale", [30.0, 300.0])
def test_xent_large_logits(scale):
    """Logits far apart: one column takes all, sums neither overflow nor vanish."""
    h, w, y, grad = xent_case(70, 64, 600, torch.bfloat16, 0.0, 5)
    xent_check((h.float() * scale).to(h.dtype), w, y, grad)


def test_xent_small_gradients_in_f16():
    """The gradient of a mean over many rows, in a type whose smallest normal
    number is 6e-5: entries of D down to 1e-9 of the largest must survive."""
    h, w, y, grad = xent_case(200, 64, 3001, torch.float16, 0.0, 6)
    xent_check(h * 30, w, y, grad * 1e-3)
    xent_check(h, w, y, grad * 0)


def test_xent_non_finite():
    h, w, y, grad = xent_case(40, 64, 300, torch.bfloat16, 0.0, 8)
    h2 = h.clone()
    h2[3, 5] = math.nan
    loss, lse = os2.xent(h2, w, y)
    base, _ = os2.xent(h, w, y)
    assert torch.isnan(loss[3]) and torch.isnan(lse[3])
    rest = torch.arange(40, device="cuda") != 3
    assert torch.equal(loss[rest], base[rest])
    dh, _ = os2.xent_backward(h2, w, y, lse, grad)
    assert torch.isnan(dh[3]).all() and not torch.isnan(dh[rest]).any()


def test_xent_label_out_of_range_is_reported():
    h, w, y, grad = xent_case(20, 64, 300, torch.bfloat16, 0.0, 9)
    base, lse0 = os2.xent(h, w, y)
    for bad in (300, -1, 1 << 40):
        y2 = y.clone()
        y2[4] = bad
        loss, lse = os2.xent(h, w, y2)
        assert os2.get_status() == os2.binding.ERR_RANGE
        assert loss[4] == 0 and lse[4] == 0
        rest = torch.arange(20, device="cuda") != 4
        assert torch.equal(loss[rest], base[rest])
    y2 = y.clone()
    y2[4] = 7
    loss, _ = os2.xent(h, w, y2, ignore_index=7)
    assert loss[4] == 0 and os2.get_status() == 0


def test_xent_gradient_against_differences():
    """d/dt loss(H + t A, W + t B) by central differences of the 64-bit
    definition, against the kernel's gradients."""
    h, w, y, grad = xent_case(24, 40, 90, torch.float16, 0.25, 11)
    loss, lse = os2.xent(h, w, y)
    dh, dw = os2.xent_backward(h, w, y, lse, grad)
    valid = y != -100

    def f(hh, ww):
        z = hh @ ww.t()
        l = torch.logsumexp(z, 1) - z.gather(1, torch.where(valid, y, 0)[:, None])[:, 0]
        return (torch.where(valid, l, 0.0) * grad.double()).sum()

    g = gen(12)
    a, b = randn(g, 24, 40).double(), randn(g, 90, 40).double()
    t = 1e-5
    h64, w64 = h.double(), w.double()
    _, (_, _, th, tw) = xent_want(h, w, y, grad)
    for da, db in ((a, 0 * b), (0 * a, b)):
        num = (f(h64 + t * da, w64 + t * db) - f(h64 - t * da, w64 - t * db)) / (2 * t)
        got = (dh.double() * da).sum() + (dw.double() * db).sum()
        bound = (th * da.abs()).sum() + (tw * db.abs()).sum() + 1e-9
        assert abs(num - got) <= bound


def test_xent_autograd():
    h, w, y, _ = xent_case(50, 64, 500, torch.bfloat16, 0.3, 13)
    h.requires_grad_(True)
    w.requires_grad_(True)
    loss = os2.XentFunction.apply(h, w, y, -100).sum() / (y != -100).sum()
    loss.backward()
    grad = (y != -100).float() / (y != -100).sum()
    (want, _, dh, dw), (tl, _, th, tw) = xent_want(h.detach(), w.detach(), y, grad)
    close(loss.detach(), (want * grad.double()).sum(), (tl * grad.double()).sum() + 1e-6)
    close(h.grad, dh, th)
    close(w.grad, dw, tw)


def test_xent_pieces_of_the_vocabulary():
    """So many rows that D comes in pieces of 2048 columns, the last one short."""
    n, k, v = 66000, 64, 4100
    h, w, y, grad = xent_case(n, k, v, torch.bfloat16, 0.1, 14)
    loss, lse = os2.xent(h, w, y)
    dh, dw = os2.xent_backward(h, w, y, lse, grad)
    wantw, tolw = 0, 0
    for r in torch.arange(n, device="cuda").split(16500):
        (l, s, ph, pw), (tl, _, th, tw) = xent_want(h[r], w, y[r], grad[r])
        close(loss[r], l, tl)
        close(dh[r], ph, th)
        wantw, tolw = wantw + pw, tolw + tw
    close(dw, wantw, tolw + (n / 16) * 2.0 ** -22 * 4)


def test_xent_empty():
    h, w, y, grad = xent_case(0, 64, 50, torch.bfloat16, 0.0, 15)
    loss, lse = os2.xent(h, w, y)
    dh, dw = os2.xent_backward(h, w, y, lse, grad)
    assert loss.shape == (0,) and dh.shape == (0, 64) and (dw == 0).all()


def test_xent_refuses_what_does_not_match():
    h, w, y, grad = xent_case(6, 16, 50, torch.bfloat16, 0.0, 16)
    for f in (lambda: os2.xent(h.float(), w.float(), y), lambda: os2.xent(h, w.half(), y),
              lambda: os2.xent(h, w[:, :8], y), lambda: os2.xent(h, w, y.int()), lambda: os2.xent(h, w, y[:5]),
              lambda: os2.xent(h.t(), w, y), lambda: os2.xent_backward(h, w, y, grad[:5], grad),
              lambda: os2.xent_backward(h, w, y, grad, grad.double())):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(os2.Os2Error):
        os2.xent(h, w, y, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


# -------------------------------------------------------------------- AdamW
B1, B2, EPS, WD, LR = 0.9, 0.97, 1e-8, 0.1, 3e-3
f32 = np.float32


def np_of(t):
    return t.detach().float().cpu().numpy()


def update32(m, v, g):
    return m * f32(B1) + g * f32(1 - B1), v * f32(B2) + (g * g) * f32(1 - B2)


def p_want(p, m, v, step):
    """The parameters in 64 bits from the new moments, and their bound: four FP32
    roundings of p, and 2^-20 of the update (square root, quotient, constants)."""
    p, m, v = (x.astype(np.float64) for x in (p, m, v))
    up = LR * (m / (1 - B1 ** step)) / (np.sqrt(v / (1 - B2 ** step)) + EPS)
    return p * (1 - LR * WD) - up, np.abs(p) * 2.0 ** -22 + np.abs(up) * 2.0 ** -20


def encode(m, v):
    """Codes and scales of one tensor, FP32 operation by operation."""
    n = m.size
    pad = -n % 256
    m, v = np.pad(m, (0, pad)).reshape(-1, 256), np.pad(v, (0, pad)).reshape(-1, 256)
    am, av = np.abs(m).max(1), v.max(1)
    dm, dv = np.where(am > 0, am, f32(1))[:, None], np.where(av > 0, av, f32(1))[:, None]
    cm = np.rint(np.sqrt(np.abs(m) / dm) * f32(127)) * np.sign(m)
    cv = np.rint(np.sqrt(np.sqrt(v / dv)) * f32(255))
    cv = np.where(v > 0, np.maximum(cv, 1), cv)
    return cm.astype(np.int8).reshape(-1)[:n], am, cv.astype(np.uint8).reshape(-1)[:n], av


def decode(cm, am, cv, av):
    a = cm.astype(f32) * f32(1 / 127)
    b = cv.astype(f32) * f32(1 / 255)
    b = b * b
    return np.repeat(am, 256)[:cm.size] * (a * np.abs(a)), np.repeat(av, 256)[:cv.size] * (b * b)


SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 10000, 0, 3]


@pytest.mark.parametrize("pt,gt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("align", [0, 1])
def test_adamw_32(pt, gt, align):
    """align 1: tensors that start off every 16-byte boundary."""
    g = gen(5)
    sizes = SIZES * 30                       # more tensors than one launch takes
    store = lambda dt, s: [(randn(g, n + align) * s).to(dt)[align:] for n in sizes]  # noqa: E731
    p, gr = store(DT[pt], 0.05), store(DT[gt], 1e-2)
    m, v = store(torch.float32, 1e-3), [x.square() for x in store(torch.float32, 1e-2)]
    if align:
        v = [torch.cat([x[:1], x])[1:] if x.numel() else x for x in v]
    p0, g0, m0, v0 = ([np_of(x) for x in xs] for xs in (p, gr, m, v))
    os2.adamw(p, gr, m, v, step=3, lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD)
    for i in range(len(sizes)):
        mw, vw = update32(m0[i], v0[i], g0[i])
        assert np.array_equal(np_of(m[i]), mw) and np.array_equal(np_of(v[i]), vw)
        want, tol = p_want(p0[i], mw, vw, 3)
        u = U[DT[pt]] * 1.01 * np.abs(want) + TINY[DT[pt]] if pt != "f32" else 0
        assert (np.abs(np_of(p[i]) - want) <= tol + u).all()


@pytest.mark.parametrize("pt,gt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_adamw_8bit(pt, gt):
    """Three steps from zero moments: the codes and scales are those of the
    definition, bit for bit, and the parameters follow."""
    g = gen(6)
    p = [(randn(g, n) * 0.05).to(DT[pt]) for n in SIZES]
    z = lambda dt, d: [torch.zeros(-(-n // d), dtype=dt, device="cuda") for n in SIZES]  # noqa: E731
    cm, cv, am, av = z(torch.int8, 1), z(torch.uint8, 1), z(torch.float32, 256), z(torch.float32, 256)
    for step in (1, 2, 3):
        gr = [(randn(g, n) * torch.exp(3 * randn(g, n)) * 1e-3).to(DT[gt]) for n in SIZES]
        gr[8][100:900] = 0                   # blocks of zeros, and zeros within blocks
        before = [[np_of(x) if x.is_floating_point() else x.cpu().numpy() for x in xs] for xs in (p, gr, cm, am, cv, av)]
        os2.adamw(p, gr, cm, cv, step=step, lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, exp_avg_scales=am,
                  exp_avg_sq_scales=av)
        for i, n in enumerate(SIZES):
            if not n:
                continue
            p0, g0, c0, a0, d0, b0 = (x[i] for x in before)
            mw, vw = update32(*decode(c0, a0, d0, b0), g0)
            want, tol = p_want(p0, mw, vw, step)
            u = U[DT[pt]] * 1.01 * np.abs(want) + TINY[DT[pt]] if pt != "f32" else 0
            assert (np.abs(np_of(p[i]) - want) <= tol + u).all()
            ec, ea, ed, eb = encode(mw, vw)
            assert np.array_equal(am[i].cpu().numpy(), ea) and np.array_equal(av[i].cpu().numpy(), eb)
            assert np.array_equal(cm[i].cpu().numpy(), ec) and np.array_equal(cv[i].cpu().numpy(), ed)
            mm, vv = os2.adamw_moments(cm[i], am[i], cv[i], av[i])
            md, vd = decode(ec, ea, ed, eb)
            assert np.array_equal(np_of(mm), md) and np.array_equal(np_of(vv), vd)
            assert ((vd > 0) == (vw > 0)).all()


def test_adamw_8bit_codes_near_ties():
    """Moments chosen so that their codes lie at, and one bit beside, the ties of
    the rounding: still the definition's."""
    c = torch.arange(0, 127, device="cuda", dtype=torch.float32)
    mid = ((c + 0.5) / 127).square() * 0.7
    vals = torch.cat([torch.nextafter(mid, torch.zeros_like(mid)), mid])
    m = torch.cat([vals, torch.full((1,), 0.7, device="cuda"), torch.zeros(1, device="cuda")])
    c = torch.arange(0, 127, device="cuda", dtype=torch.float32) * 2 + 0.5
    mid = (c / 255).square().square() * 0.31
    g2 = torch.cat([torch.nextafter(mid, torch.ones_like(mid)), mid, torch.full((2,), 0.31, device="cuda")])
    # beta1 = beta2 = 0: the new moments are the gradient and its square
    for grad in (m, -m, g2.sqrt()):
        p = torch.zeros(256, device="cuda")
        cm, cv = torch.zeros(256, dtype=torch.int8, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
        am, av = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        os2.adamw([p], [grad], [cm], [cv], step=1, lr=1e-3, beta1=0.0, beta2=0.0, exp_avg_scales=[am], exp_avg_sq_scales=[av])
        gn = np_of(grad)
        ec, ea, ed, eb = encode(gn, gn * gn)
        assert np.array_equal(cm.cpu().numpy(), ec) and np.array_equal(cv.cpu().numpy(), ed)


def test_adamw_non_finite_gradients_stay_local():
    for q8 in (False, True):
        p = torch.ones(1000, device="cuda")
        g = torch.ones(1000, device="cuda") * 1e-3
        g[10] = math.nan
        if q8:
            m, v = torch.zeros(1000, dtype=torch.int8, device="cuda"), torch.zeros(1000, dtype=torch.uint8, device="cuda")
            kw = dict(exp_avg_scales=[torch.zeros(4, device="cuda")], exp_avg_sq_scales=[torch.zeros(4, device="cuda")])
        else:
            m, v, kw = torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda"), {}
        os2.adamw([p], [g], [m], [v], step=1, lr=1e-3, **kw)
        assert torch.isnan(p[10])
        bad = torch.isnan(p)
        bad[10] = False
        assert not bad.any()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_adamw_8bit_non_finite_blocks(bad):
    """A non-finite gradient shows in the moments of its block, and in no other."""
    p, g = torch.ones(1000, device="cuda"), torch.full((1000,), 1e-3, device="cuda")
    g[300] = bad
    m, v = torch.zeros(1000, dtype=torch.int8, device="cuda"), torch.zeros(1000, dtype=torch.uint8, device="cuda")
    am, av = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    kw = dict(exp_avg_scales=[am], exp_avg_sq_scales=[av])
    os2.adamw([p], [g], [m], [v], step=1, lr=1e-3, **kw)
    mm, vv = os2.adamw_moments(m, am, v, av)
    for x in (mm, vv):
        assert torch.isfinite(x[:256]).all() and torch.isfinite(x[512:]).all()
        assert not torch.isfinite(x[256:512]).any()
    os2.adamw([p], [torch.full_like(g, 1e-3)], [m], [v], step=2, lr=1e-3, **kw)
    assert torch.isnan(p[256:512]).all() and torch.isfinite(p[:256]).all() and torch.isfinite(p[512:]).all()


def test_adamw_large_tensor_offsets():
    """Elements past 2^31: the last ones are updated like the first."""
    n = (1 << 31) + 1000
    if torch.cuda.mem_get_info()[0] < 12 * n:
        pytest.skip("not enough free memory")
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[:300] = 1e-2
    g[-300:] = 1e-2
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    nb = -(-n // 256)
    am, av = torch.zeros(nb, device="cuda"), torch.zeros(nb, device="cuda")
    os2.adamw([p], [g], [m], [v], step=1, lr=1e-3, exp_avg_scales=[am], exp_avg_sq_scales=[av])
    assert torch.equal(p[:300], p[-300:]) and (p[:300] != 0).all() and (p[300:1000] == 0).all()
    assert (m[-300:] == 127).all() and (v[-300:] == 255).all() and (m[-1000:-300] == 0).all()


def test_adamw_refuses_what_does_not_match():
    x = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    kw = dict(step=1, lr=1e-3)
    i8, u8 = torch.int8, torch.uint8
    for f in (lambda: os2.adamw([x(4)], [x(5)], [x(4)], [x(4)], **kw),
              lambda: os2.adamw([x(4)], [x(4)], [x(4), x(4)], [x(4)], **kw),
              lambda: os2.adamw([x(4)], [x(4)], [x(4).half()], [x(4)], **kw),
              lambda: os2.adamw([x(4, 4).t()], [x(4, 4)], [x(4, 4)], [x(4, 4)], **kw),
              lambda: os2.adamw([x(4), x(4).half()], [x(4)] * 2, [x(4)] * 2, [x(4)] * 2, **kw),
              lambda: os2.adamw([x(4)], [x(4)], [x(4, dt=i8)], [x(4, dt=u8)], **kw),
              lambda: os2.adamw([x(4)], [x(4)], [x(4, dt=i8)], [x(4, dt=u8)], exp_avg_scales=[x(1)], **kw),
              lambda: os2.adamw([x(300)], [x(300)], [x(300, dt=i8)], [x(300, dt=u8)], exp_avg_scales=[x(1)],
                                exp_avg_sq_scales=[x(2)], **kw),
              lambda: os2.adamw_moments(x(300, dt=i8), x(1), x(300, dt=u8), x(2))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(os2.Os2Error):
        os2.adamw([x(4)], [x(4)], [x(4)], [x(4)], step=0, lr=1e-3)


# ------------------------------------------------------------------ streams
def test_calls_on_another_stream():
    """Everything a call reads, writes and allocates is ordered on its stream."""
    s = torch.cuda.Stream()
    h, w, y, grad = xent_case(300, 256, 3000, torch.bfloat16, 0.2, 17)
    x = randn(gen(18), 40, 700)
    wq, sb = os2.quantize_rows(randn(gen(19), 500, 700))
    base = os2.xent(h, w, y)
    base_g = os2.xent_backward(h, w, y, base[1], grad)
    base_y = os2.i8linear(x, wq, sb)
    p = torch.ones(5000, device="cuda")
    m, v, g = torch.zeros_like(p), torch.zeros_like(p), torch.full_like(p, 1e-3)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        # work in front, so that a call that did not wait for it would read too early
        h2 = torch.zeros_like(h)
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = big @ big * 1e-3
        h2.copy_(h)
    loss, lse = os2.xent(h2, w, torch.stack([y, y], 1)[:, 0], stream=s)
    dh, dw = os2.xent_backward(h2, w, y, lse, grad, stream=s)
    yy = os2.i8linear(x, wq, sb, stream=s.cuda_stream)
    os2.adamw([p], [g], [m], [v], step=1, lr=1e-3, stream=s)
    s.synchronize()
    assert torch.equal(loss, base[0]) and torch.equal(dh, base_g[0]) and torch.equal(dw, base_g[1])
    assert torch.equal(yy, base_y)
    assert (p != 1).all()


def test_calls_from_several_threads():
    """Threads that share a stream do not share a workspace, streams neither: every
    call's result is its own."""
    import threading
    x = [randn(gen(30 + i), 5 + 30 * i, 640) for i in range(4)]
    wq, sb = os2.quantize_rows(randn(gen(40), 700, 640))
    h, w, y, _ = xent_case(60, 128, 900, torch.bfloat16, 0.2, 41)
    want = [os2.i8linear(v, wq, sb) for v in x]
    base = os2.xent(h, w, y)[0]
    torch.cuda.synchronize()
    bad = []

    def work(i, stream):
        for _ in range(50):
            if not torch.equal(os2.i8linear(x[i], wq, sb, stream=stream), want[i]):
                bad.append(i)
            if not torch.equal(os2.xent(h, w, y, stream=stream)[0], base):
                bad.append(-1)

    s = torch.cuda.Stream()

    def run(i):
        with torch.cuda.stream(s if i < 2 else torch.cuda.Stream()):
            work(i, None)

    ts = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_repeats_are_bit_identical():
    h, w, y, grad = xent_case(700, 300, 3000, torch.bfloat16, 0.2, 20)
    x = randn(gen(21), 70, 1500).bfloat16()
    wq, sb = os2.quantize_rows(randn(gen(22), 900, 1500))
    runs = []
    for _ in range(3):
        loss, lse = os2.xent(h, w, y)
        runs.append((loss, lse, *os2.xent_backward(h, w, y, lse, grad), os2.i8linear(x, wq, sb)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_calls_can_be_captured_in_a_graph():
    h, w, y, grad = xent_case(100, 128, 1000, torch.bfloat16, 0.2, 23)
    wq, sb = os2.quantize_rows(randn(gen(24), 300, 128))
    loss, lse = os2.xent(h, w, y)
    want = (loss, *os2.xent_backward(h, w, y, lse, grad), os2.i8linear(h, wq, sb))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = os2.xent(h, w, y)
        got = (loss, *os2.xent_backward(h, w, y, lse, grad), os2.i8linear(h, wq, sb))
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
