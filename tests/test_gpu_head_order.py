"""Calls of the vocabulary-head operators one right after another: their launches
overlap, and each still sees what the ones before it wrote, to the last bit."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2

pytestmark = pytest.mark.gpu
TURNS = 12


def inputs(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(*shape, generator=g, device="cuda") * 0.3).to(dtype) for _ in range(TURNS)]


@pytest.mark.parametrize("m", [1, 12, 40, 70, 300])
@pytest.mark.parametrize("k", [2048, 1777])
def test_weights_quantised_just_before(m, k):
    n = 4096
    ws, xs = inputs(1, n, k), inputs(2, m, k)
    q, s = os2.quantize_rows(ws[0])
    apart = []
    for w, x in zip(ws, xs):
        q, s = os2.quantize_rows(w)
        torch.cuda.synchronize()
        apart.append(os2.i8linear(x, q, s))
        torch.cuda.synchronize()
    q, s = torch.zeros_like(q), torch.zeros_like(s)
    at_once = []
    for w, x in zip(ws, xs):
        os2.quantize_rows(w, out=q, scale=s)
        at_once.append(os2.i8linear(x, q, s))
    assert all(torch.equal(a, b) for a, b in zip(at_once, apart))
    # what one call gives goes into the next
    square = torch.randint(-127, 128, (k, k), dtype=torch.int8, device="cuda")
    scale = torch.full((k,), 1e-3, device="cuda")
    a = b = xs[0]
    for _ in range(TURNS):
        a = os2.i8linear(a, square, scale)
        torch.cuda.synchronize()
    for _ in range(TURNS):
        b = os2.i8linear(b, square, scale)
    assert torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("n", [1, 16, 100, 600])
@pytest.mark.parametrize("k", [512, 511])
def test_head_changed_just_before(n, k):
    v = 9000
    ws, hs = inputs(3, v, k), inputs(4, n, k)
    y = torch.randint(0, v, (n,), device="cuda")
    if n > 1:
        y[::3] = -100
    g = torch.rand(n, device="cuda")

    def run(wait):
        W, H, out = torch.zeros_like(ws[0]), torch.zeros_like(hs[0]), []
        for w, h in zip(ws, hs):
            W.copy_(w)
            H.copy_(h)
            wait()
            loss, lse = os2.xent(H, W, y)
            wait()
            dh, dw = os2.xent_backward(H, W, y, lse, g)
            wait()
            only_h, none = os2.xent_backward(H, W, y, lse, g, need_dw=False)
            none2, only_w = os2.xent_backward(H, W, y, lse, g, need_dh=False)
            assert none is None and none2 is None
            out += [loss, lse, dh, dw, only_h, only_w]
        wait()
        return out

    apart, at_once = run(torch.cuda.synchronize), run(lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(at_once, apart))
    for i in range(0, len(apart), 6):
        assert torch.equal(apart[i + 2], apart[i + 4]) and torch.equal(apart[i + 3], apart[i + 5])


def test_pieces_of_the_vocabulary_in_turn():
    """Several pieces, each adding to the FP32 sums of dH beside dW's product."""
    n, k, v = 60000, 64, 6000
    h, w = inputs(5, n, k)[0], inputs(6, v, k)[0]
    y = torch.randint(0, v, (n,), device="cuda")
    loss, lse = os2.xent(h, w, y)
    g = torch.full((n,), 1.0 / n, device="cuda")
    first = os2.xent_backward(h, w, y, lse, g)
    for _ in range(3):
        again = os2.xent_backward(h, w, y, lse, g)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    z = h.double() @ w.double().t()
    d = torch.softmax(z, 1)
    d[torch.arange(n), y] -= 1
    d /= n
    # D is rounded once, relative 2^-8 an entry; the sums and the results' roundings are below that
    for got, want, size in ((first[0], d @ w.double(), d.abs() @ w.double().abs()),
                            (first[1], d.t() @ h.double(), d.abs().t() @ h.double().abs())):
        assert ((got.double() - want).abs() <= 2.0 ** -7 * size + 1e-12).all()


def test_lists_are_checked():
    p = [torch.zeros(300, device="cuda"), torch.zeros(3, 5, device="cuda")]
    z = [torch.zeros_like(t) for t in p]
    q = [torch.zeros_like(t, dtype=torch.int8) for t in p]
    u = [torch.zeros_like(t, dtype=torch.uint8) for t in p]
    sc = [torch.zeros(2, device="cuda"), torch.zeros(1, device="cuda")]
    ok = dict(step=1, lr=1e-3)
    for f in (lambda: os2.adamw(p, z[:1], z, z, **ok), lambda: os2.adamw(p, [z[0], None], z, z, **ok),
              lambda: os2.adamw(p, [z[0], z[1].t()], z, z, **ok), lambda: os2.adamw(p, [z[0], z[1].half()], z, z, **ok),
              lambda: os2.adamw(p, z, [z[0].cpu(), z[1]], z, **ok), lambda: os2.adamw(p, z, [t.half() for t in z], z, **ok),
              lambda: os2.adamw(p, z, q, u, **ok), lambda: os2.adamw(p, z, q, u, exp_avg_scales=sc, **ok),
              lambda: os2.adamw(p, z, q, u, exp_avg_scales=sc, exp_avg_sq_scales=sc[::-1], **ok)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        os2.adamw(p, 3, z, z, **ok)
    with pytest.raises(TypeError):
        os2.adamw(p, z, z, z, step=1, lr="much")
    with pytest.raises(os2.Os2Error):
        os2.adamw(p, z, z, z, step=0, lr=1e-3)
    os2.adamw((t for t in p), tuple(z), z, z, **ok)          # any iterables
    os2.adamw(p, z, q, u, exp_avg_scales=sc, exp_avg_sq_scales=sc, **ok)
    assert all((t == 0).all() for t in p)
