"""An output of the caller's that lies over weight, bias or another output is refused; beside them it is taken."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from test_gpu_head import clean_status, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def test_outputs_over_weights_and_scales():
    g = gen(1)
    n, d = 24, 64
    x, r = randn(g, n, d).bfloat16(), randn(g, n, d).bfloat16()
    y, h = torch.zeros(n + 1, d, device="cuda").bfloat16(), torch.zeros(n + 1, d, device="cuda").bfloat16()
    q, s = torch.zeros(n + 1, d, dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda")
    w = torch.ones(d, device="cuda").bfloat16()
    W = randn(g, d, d).bfloat16()

    def floats(t, off=0):                              # n float32 values of t's memory
        return t.view(-1).view(torch.float32)[off:off + n]

    for name, wrong in (
            ("out must not overlap weight", lambda: os2.rmsnorm(x, y[n], out=y[1:])),
            ("out must not overlap weight", lambda: os2.rmsnorm(x, y[3], residual=r, out=y[:n], out_h=h[:n])),
            ("out must not overlap weight", lambda: os2.rmsnorm(x, y.view(-1)[5:5 + d], out=y[:n])),
            ("out_h must not overlap weight", lambda: os2.rmsnorm(x, h[0], residual=r, out_h=h[:n])),
            ("out must not overlap weight", lambda: os2.rmsnorm_quantize(x, q.view(-1).view(torch.bfloat16)[:d], out=q[:n])),
            ("out_h must not overlap weight", lambda: os2.rmsnorm_quantize(x, h[n - 1], residual=r, out_h=h[:n])),
            ("scale must not overlap X", lambda: os2.rmsnorm_quantize(x, w, scale=floats(x))),
            ("scale must not overlap X", lambda: os2.rmsnorm_quantize(x[:, :32], w[:32], scale=floats(x, 10))),
            ("scale must not overlap residual", lambda: os2.rmsnorm_quantize(x, w, residual=r, scale=floats(r, n * d // 2 - n))),
            ("scale must not overlap weight", lambda: os2.rmsnorm_quantize(x, w, scale=floats(w))),
            ("scale must not overlap out", lambda: os2.rmsnorm_quantize(x, w, out=q[:n], scale=floats(q, 3))),
            ("scale must not overlap out_h", lambda: os2.rmsnorm_quantize(x, w, residual=r, out_h=h[:n], scale=floats(h, 7))),
            ("out must not overlap bias", lambda: os2.linear(x, W, bias=y[2], out=y[:n])),
            ("out must not overlap bias", lambda: os2.linear(x, W, bias=y.view(-1).view(torch.float32)[:d], out=y[:n]))):
        with pytest.raises(ValueError, match=name):
            wrong()
    assert (y == 0).all() and (h == 0).all() and (q == 0).all() and (s == 0).all()


def test_outputs_beside_weights_and_scales():
    g = gen(2)
    n, d = 24, 64
    x, r, w, b = randn(g, n, d).bfloat16(), randn(g, n, d).bfloat16(), 1 + randn(g, d).bfloat16() / 4, randn(g, d)
    W = (randn(g, d, d) / 8).bfloat16()
    y, h = os2.rmsnorm(x, w, residual=r)
    q, s, _ = os2.rmsnorm_quantize(x, w, residual=r)
    z = os2.linear(x, W, bias=b)
    room = torch.zeros(n + 1, 4 * d, device="cuda").bfloat16()
    wide = room[:, d:2 * d]
    room[3, :d] = w                                    # the weight in the gap between out's rows,
    wv = room[3, :d]
    os2.rmsnorm(x, wv, residual=r, out=wide[:n], out_h=room[:n, 2 * d:3 * d])
    assert torch.equal(wide[:n], y) and torch.equal(room[:n, 2 * d:3 * d], h) and torch.equal(wv, w)
    room[n, d:2 * d] = w                               # and behind its last row
    os2.rmsnorm(x, room[n, d:2 * d], residual=r, out=wide[:n])
    assert torch.equal(wide[:n], y)
    flat = torch.zeros(n * d // 4 + n, device="cuda")  # integers and scales in one buffer
    qv, sv = flat[:n * d // 4].view(torch.int8).view(n, d), flat[n * d // 4:]
    os2.rmsnorm_quantize(x, w, residual=r, out=qv, scale=sv)
    assert torch.equal(qv, q) and torch.equal(sv, s)
    room[5, :2 * d].view(torch.float32)[:] = b         # a float32 bias in the gap
    bv = room[5, :2 * d].view(torch.float32)
    os2.linear(x, W, bias=bv, out=room[:n, 2 * d:3 * d])
    assert torch.equal(room[:n, 2 * d:3 * d], z)
