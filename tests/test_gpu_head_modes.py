"""What looks on in PyTorch's dispatcher sees the head operators' outputs come into being."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import rns_emulated_fp64_gb300 as os2
from test_gpu_head import clean_status, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in str(func):
            self.shapes.append(tuple(out.shape))
        return out


def calls():
    g = gen(1)
    x, w, v = randn(g, 20, 64).bfloat16(), torch.ones(64, device="cuda"), (randn(g, 48, 64) / 8).bfloat16()
    u, dy = torch.rand(20, generator=g, device="cuda"), randn(g, 20, 48).bfloat16()
    q, s = os2.quantize_rows(v)
    labels = torch.arange(20, device="cuda")
    lse = os2.xent(x, v, labels)[1]
    return {"quantize_rows": (lambda: os2.quantize_rows(x), [(20, 64), (20,)]),
            "i8linear": (lambda: (os2.i8linear(x, q, s),), [(20, 48)]),
            "xent": (lambda: os2.xent(x, v, labels), [(20,), (20,)]),
            "xent_backward": (lambda: os2.xent_backward(x, v, labels, lse, torch.ones_like(lse)), [(20, 64), (48, 64)]),
            "rmsnorm": (lambda: os2.rmsnorm(x, w, residual=x), [(20, 64), (20, 64)]),
            "rmsnorm_quantize": (lambda: os2.rmsnorm_quantize(x, w), [(20, 64), (20,)]),
            "rmsnorm_backward": (lambda: os2.rmsnorm_backward(x, w, x), [(20, 64), (64,)]),
            "linear": (lambda: os2.linear(x, v, return_pre=True), [(20, 48), (20, 48)]),
            "linear_backward": (lambda: os2.linear_backward(x, v, dy, need_db=True), [(20, 64), (48, 64), (48,)]),
            "sample": (lambda: os2.sample(dy, u), [(20,), (20,)])}


@pytest.mark.parametrize("name", ["quantize_rows", "i8linear", "xent", "xent_backward", "rmsnorm", "rmsnorm_quantize", "rmsnorm_backward",
                                  "linear", "linear_backward", "sample"])
def test_outputs_are_seen(name):
    f, shapes = calls()[name]
    want = f()
    with Seen() as seen:
        got = f()
    assert sorted(s for s in seen.shapes if s in shapes) == sorted(shapes)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.autograd.profiler.profile() as prof:
        got = f()
    assert sum(e.count for e in prof.key_averages() if e.key == "aten::empty") >= len(shapes)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        got = f()
    finally:
        torch.use_deterministic_algorithms(before)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
