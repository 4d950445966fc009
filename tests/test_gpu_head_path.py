"""The vocabulary head's operators together, as a user runs them, and over the
debug build, whose kernels check their hand-computed indices."""
import importlib.util
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns_and_serves():
    """200 steps take the loss from about log 1000 to below 0.5 (labels follow a rule
    that a 128-wide head can hold), and the 8-bit head serves what it learned."""
    spec = importlib.util.spec_from_file_location("vocab_head", os.path.join(ROOT, "examples", "vocab_head.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, right = ex.main(["--steps", "200"])
    assert losses[0] > 5.0 and losses[-1] < 0.5
    assert right > 0.95


SCRIPT = r'''
import torch
import rns_emulated_fp64_gb300 as os2
assert os2.binding.lib_path().endswith("_build_debug/libos2.so"), os2.binding.lib_path()
g = torch.Generator(device="cuda")
g.manual_seed(1)
randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
for m, n, k in [(1, 5, 7), (3, 300, 200), (17, 1000, 700), (40, 260, 1100), (130, 700, 333), (600, 900, 1500)]:
    w, sb = os2.quantize_rows(randn(n, k))
    x = randn(m, k)
    q, sa = os2.quantize_rows(x)
    y = os2.i8linear(x, w, sb, out_dtype=torch.float32)
    want = (q.double() @ w.double().t()) * sa.double()[:, None] * sb.double()
    assert (y.double() - want).abs().max() <= 1e-6 * want.abs().max()
for n, k, v in [(1, 8, 3), (5, 64, 500), (40, 33, 257), (300, 520, 1100)]:
    h, w = randn(n, k).bfloat16(), (randn(v, k) * k ** -0.5).bfloat16()
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::3] = -100
    loss, lse = os2.xent(h, w, t)
    dh, dw = os2.xent_backward(h, w, t, lse, torch.ones(n, device="cuda"))
    z = h.double() @ w.double().t()
    want = torch.where(t >= 0, torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0)
    assert (loss.double() - want).abs().max() < 1e-4
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()
for q8 in (False, True):
    p = [torch.ones(s, device="cuda") for s in (1, 300, 5000)]
    gr = [torch.full_like(x, 1e-3) for x in p]
    mt, vt = (torch.int8, torch.uint8) if q8 else (torch.float32, torch.float32)
    m, v = ([torch.zeros(x.shape, dtype=d, device="cuda") for x in p] for d in (mt, vt))
    kw = {}
    if q8:
        kw = {a: [torch.zeros(-(-x.numel() // 256), device="cuda") for x in p]
              for a in ("exp_avg_scales", "exp_avg_sq_scales")}
    os2.adamw(p, gr, m, v, step=1, lr=1e-2, **kw)
    assert all((x < 1).all() for x in p)
torch.cuda.synchronize()
st = os2.get_status()
assert st == 0, os2.status_string(st)
print("debug build ok")
'''


def test_debug_build_finds_no_bad_index():
    from rns_emulated_fp64_gb300 import build as b
    lib = b.build(debug=True)
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env={**os.environ, "OS2_LIB": lib},
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "debug build ok" in r.stdout
