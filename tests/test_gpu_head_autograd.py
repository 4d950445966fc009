"""The vocabulary-head operators and autograd: what they write in place is seen."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from test_gpu_head import clean_status, gen, randn, xent_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
def test_a_step_before_the_gradient_is_refused(q8):
    """The loss saves W; a step that changes W before the gradient is taken would
    give the new W's, so autograd raises, as after any in-place operation."""
    h, w, y, _ = xent_case(50, 64, 500, torch.bfloat16, 0.0, 31)
    w.requires_grad_(True)
    m, v = ((torch.zeros(w.shape, dtype=d, device="cuda") for d in (torch.int8, torch.uint8)) if q8 else
            (torch.zeros(w.shape, device="cuda") for _ in range(2)))
    kw = {k: [torch.zeros(w.numel() // 256, device="cuda")] for k in ("exp_avg_scales", "exp_avg_sq_scales")} if q8 else {}
    g = torch.full_like(w, 1e-3, requires_grad=False)

    def step():
        written = [w, m, v] + [t for x in kw.values() for t in x]
        before = [t._version for t in written + [g]]
        os2.adamw([w.detach()], [g], [m], [v], step=1, lr=1e-3, **kw)
        assert [t._version - b for t, b in zip(written, before)] == [1] * len(written)
        assert g._version == before[-1]

    loss = os2.XentFunction.apply(h, w, y, -100).sum()
    step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    loss = os2.XentFunction.apply(h, w, y, -100).sum()
    loss.backward()                              # in the usual order
    step()
    with pytest.raises(os2.Os2Error):            # a call that fails writes nothing
        before = w._version
        os2.adamw([w.detach()], [g], [m], [v], step=0, lr=1e-3, **kw)
    assert w._version == before


def test_outputs_given_by_the_caller_are_written_in_place():
    x = randn(gen(3), 40, 64)
    q, s = torch.empty(40, 64, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    y = torch.empty(40, 40, device="cuda")
    v = [t._version for t in (q, s, y, x)]
    os2.quantize_rows(x, out=q, scale=s)
    os2.i8linear(x, q, s, out=y)
    os2.i8gemm(q, s, q, s, out=y)
    assert [t._version - b for t, b in zip((q, s, y, x), v)] == [1, 1, 2, 0]


def test_inference_tensors():
    with torch.inference_mode():
        p, g = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
        m, v = torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda")
        os2.adamw([p], [g], [m], [v], step=1, lr=1e-3)
    os2.adamw([p], [g], [m], [v], step=2, lr=1e-3)
    assert (p < 1).all()
