"""What the cross entropy's backward pass asks for as workspace."""
import ctypes as ct

import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from rns_emulated_fp64_gb300 import binding as b

P = ct.c_void_p(0x1000)       # never dereferenced
FWD, BWD, BWD_BF16 = 0, 1, 2
F16, BF16 = 1, 2


def test_only_f16_holds_the_logits_gradients_twice():
    lib = os2.load()
    size = lib.os2_xent_workspace_size
    n, k, v = 2048, 2048, 32768
    d = n * v * 2                                 # one piece: the whole vocabulary
    one, two = size(n, k, v, P, k, BWD_BF16), size(n, k, v, P, k, BWD)
    assert two - one == d and d < one < d + 2 * n * k * 4 * 2 + (1 << 20)
    for n in (1, 300, 1 << 16, 1 << 20):
        npad = -(-n // 256) * 256
        one, two = size(n, 64, 1 << 18, P, 64, BWD_BF16), size(n, 64, 1 << 18, P, 64, BWD)
        assert 0 < two - one <= max(npad * 2048 * 2, 1 << 28)


def test_a_call_refuses_less_than_its_size():
    lib = os2.load()
    size = lib.os2_xent_workspace_size
    small, large = size(40, 8, 500, P, 8, BWD_BF16), size(40, 8, 500, P, 8, BWD)
    assert size(40, 8, 500, P, 8, FWD) < small < large
    for dt, nb in ((BF16, small - 1), (F16, large - 1), (F16, small)):
        assert lib.os2_xent_backward(40, 8, 500, dt, P, 8, P, 8, P, -100, P, P, P, 8, P, 8, P, nb, None) == b.ERR_WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_a_workspace_of_exactly_that_size(dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    n, k, v = 300, 128, 3001
    h, w = (torch.randn(s, k, generator=g, device="cuda").to(dt) for s in (n, v))
    y = torch.randint(0, v, (n,), generator=g, device="cuda")
    grad = 2.0 ** torch.linspace(-20, 0, n, device="cuda")
    loss, lse = os2.xent(h, w, y)
    want = os2.xent_backward(h, w, y, lse, grad)
    need = os2.load().os2_xent_workspace_size(n, k, v, w.data_ptr(), k, BWD_BF16 if dt == torch.bfloat16 else BWD)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    got = os2.xent_backward(h, w, y, lse, grad, workspace=room[:need])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (room[need:] == 77).all()
    with pytest.raises(os2.Os2Error):
        os2.xent_backward(h, w, y, lse, grad, workspace=room[:need - 256])
