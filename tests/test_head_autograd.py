"""``XentFunction`` in autograd, with the operators themselves in plain PyTorch."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from rns_emulated_fp64_gb300 import head


@pytest.fixture
def plain(monkeypatch):
    def xent(H, W, labels, ignore_index=-100):
        z = H @ W.t()
        lse = torch.logsumexp(z, 1)
        return lse - z.gather(1, labels[:, None])[:, 0], lse

    def backward(H, W, labels, lse, grad, ignore_index, need_dh, need_dw):
        d = torch.exp(H @ W.t() - lse[:, None])
        d.scatter_add_(1, labels[:, None], torch.full_like(d[:, :1], -1.0))
        d *= grad[:, None]
        return d @ W if need_dh else None, d.t() @ H if need_dw else None

    monkeypatch.setattr(head, "xent", xent)
    monkeypatch.setattr(head, "xent_backward", backward)


def case():
    g = torch.Generator().manual_seed(1)
    H, W = torch.randn(5, 7, generator=g), torch.randn(11, 7, generator=g)
    return H.requires_grad_(True), W.requires_grad_(True), torch.randint(0, 11, (5,), generator=g)


def test_first_gradients(plain):
    H, W, y = case()
    os2.XentFunction.apply(H, W, y).mean().backward()
    got = H.grad, W.grad
    H.grad = W.grad = None
    torch.nn.functional.cross_entropy(H @ W.t(), y).backward()
    for a, b in zip(got, (H.grad, W.grad)):
        assert torch.allclose(a, b, atol=1e-5)
    H.grad = W.grad = None
    W.requires_grad_(False)
    os2.XentFunction.apply(H, W, y).mean().backward()
    assert W.grad is None and torch.allclose(H.grad, got[0], atol=1e-6)


def test_a_gradient_of_the_gradient_is_refused(plain):
    """A penalty on the gradient would lose this operator's part without a word."""
    H, W, y = case()
    message = "no gradient of its own"
    for weights in (torch.ones(5), torch.rand(5, requires_grad=True)):
        dh, dw = torch.autograd.grad((os2.XentFunction.apply(H, W, y) * weights).sum(), (H, W), create_graph=True)
        with pytest.raises(RuntimeError, match=message):
            dh.square().sum().backward(retain_graph=True)
        # nor as a part of a larger sum, whose other parts do have a graph
        with pytest.raises(RuntimeError, match=message):
            (dw.square().sum() + H.square().sum()).backward()
    # with create_graph and no second pass, the gradients are what they were
    other = torch.autograd.grad(os2.XentFunction.apply(H, W, y).sum(), (H, W))
    for a, b in zip(torch.autograd.grad(os2.XentFunction.apply(H, W, y).sum(), (H, W), create_graph=True), other):
        assert torch.equal(a, b) and a.requires_grad and not b.requires_grad
    W.requires_grad_(False)
    dh, = torch.autograd.grad(os2.XentFunction.apply(H, W, y).sum(), H, create_graph=True)
    with pytest.raises(RuntimeError, match=message):
        dh.square().sum().backward()
