"""The stream of a call of the vocabulary-head operators, given by its handle."""
import contextlib

import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from rns_emulated_fp64_gb300 import head


class OnDevice:
    def get_device(self):
        return 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its device's current stream would be the call's, not the tensors'."""
    class Stream:
        def __init__(self, index):
            self.device_index = index

    seen = []
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: seen.append(s) or contextlib.nullcontext())
    assert head._run(lambda: 3, Stream(0), OnDevice()) == 3 and len(seen) == 1
    with pytest.raises(ValueError, match="cuda:1"):
        head._run(lambda: 3, Stream(1), OnDevice())
    with pytest.raises(ValueError, match="one CUDA device"):
        head._run(lambda: 3, Stream(0), torch.zeros(2))
    assert len(seen) == 1
    for stream in (Stream(0), 0):                 # what is no tensor is the call's to refuse
        os2.adamw([], [], [], [], step=1, lr=1e-3, stream=stream)
        with pytest.raises(ValueError, match="must be a tensor"):
            os2.quantize_rows([1.0], stream=stream)


def test_the_default_streams_handles(monkeypatch):
    seen = []
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device: ("external", ptr, device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: seen.append(s) or contextlib.nullcontext())

    for stream in (0, 1, 2, 0x7F0010):
        assert head._run(lambda x: x, stream, OnDevice(), 5) == 5
    assert head._run(lambda x: x, None, OnDevice(), 6) == 6
    assert seen == [("default", 0), ("default", 0), ("external", 2, 0), ("external", 0x7F0010, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [0, 1])
def test_calls_on_the_default_stream_by_its_handle(handle):
    """Work in front on the default stream writes what the call reads; the call, made
    while another stream is the current one, waits for it."""
    assert torch.cuda.default_stream().cuda_stream == 0
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, w, x = randn(300, 256).bfloat16(), (randn(3000, 256) / 8).bfloat16(), randn(40, 700)
    y = torch.randint(0, 3000, (300,), generator=g, device="cuda")
    grad = torch.full((300,), 1 / 300, device="cuda")
    wq, sb = os2.quantize_rows(randn(500, 700))
    q, sa = os2.quantize_rows(x)
    p, pg = randn(5000), randn(5000)
    codes = torch.randint(-127, 128, (5000,), generator=g, device="cuda").to(torch.int8)
    scales = torch.rand(20, generator=g, device="cuda")
    loss, lse = os2.xent(h, w, y)

    def calls(t, stream):
        """t: the tensors that the work in front writes"""
        h, x, q, pg, codes = t
        m, v, p2 = torch.zeros_like(p), torch.zeros_like(p), p.clone()
        torch.cuda.current_stream().synchronize()

        def step():
            os2.adamw([p2], [pg], [m], [v], step=1, lr=1e-3, stream=stream)
            return p2, m, v

        return [lambda: os2.quantize_rows(x, stream=stream), lambda: (os2.i8gemm(q, sa, wq, sb, stream=stream),),
                lambda: (os2.i8linear(x, wq, sb, stream=stream),), lambda: os2.xent(h, w, y, stream=stream),
                lambda: os2.xent_backward(h, w, y, lse, grad, stream=stream), step,
                lambda: os2.adamw_moments(codes, scales, codes.view(torch.uint8), scales, stream=stream)]

    real = [h, x, q, pg, codes]
    want = [f() for f in calls(real, None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late = [torch.zeros_like(t) for t in real]
        for i, call in enumerate(calls(late, handle)):
            for t in late:
                t.zero_()
            side.synchronize()
            with torch.cuda.stream(torch.cuda.default_stream()):
                big = torch.randn(4096, 4096, device="cuda")
                for _ in range(20):
                    big = big @ big * 1e-3
                for t, r in zip(late, real):
                    t.copy_(r)
            got = call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
    assert os2.get_status() == 0
