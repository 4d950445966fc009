"""Matrices whose rows repeat or overlap (expanded tensors, sliding windows) are
refused by every entry point: read at a pitch of their width they would be read
past the end of their storage."""
import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from rns_emulated_fp64_gb300 import binding

ROWS, K, N = 6, 40, 6


def overlapping(dtype, device, rows=ROWS, k=K):
    """The same row again and again; a window that moves by one and by half."""
    x = torch.ones(4 * rows * k, dtype=dtype, device=device)
    return [x[:k].unsqueeze(0).expand(rows, k), x.as_strided((rows, k), (1, 1)), x.as_strided((rows, k), (k // 2, 1)),
            x[:1].unsqueeze(0).expand(rows, 1)]


def head_calls(device):
    """(type of the matrix, call that takes it)"""
    f32, bf, i8 = torch.float32, torch.bfloat16, torch.int8
    ones = lambda n, dt=f32: torch.ones(n, dtype=dt, device=device)  # noqa: E731
    mat = lambda x, dt=None: torch.ones(ROWS, x.shape[1], dtype=dt or x.dtype, device=device)  # noqa: E731
    labels, e = torch.zeros(ROWS, dtype=torch.int64, device=device), ones(ROWS)
    return [(f32, lambda x: os2.quantize_rows(x)),
            (i8, lambda x: os2.i8gemm(x, e, mat(x), e)), (i8, lambda x: os2.i8gemm(mat(x), e, x, e)),
            (bf, lambda x: os2.i8linear(x, mat(x, i8), e)), (i8, lambda x: os2.i8linear(mat(x, bf), x, e)),
            (bf, lambda x: os2.xent(x, mat(x), labels)), (bf, lambda x: os2.xent(mat(x), x, labels)),
            (bf, lambda x: os2.xent_backward(x, mat(x), labels, e, e)),
            (bf, lambda x: os2.xent_backward(mat(x), x, labels, e, e))]


def refused(calls, device):
    for dtype, call in calls:
        for x in overlapping(dtype, device):
            with pytest.raises(ValueError, match="overlap"):
                call(x)


def test_head_refuses_overlapping_rows_on_the_host():
    """The first matrix of a call: the second is looked at after the first is found to be on a device."""
    refused([c for i, c in enumerate(head_calls("cpu")) if i in (0, 1, 3, 5, 7)], "cpu")


def test_leading_dimension():
    x = torch.zeros(5, 12, dtype=torch.float64)
    assert binding._ld(x, "x") == 12 and binding._ld(x[:, 2:7], "x") == 12 and binding._ld(x[::2], "x") == 24
    assert binding._ld(x[:1].expand(1, 12), "x") == 12 and binding._ld(x[:0], "x") == 12
    assert binding._ld(torch.zeros(3, 0), "x") == 1 and binding._ld(x[:1, :1].expand(1, 1), "x") == 1
    for y in overlapping(torch.float64, "cpu"):
        with pytest.raises(ValueError, match="overlap"):
            binding._ld(y, "y")


def test_host_products_refuse_overlapping_rows():
    x = torch.ones(ROWS, K, dtype=torch.float64)
    c = torch.zeros(ROWS, N, dtype=torch.float64)
    for y, z in zip(overlapping(torch.float64, "cpu")[:3], overlapping(torch.float64, "cpu", k=N)):
        for args in ((y, x, c), (x, y, c), (x, x, z)):
            with pytest.raises(ValueError, match="overlap"):
                os2.gemm_host(*args)


@pytest.mark.gpu
def test_overlapping_rows_on_the_device():
    dev = "cuda"
    refused(head_calls(dev), dev)
    f64, f32, c128 = torch.float64, torch.float32, torch.complex128
    mat = lambda x, n=None: torch.ones(ROWS, n or x.shape[1], dtype=x.dtype, device=dev)  # noqa: E731
    e = torch.zeros(ROWS, dtype=torch.int32, device=dev)
    calls = []
    for dt, f in ((f64, os2.gemm), (f64, binding.gemm_noalloc), (f32, os2.sgemm), (c128, os2.zgemm)):
        calls += [(dt, lambda x, f=f: f(x, mat(x))), (dt, lambda x, f=f: f(mat(x), x)),
                  (dt, lambda x, f=f: f(mat(x), torch.ones(x.shape[1], x.shape[1], dtype=x.dtype, device=dev), out=x))]
    calls += [(f64, lambda x: binding.scale(x, mat(x))), (f64, lambda x: binding.scale(mat(x), x)),
              (f64, lambda x: binding.residues(x, e, 4)), (f64, lambda x: binding.scale_bounds(x, mat(x))),
              (f64, lambda x: binding.gemm_exponents(mat(x), x, 4, e, e))]
    # (a width of one: the older checks ask for a column stride of 1, which that view does not have)
    for dtype, call in calls:
        for x in overlapping(dtype, dev)[:3]:
            with pytest.raises(ValueError, match="overlap"):
                call(x)
    assert os2.get_status() == 0


@pytest.mark.gpu
def test_rows_apart_and_single_rows_still_work():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    big = torch.randn(8, 200, generator=g, device="cuda")
    q, s = os2.quantize_rows(big[::2, 10:110])
    q2, s2 = os2.quantize_rows(big[::2, 10:110].contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)
    one = big[0, :100].unsqueeze(0).expand(1, 100)          # a single row may have any stride
    assert torch.equal(os2.quantize_rows(one)[0], os2.quantize_rows(one.contiguous())[0])
    A, B = big[:, :64].double(), torch.randn(5, 90, generator=g, device="cuda").double()[:, 3:67]
    assert torch.equal(os2.gemm(A, B), os2.gemm(A.contiguous(), B.contiguous()))
    assert os2.get_status() == 0
