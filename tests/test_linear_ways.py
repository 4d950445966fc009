"""The query for a linear layer's kernels: arguments and names.  No GPU needed."""
import pytest

import rns_emulated_fp64_gb300 as os2
from rns_emulated_fp64_gb300 import binding as b


def test_query():
    w = os2.linear_ways(1, 4096, 4096)
    assert set(w) == {"way", "tokens", "cluster", "parts", "dx_way", "dx_tokens", "dx_cluster", "dx_parts", "dw_parts"}
    assert w["way"] == w["dx_way"] == 0 and w["tokens"] == w["dx_tokens"] == 16 and w["parts"] == w["dx_parts"] == 1
    w = os2.linear_ways(8192, 16384, 4096, "silu", pre=True)
    assert w["way"] == 1 and w["tokens"] == 256 and w["parts"] == 1


def test_refusals():
    for args, status in (((0, 8, 8), b.ERR_INVALID_ARG), ((1, 0, 8), b.ERR_INVALID_ARG), ((1, 8, 0), b.ERR_INVALID_ARG),
                         (((1 << 22) + 1, 8, 8), b.ERR_UNSUPPORTED), ((1, 8, 1 << 24), b.ERR_UNSUPPORTED)):
        with pytest.raises(os2.Os2Error) as e:
            os2.linear_ways(*args)
        assert e.value.status == status
    with pytest.raises(ValueError):
        os2.linear_ways(1, 8, 8, "swish")
    assert os2.load().os2_linear_ways(1, 8, 8, 0, 0, 0, 1, None) == b.ERR_INVALID_ARG
    assert os2.load().os2_linear_ways(1, 8, 8, 9, 0, 0, 1, None) == b.ERR_INVALID_ARG
