"""The combine's weight gradient reads no row that y does not have."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


@pytest.mark.parametrize("T,N,k", [(3, 8, 1), (2600, 64, 8), (50, 264, 3), (700, 1032, 5), (9, 7168, 11)])
def test_row_numbers_past_the_last_row_are_missing(F, T, N, k):
    """The bits that -1 in their place gives: y is the first part of a buffer
    whose other rows hold NaN, and the numbers reach from its end to 2^31 - 1."""
    g = torch.Generator().manual_seed(N)
    rows = T * k // 2 + 1
    buf = torch.full((T * k + 8, N), float("nan"), dtype=torch.bfloat16)
    buf[:rows] = torch.randn(rows, N, generator=g).to(torch.bfloat16)
    y, dout = buf.to(DEV)[:rows], torch.randn(T, N, generator=g).to(torch.bfloat16).to(DEV)
    row_of = torch.randint(0, T * k, (T, k), generator=g).to(torch.int32)
    row_of[0, 0] = rows
    row_of[T - 1, k - 1] = 2 ** 31 - 1
    row_of[T // 2, 0] = -2 ** 31
    missing = torch.where((row_of < 0) | (row_of >= rows), torch.full_like(row_of, -1), row_of)
    got = F.fp8moe_route_weight_grad(dout, y, row_of.to(DEV))
    assert torch.equal(got, F.fp8moe_route_weight_grad(dout, y, missing.to(DEV)))
    assert bool(torch.isfinite(got).all()) and not got[(missing < 0).to(DEV)].any()
    # without rows everything is missing
    assert not F.fp8moe_route_weight_grad(dout, y[:0], row_of.to(DEV)).any()
