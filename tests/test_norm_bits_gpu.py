"""The norm backward's mean is a division by the row's length."""
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


@pytest.mark.parametrize("H", [24, 40, 56, 88, 200, 328, 1064, 2072, 5160, 8200, 13336, 16440, 40040])
def test_equal_gradients_along_a_row_of_equal_values_cancel(F, H):
    """h = rstd = w = 1 and dy = c: dx = c - c H / H, and c H has no rounding
    (8 bits times at most 16)."""
    T = 256
    dy = (1.0 + torch.arange(T) / 128 % 1).to(torch.bfloat16)[:, None].expand(T, H).contiguous().to(DEV)
    h = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    for dh in (None, torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)):
        for w in (torch.ones(H, device=DEV), torch.ones(H, dtype=torch.bfloat16, device=DEV)):
            dx, _ = F.fp8moe_add_rmsnorm_bwd(dy, h, torch.ones(T, device=DEV), w, dh)
            assert not dx.any()


@pytest.mark.parametrize("H", [24, 1064, 5160, 16440])
def test_infinite_sum(F, H):
    """A row whose sum overflows: -inf times each value, as by a division."""
    big = torch.full((3, H), 2.0 ** 126, dtype=torch.bfloat16, device=DEV)
    h = torch.ones(3, H, dtype=torch.bfloat16, device=DEV)
    h[:, 1] = -1.0
    w = torch.ones(H, device=DEV)
    dx, _ = F.fp8moe_add_rmsnorm_bwd(big, h, torch.ones(3, device=DEV), w)
    assert bool((dx == -float("inf") * h).all())
