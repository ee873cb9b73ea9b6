"""A NaN (or an infinity) in a block of an operator's result gives the scale
byte that the quantizers give to such a block, 247, and the codes under it;
the rowwise output likewise."""
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


def _same(q, s, x, F):
    """Codes and bytes of ``x``'s blocks, in the blocks that are not finite."""
    want_q, want_s = F.fp8moe_mxfp8_quantize_dim0(x)
    bad = ~torch.isfinite(x.float()).unflatten(-1, (-1, 32)).all(-1)
    assert bool(bad.any()) and bool((want_s[bad] == 247).all())
    assert torch.equal(s.view_as(want_s)[bad], want_s[bad])
    assert torch.equal(q.unflatten(-1, (-1, 32))[bad], want_q.unflatten(-1, (-1, 32))[bad])
    assert not bool((s.view_as(want_s)[~bad] == 247).any())


@pytest.mark.parametrize("M", [64, 20480])
@pytest.mark.parametrize("bwd", [False, True])
def test_activation(F, M, bwd):
    Fd = 128
    g = torch.Generator().manual_seed(2)
    h, d = torch.randn(M, 2 * Fd, generator=g).to(torch.bfloat16), torch.randn(M, Fd, generator=g).to(torch.bfloat16)
    h[3, 40], h[5, Fd + 70], h[M - 1, 2 * Fd - 1] = float("nan"), float("nan"), float("inf")
    call = (lambda **k: F.fp8moe_swiglu_bwd(d.to(DEV), h.to(DEV), **k)) if bwd else (lambda **k: F.fp8moe_swiglu_fwd(h.to(DEV), **k))
    out, q0, s0, q1, s1 = call(dim0=True, dim1=True, s0_layout=F.SCALES_ROWMAJOR, s1_layout=F.SCALES_ROWMAJOR)
    _same(q0, s0, out, F)
    _same(q1, s1, out.t().contiguous(), F)


@pytest.mark.parametrize("H", [64, 512, 2048, 8192, 20480])
def test_norm(F, H):
    """A NaN input makes its row NaN; an infinite weight or a NaN one its column."""
    g = torch.Generator().manual_seed(H)
    for T in (5, 400):
        x, w = torch.randn(T, H, generator=g).to(torch.bfloat16), torch.ones(H)
        x[1, 7] = float("nan")
        w[H - 3], w[H - 40] = float("inf"), float("nan")
        x[2, H - 3] = 1.0
        _, y, _, q, s = F.fp8moe_add_rmsnorm_fwd(x.to(DEV), w.to(DEV), recipe=F.MXFP8)
        _same(q, s, y, F)


@pytest.mark.parametrize("H", [64, 512, 2048, 8192, 20480])
@pytest.mark.parametrize("kind", [0, 1])
def test_norm_rowwise(F, H, kind):
    g = torch.Generator().manual_seed(H)
    for T in (5, 400):
        x, w = torch.randn(T, H, generator=g).to(torch.bfloat16), torch.ones(H)
        w[H - 40] = float("nan")
        _, y, _, q, inv = F.fp8moe_add_rmsnorm_fwd(x.to(DEV), w.to(DEV), recipe=F.ROWWISE, kind=kind)
        want_q, want_inv = F.fp8moe_quantize_rowwise(y, kind)
        assert torch.equal(inv, want_inv) and torch.equal(q, want_q)
