"""NaN in the gated activation's inputs, forward and backward, in the form for
few tiles and in the one for many."""
import numpy as np
import pytest
import torch

from oracle import moe_ops as OM

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _np(t):
    return t.double().cpu().numpy()


def _call(F, h, d, **kw):
    h = h.to(DEV)
    if d is None:
        return F.fp8moe_swiglu_fwd(h, **kw)
    return F.fp8moe_swiglu_bwd(d.to(DEV), h, **kw)


@pytest.mark.parametrize("rows", [64, 19712])
@pytest.mark.parametrize("bwd", [False, True])
def test_nan_stays_where_it_belongs(F, bwd, rows):
    """A NaN reaches exactly the results that depend on it."""
    Fd = 128
    gen = torch.Generator().manual_seed(1)
    h = torch.randn(rows, 2 * Fd, generator=gen).to(torch.bfloat16)
    d = torch.randn(rows, Fd, generator=gen).to(torch.bfloat16) if bwd else None
    nan = float("nan")
    h[1, 3], h[1, Fd + 5] = nan, nan
    h[rows - 1, 64], h[rows - 2, Fd + 65] = nan, nan
    if bwd:
        d[5, 1], d[rows - 3, 66] = nan, nan
    out, q0, s0, q1, s1 = _call(F, h, d, dim0=True, dim1=True, s0_layout=F.SCALES_ROWMAJOR, s1_layout=F.SCALES_ROWMAJOR)
    with np.errstate(invalid="ignore"):
        v = OM.swiglu(_np(h)) if d is None else OM.swiglu_grad(_np(d), _np(h))
        got = _np(out)
        assert np.array_equal(np.isnan(got), np.isnan(v))
        fin = np.isfinite(v)
        assert np.all(np.abs(got[fin] - v[fin]) <= 2.0 ** -7 * np.abs(v[fin]) + 1e-6)
    assert np.array_equal(q0.cpu().numpy() & 0x7F == 0x7F, np.isnan(v))
    assert np.array_equal((q1.cpu().numpy() & 0x7F == 0x7F).T, np.isnan(v))
