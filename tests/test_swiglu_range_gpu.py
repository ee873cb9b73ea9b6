"""The gated activation over the whole range of its inputs: gates far out on
both sides, factors whose product leaves fp32 although the result does not,
NaN and infinities, forward and backward, in the form for few tiles and in the
one for many.

Tolerances as in test_swiglu_gpu: 1e-6 of the terms that are added; below the
normal range fp32 values and products are off by 2^-150 each, a handful of
them, times a gate of at most 80: 2e-43."""
import numpy as np
import pytest
import torch

from code_bounds import check_bf16, check_mx
from oracle import moe_ops as OM

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL, TINY = 1e-6, 2e-43
MAX = 3.3895313892515355e38   # bf16's largest
GATES = [MAX, 3e38, 1e30, 1e10, 300.0, 200.0, 190.0, 177.0, 160.0, 140.0, 120.0, 104.0, 100.0, 96.0, 92.0, 90.0, 89.0, 88.5,
         88.0, 87.5, 87.0, 85.5, 81.0, 80.5, 80.0, 79.5, 64.0, 40.0, 20.0, 1.28125, 0.5, 1e-38]
UPS = [0.0, 1e-38, 1e-30, 1e-20, 1e-10, 1e-3, 1.0, 2.0, 3.0, 1e4, 1e10, 9e18, 1e19, 2e19, 1e25, 1e30, 1e33, 3e36, 1e37, 1e38,
       2e38, MAX]


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _np(t):
    return t.double().cpu().numpy()


def _bf(v):
    return torch.tensor(v, dtype=torch.float64).to(torch.bfloat16)


def _signed(v):
    return v + [-x for x in v]


# rows: 64 gates; columns: ups (and output gradients) in every combination
def _case(bwd, rows):
    g = _bf(_signed(GATES))
    if bwd:
        few = _signed([1e-38, 1e-20, 1.0, 3.0, 1e10, 1e20, 1e30, MAX])
        u, d = _bf(few).repeat(16), _bf(few).repeat_interleave(16)
    else:
        u, d = _bf(_signed(UPS) + [0.25] * 20), None
    F, n = u.numel(), g.numel()
    h = torch.cat([g[:, None].expand(n, F), u[None].expand(n, F)], 1).repeat(rows // n, 1).contiguous()
    return h, None if d is None else d[None].expand(rows, F).contiguous()


def _ref(h, d):
    with np.errstate(over="ignore", invalid="ignore"):
        if d is None:
            v = OM.swiglu(_np(h))
            return v, REL * np.abs(v) + TINY
        v = OM.swiglu_grad(_np(d), _np(h))
        g, u = np.split(_np(h), 2, axis=1)
        s = OM._sig(g)
        size = np.concatenate([np.abs(_np(d) * u) * s * (1 + np.abs(g) * (1 - s)), np.abs(_np(d) * g) * s], axis=1)
        return v, REL * size + TINY


def _call(F, h, d, **kw):
    h = h.to(DEV)
    if d is None:
        return F.fp8moe_swiglu_fwd(h, **kw)
    return F.fp8moe_swiglu_bwd(d.to(DEV), h, **kw)


# 64 x 128 tiles: below and above the number of SMs
@pytest.mark.parametrize("rows", [64, 19712])
@pytest.mark.parametrize("bwd", [False, True])
def test_whole_range(F, bwd, rows):
    h, d = _case(bwd, rows)
    out = _call(F, h, d)[0]
    assert bool((out.view(rows // 64, 64, -1).view(torch.int16) == out[:64].view(torch.int16)).all())
    v, tol = _ref(h[:64], None if d is None else d[:64])
    with np.errstate(over="ignore"):
        check_bf16(out[:64], v, tol, "bf16")


@pytest.mark.parametrize("rows", [64, 19712])
@pytest.mark.parametrize("bwd", [False, True])
def test_codes_of_far_gates(F, bwd, rows):
    """Blocks along both dims whose values are finite in fp32."""
    h, d = _case(bwd, rows)
    v, tol = _ref(h, d)
    h[:, h.shape[1] // 2:][torch.from_numpy(np.abs(v[:, :h.shape[1] // 2]) > 1e38)] = 0.0
    if bwd:
        d[torch.from_numpy(np.abs(v[:, d.shape[1]:]) > 1e38)] = 0.0
    v, tol = _ref(h, d)
    assert np.abs(v).max() < 2e38
    _, q0, s0, q1, s1 = _call(F, h, d, s0_layout=F.SCALES_ROWMAJOR, s1_layout=F.SCALES_ROWMAJOR, dim0=True, dim1=True)
    W = v.shape[1]
    check_mx(q0.cpu().numpy(), s0.cpu().numpy().reshape(rows, W // 32), v, tol, "dim0")
    check_mx(q1.cpu().numpy(), s1.cpu().numpy().reshape(W, rows // 32), v.T, tol.T, "dim1")


@pytest.mark.parametrize("rows", [64, 19712])
@pytest.mark.parametrize("bwd", [False, True])
def test_nan_and_infinity_stay_where_they_belong(F, bwd, rows):
    """A NaN or an infinity reaches exactly the results that depend on it, with
    the values that the formulas give in 64 bits."""
    Fd = 128
    gen = torch.Generator().manual_seed(1)
    h = torch.randn(rows, 2 * Fd, generator=gen).to(torch.bfloat16)
    d = torch.randn(rows, Fd, generator=gen).to(torch.bfloat16) if bwd else None
    inf, nan = float("inf"), float("nan")
    h[1, 3], h[1, Fd + 5], h[2, 7], h[2, 9], h[3, Fd + 1], h[3, Fd + 2] = nan, nan, inf, -inf, inf, -inf
    h[4, 11], h[4, Fd + 11] = -300.0, inf
    h[rows - 1, 64], h[rows - 2, Fd + 65] = nan, nan
    if bwd:
        d[5, 1], d[5, 2], d[rows - 3, 66] = nan, inf, nan
    out, q0, s0, q1, s1 = _call(F, h, d, dim0=True, dim1=True, s0_layout=F.SCALES_ROWMAJOR, s1_layout=F.SCALES_ROWMAJOR)
    with np.errstate(over="ignore", invalid="ignore"):
        v = OM.swiglu(_np(h)) if d is None else OM.swiglu_grad(_np(d), _np(h))
        got = _np(out)
        assert np.array_equal(np.isnan(got), np.isnan(v))
        assert np.array_equal(np.isinf(got), np.isinf(v)) and np.array_equal(np.sign(got[np.isinf(v)]), np.sign(v[np.isinf(v)]))
        fin = np.isfinite(v)
        assert np.all(np.abs(got[fin] - v[fin]) <= 2.0 ** -7 * np.abs(v[fin]) + 1e-6)
    assert np.array_equal(q0.cpu().numpy() & 0x7F == 0x7F, np.isnan(v))
    assert np.array_equal((q1.cpu().numpy() & 0x7F == 0x7F).T, np.isnan(v))
