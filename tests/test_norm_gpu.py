"""Residual addition + RMS norm with an 8-bit output against the float64
definition.

Tolerances.  Forward: the sum of squares has positive terms, at most 32 added
in a row by a thread, then 5 shuffles and at most 32 warps: a relative error
of at most 70 * 2^-24, halved by the root, plus a few ulp of the root, the
division and the two products: below 4e-6 of |y|.  Backward: the same count
on sum |g xh|, doubled for the products inside.  bf16 outputs lie between
the roundings of the two ends."""
import numpy as np
import pytest
import torch

from code_bounds import check_bf16, check_mx, check_rows
from oracle import formats as OF, moe_ops as OM, swizzle as OS

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL, GREL = 4e-6, 1e-5
EPS = 1e-5


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def _np(t):
    return t.double().cpu().numpy()


def _near(got, ref, tol, what):
    lim = tol + np.abs(ref) * 2.0 ** -23 + 1e-38
    assert np.all(np.abs(got - ref) <= lim), f"{what}: {float((np.abs(got - ref) / lim).max())} of the bound"


def _weight(H, seed, w32):
    w = 1.0 + 0.2 * torch.randn(H, generator=torch.Generator().manual_seed(seed))
    return w if w32 else w.to(torch.bfloat16)


# row lengths: one warp, ragged warps, every chunk count per thread, and the
# rows that are read again (H > 16384)
SIZES = [(1, 32), (5, 96), (3, 1024), (17, 2048), (2, 2080), (9, 4096), (4, 5120), (3, 7168), (2, 16384), (3, 16416),
         (2, 40960), (700, 256)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("residual,w32,tiled", [(True, False, False), (False, True, True)])
def test_forward_mx(F, T, H, residual, w32, tiled):
    x, w = _bf16((T, H), H + T), _weight(H, 7, w32)
    r = _bf16((T, H), H + T + 1, 3.0) if residual else None
    x[:, 3] *= 40
    if T > 2:
        x[1] = 0
        if residual:
            r[1] = 0
    a, rstd, y = OM.add_rmsnorm(_np(x), None if r is None else _np(r), _np(w), EPS)
    layout = F.NO_GROUPS if tiled else F.SCALES_ROWMAJOR
    h, yo, rs, q, s = F.fp8moe_add_rmsnorm_fwd(x.to(DEV), w.to(DEV), None if r is None else r.to(DEV), eps=EPS,
                                               recipe=F.MXFP8, scale_layout=layout)
    if residual:
        assert torch.equal(h.cpu(), (x.float() + r.float()).to(torch.bfloat16))
    else:
        assert h is None
    check_bf16(yo, y, REL * np.abs(y), "y")
    _near(_np(rs), rstd, REL * rstd, "rstd")
    byte = s.cpu().numpy()
    if tiled:
        rp, cp = OS.swizzled_shape(T, H // 32)
        full = OS.unswizzle(byte[:rp * cp], rp, cp)
        byte = full[:T, :H // 32].copy()
        full[:T, :H // 32] = 0
        assert not full.any(), "padding bytes"
    check_mx(q.cpu().numpy(), byte, y, REL * np.abs(y), "codes")


def test_tiled_padding_is_written(F):
    """A scale buffer of any contents ends with zero padding bytes."""
    T, H = 131, 160
    n = F.fp8moe_swizzled_scales_bytes(1, T, H // 32)
    s = torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)
    x = _bf16((T, H), 3).to(DEV)
    F.fp8moe_add_rmsnorm_fwd(x, _weight(H, 1, False).to(DEV), recipe=F.MXFP8, scale_layout=F.NO_GROUPS, scale=s)
    rp, cp = OS.swizzled_shape(T, H // 32)
    full = OS.unswizzle(s.cpu().numpy(), rp, cp)
    assert not full[T:].any() and not full[:, H // 32:].any() and full[:T, :H // 32].all()


@pytest.mark.parametrize("T,H", [(1, 16), (5, 48), (3, 1040), (6, 4096), (2, 8192), (2, 16400)])
@pytest.mark.parametrize("kind,okind", [(0, OF.FN), (1, OF.FNUZ)])
def test_forward_rowwise(F, T, H, kind, okind):
    x, r, w = _bf16((T, H), H), _bf16((T, H), H + 1), _weight(H, 2, True)
    if T > 1:
        x[1], r[1] = 0, 0
    _, _, y = OM.add_rmsnorm(_np(x), _np(r), _np(w), EPS)
    _, yo, rs, q, inv = F.fp8moe_add_rmsnorm_fwd(x.to(DEV), w.to(DEV), r.to(DEV), eps=EPS, recipe=F.ROWWISE, kind=kind,
                                                 need_y=False, need_rstd=False)
    assert yo is None and rs is None
    check_rows(q.cpu().numpy(), _np(inv), y, REL, okind, "codes")


def test_strides_in_place_and_bf16_only(F):
    """Row strides above H, the residual stream updated in place, H a multiple
    of 8 alone, no 8-bit output."""
    T, H = 13, 200
    wide, rw = _bf16((T, H + 24), 5).to(DEV), _bf16((T, H + 56), 6).to(DEV)
    x, r, w = wide[:, :H], rw[:, 8:8 + H], _weight(H, 3, False).to(DEV)
    a, _, y = OM.add_rmsnorm(_np(x), _np(r), _np(w), EPS)
    h, yo, _, q, s = F.fp8moe_add_rmsnorm_fwd(x, w, r, eps=EPS)
    assert q is None and s is None
    assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16))
    check_bf16(yo, y, REL * np.abs(y), "y")
    for H2 in (200, 16800):     # both kernels
        x2, r2 = _bf16((T, H2), 8).to(DEV), _bf16((T, H2), 9).to(DEV)
        w2 = _weight(H2, 3, False).to(DEV)
        want = F.fp8moe_add_rmsnorm_fwd(x2, w2, r2)
        stream = r2.clone()
        got = F.fp8moe_add_rmsnorm_fwd(x2, w2, stream, h=stream)
        assert got[0] is stream and torch.equal(stream, want[0]) and torch.equal(got[1], want[1])


def test_extremes(F):
    """Rows of zeros, of the type's largest value (the squares overflow: the
    root is 0), and a NaN that stays in its row."""
    H = 512
    x = _bf16((4, H), 1)
    x[0] = 0
    x[1] = torch.finfo(torch.bfloat16).max
    x[2, 5] = float("nan")
    _, y, rstd, q, s = F.fp8moe_add_rmsnorm_fwd(x.to(DEV), torch.ones(H, device=DEV), eps=EPS, recipe=F.MXFP8)
    assert not y[:2].any() and torch.isnan(y[2]).all() and torch.isfinite(y[3]).all()
    assert float(rstd[0]) == pytest.approx(EPS ** -0.5, rel=1e-6) and float(rstd[1]) == 0.0
    assert not q[:2].any() and not s[:2].any()


@pytest.mark.parametrize("T,H", [(1, 8), (2, 32), (40, 256), (33, 2056), (300, 5120), (7, 7168), (5, 16384), (3, 16392),
                                 (1500, 512)])
@pytest.mark.parametrize("stream,w32", [(True, False), (False, True)])
def test_backward(F, T, H, stream, w32):
    h, dy, w = _bf16((T, H), H + T), _bf16((T, H), H + T + 1), _weight(H, 9, w32)
    dh = _bf16((T, H), H + T + 2) if stream else None
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dw = F.fp8moe_add_rmsnorm_bwd(dy.to(DEV), h.to(DEV), rstd.to(DEV), w.to(DEV), None if dh is None else dh.to(DEV))
    rdx, rdw = OM.add_rmsnorm_grad(_np(dy), _np(h), _np(rstd), _np(w), None if dh is None else _np(dh))
    xh, g = _np(h) * _np(rstd)[:, None], _np(dy) * _np(w)
    size = _np(rstd)[:, None] * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    check_bf16(dx, rdx, GREL * size + 2.0 ** -22 * (0 if dh is None else np.abs(_np(dh))), "dx")
    _near(_np(dw), rdw, GREL * np.abs(_np(dy) * xh).sum(0), "dw")


@pytest.mark.parametrize("T,H", [(77, 264), (201, 904), (1303, 1568), (31, 2048), (613, 448)])
@pytest.mark.parametrize("stream,w32", [(True, True), (True, False), (False, True), (False, False)])
def test_backward_short_rows(F, T, H, stream, w32):
    """Rows of a few warps, several to a CTA, in every form of the inputs."""
    test_backward(F, T, H, stream, w32)


def test_backward_in_place_and_same_bits(F):
    """dx may be dy or dh; two calls give the same bits; a dirty workspace does not matter."""
    T, H = 3000, 1024
    h, dy, dh = (_bf16((T, H), s).to(DEV) for s in (1, 2, 3))
    w = _weight(H, 4, True).to(DEV)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    ws = torch.full((F.fp8moe_add_rmsnorm_bwd_workspace_bytes(T, H) // 4,), float("nan"), device=DEV)
    dx, dw = F.fp8moe_add_rmsnorm_bwd(dy, h, rstd, w, dh, workspace=ws)
    d1, s1 = dy.clone(), dh.clone()
    a = F.fp8moe_add_rmsnorm_bwd(d1, h, rstd, w, dh, dx=d1)
    b = F.fp8moe_add_rmsnorm_bwd(dy, h, rstd, w, s1, dx=s1)
    for o in (a, b):
        assert torch.equal(o[0], dx) and torch.equal(o[1], dw)


def test_no_rows(F):
    w = torch.ones(64, device=DEV)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    h, y, rstd, q, s = F.fp8moe_add_rmsnorm_fwd(e, w, e, recipe=F.MXFP8)
    assert h.shape == y.shape == q.shape == (0, 64) and s.shape == (0, 2)
    dx, dw = F.fp8moe_add_rmsnorm_bwd(e, e, rstd, w)
    assert dx.shape == (0, 64) and not dw.any()


def test_gradient_against_differences(F):
    """The backward kernel against differences of the forward kernel's rows in
    directions, on a step large enough for fp32: <y(x + s d) - y(x - s d), dy>
    / 2s.  The forward's y is taken before its bf16 rounding through the rowwise
    path's exact inverse: here through rstd, y = a * rstd * w in float64."""
    T, H, step = 4, 256, 2.0 ** -4
    x, w, dy = _bf16((T, H), 1), _weight(H, 2, True), _bf16((T, H), 3)
    d = torch.sign(_bf16((T, H), 4)).to(torch.bfloat16)

    def value(v):
        rstd = F.fp8moe_add_rmsnorm_fwd(v.to(DEV), w.to(DEV), eps=EPS, need_y=False)[2]
        return (_np(v) * _np(rstd)[:, None] * _np(w) * _np(dy)).sum(1)

    x = (x * 16).round() / 16   # so that x + s d is exact in bf16
    x = x.clamp(-3, 3).to(torch.bfloat16)
    plus, minus = (x.float() + step * d.float()).to(torch.bfloat16), (x.float() - step * d.float()).to(torch.bfloat16)
    assert torch.equal(plus.float() - x.float(), step * d.float())
    num = (value(plus) - value(minus)) / (2 * step)
    rstd = F.fp8moe_add_rmsnorm_fwd(x.to(DEV), w.to(DEV), eps=EPS, need_y=False)[2]
    dx, _ = F.fp8moe_add_rmsnorm_bwd(dy.to(DEV), x.to(DEV), rstd, w.to(DEV))
    got = (_np(dx) * _np(d)).sum(1)
    # bf16 rounding of dx (2^-8 each at most, of both signs: half of that over
    # a row) and the third-order term of the step
    # (s^2 / 6 of a third derivative below 6 sum|dy w| for unit rows)
    lim = 2.0 ** -9 * np.abs(_np(dx)).sum(1) + step ** 2 * np.abs(_np(dy) * _np(w)).sum(1)
    assert np.all(np.abs(got - num) <= lim)


def test_other_stream(F):
    """Inputs made on one stream, the call on another: ordered by the caller's
    wait alone, its own allocations included."""
    T, H = 4096, 1024
    x, r, w = _bf16((T, H), 1).to(DEV), _bf16((T, H), 2).to(DEV), _weight(H, 3, True).to(DEV)
    want = F.fp8moe_add_rmsnorm_fwd(x, w, r, recipe=F.MXFP8, scale_layout=F.NO_GROUPS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.fp8moe_add_rmsnorm_fwd(x, w, r, recipe=F.MXFP8, scale_layout=F.NO_GROUPS, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert F.fp8moe_get_device_status() == 0


def test_ring_wait_timeout_sets_status(F):
    """A block of rows that never arrives: the bounded wait runs out, the status
    says so, and the next call in the same context is exact."""
    T, H = 3000, 1024
    h, dy = _bf16((T, H), 1).to(DEV), _bf16((T, H), 2).to(DEV)
    w, rstd = _weight(H, 3, False).to(DEV), torch.ones(T, device=DEV)
    want = F.fp8moe_add_rmsnorm_bwd(dy, h, rstd, w)
    F.fp8moe_testing_stall_next_quant_ring()
    F.fp8moe_add_rmsnorm_bwd(dy, h, rstd, w)
    assert F.fp8moe_get_device_status() == 6
    got = F.fp8moe_add_rmsnorm_bwd(dy, h, rstd, w)
    assert F.fp8moe_get_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
