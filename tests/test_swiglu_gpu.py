"""The gated activation with MXFP8 output and its backward against the float64
definition.

Tolerances: exp, the division and the products of one value take below 8 ulp
together: 1e-6 of the terms that are added (for the gate's gradient |d u sig|
(1 + |g| (1 - sig))).  bf16 outputs lie between the roundings of the two ends."""
import numpy as np
import pytest
import torch

from code_bounds import check_bf16, check_mx
from oracle import grouped_mm as OG, moe_ops as OM, quant as OQ, swizzle as OS

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 1e-6


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


def _ref(h, dout):
    """(values, tolerance) of the forward (dout None) or the backward."""
    if dout is None:
        v = OM.swiglu(_np(h))
        return v, REL * np.abs(v) + 1e-37
    v = OM.swiglu_grad(_np(dout), _np(h))
    g, u = np.split(_np(h), 2, axis=1)
    d, s = np.abs(_np(dout)), OM._sig(g)
    size = np.concatenate([d * np.abs(u) * s * (1 + np.abs(g) * (1 - s)), d * np.abs(g) * s], axis=1)
    return v, REL * size + 1e-37


def _offs(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32)


def _check(F, h, dout, offs, s0_layout, s1_layout, dim1, ldh=None):
    hd = h.to(DEV)
    if ldh is not None:
        wide = torch.full((h.shape[0], ldh), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :h.shape[1]] = hd
        hd = wide[:, :h.shape[1]]
    od = None if offs is None else offs.to(DEV)
    kw = dict(s0_layout=s0_layout, s1_layout=s1_layout, dim0=True, dim1=dim1)
    if dout is None:
        out, q0, s0, q1, s1 = F.fp8moe_swiglu_fwd(hd, od, **kw)
    else:
        out, q0, s0, q1, s1 = F.fp8moe_swiglu_bwd(dout.to(DEV), hd, od, **kw)
    v, tol = _ref(h, dout)
    M, W = v.shape
    check_bf16(out, v, tol, "bf16")
    on = None if offs is None else offs.numpy()

    def rowmajor(s, layout, rows, cols):
        """The real bytes of a scale buffer, and that the others are zero."""
        s = s.cpu().numpy()
        if layout == F.SCALES_ROWMAJOR:
            return s.reshape(rows, cols)
        E = 0 if layout == F.NO_GROUPS else len(on)
        rp, cp = OS.swizzled_shape(rows, cols, E, layout)
        assert s.size == rp * cp
        where = OS.swizzle(np.arange(1, rows * cols + 1, dtype=np.int64).astype(np.uint8).reshape(rows, cols) * 0 + 1,
                           on, layout)
        assert not s[where == 0].any(), "padding"
        full = OS.unswizzle(s, rp, cp)
        live = OS.unswizzle(where, rp, cp).astype(bool)
        return full[live].reshape(rows, cols)

    check_mx(q0.cpu().numpy(), rowmajor(s0, s0_layout, M, W // 32), v, tol, "dim0")
    if dim1:
        check_mx(q1.cpu().numpy(), rowmajor(s1, s1_layout, W, M // 32), v.T, tol.T, "dim1")
    assert F.fp8moe_get_device_status() == 0
    return out, q0, s0, q1, s1


@pytest.mark.parametrize("M,Fd", [(1, 32), (7, 96), (33, 64), (200, 160)])
@pytest.mark.parametrize("bwd", [False, True])
def test_rows_alone(F, M, Fd, bwd):
    """Any number of rows where the column direction is not asked for."""
    h, dout = _bf16((M, 2 * Fd), M, 2.0), _bf16((M, Fd), M + 1) if bwd else None
    for layout in (F.SCALES_ROWMAJOR, F.NO_GROUPS):
        _check(F, h, dout, None, layout, F.NO_GROUPS, False)
    _check(F, h, dout, None, F.NO_GROUPS, F.NO_GROUPS, False, ldh=2 * Fd + 40)


@pytest.mark.parametrize("sizes", [[32], [0, 64, 0, 32], [128, 32, 0, 160, 96, 0], [32] * 70, [0] * 40 + [256],
                                   [96, 0] * 300])
@pytest.mark.parametrize("bwd", [False, True])
def test_groups(F, sizes, bwd):
    M, Fd = sum(sizes), 96 if sum(sizes) < 9000 else 32
    h, dout = _bf16((M, 2 * Fd), M, 2.0), _bf16((M, Fd), M + 1) if bwd else None
    offs = _offs(sizes)
    _check(F, h, dout, offs, F.GROUP_ROWS, F.GROUP_COLS, True)
    if len(sizes) == 6:
        _check(F, h, dout, offs, F.NO_GROUPS, F.GROUP_COLS, True)
        _check(F, h, dout, offs, F.GROUP_ROWS, F.SCALES_ROWMAJOR, True)
        _check(F, h, dout, None, F.SCALES_ROWMAJOR, F.NO_GROUPS, True)


@pytest.mark.parametrize("bwd", [False, True])
def test_many_tiles(F, bwd):
    """More tiles than CTAs: every CTA walks several, across row blocks and
    groups, with ragged last row blocks and a last column tile of half width."""
    for M, Fd, sizes in ((9824, 416, [32, 0, 4000, 96, 5696]), (20001, 160, None), (70016, 64, [64] * 1000 + [6016])):
        h, dout = _bf16((M, 2 * Fd), M, 2.0), _bf16((M, Fd), M + 1) if bwd else None
        offs = None if sizes is None else _offs(sizes)
        if sizes is None:
            _check(F, h, dout, None, F.NO_GROUPS, F.NO_GROUPS, False, ldh=2 * Fd + 8)
        else:
            _check(F, h, dout, offs, F.GROUP_ROWS, F.GROUP_COLS, True)


def test_invalid_offsets_with_many_tiles(F):
    M, Fd = 20480, 256
    h = _bf16((M, 2 * Fd), 1).to(DEV)
    offs = torch.tensor([64, 32, M], dtype=torch.int32, device=DEV)
    q0 = torch.full((M, Fd), 0xA5, dtype=torch.uint8, device=DEV)
    F.fp8moe_swiglu_fwd(h, offs, F.GROUP_ROWS, need_out=False, dim0=True, q0=q0)
    assert F.fp8moe_get_device_status() == 5 and bool((q0 == 0xA5).all())


@pytest.mark.parametrize("bwd", [False, True])
def test_each_output_alone(F, bwd):
    M, Fd = 160, 64
    h, dout = _bf16((M, 2 * Fd), 1).to(DEV), _bf16((M, Fd), 2).to(DEV)
    call = (lambda **k: F.fp8moe_swiglu_bwd(dout, h, **k)) if bwd else (lambda **k: F.fp8moe_swiglu_fwd(h, **k))
    need = "need_dh" if bwd else "need_out"
    out, q0, s0, q1, s1 = call(dim0=True, dim1=True)
    a = call()
    assert torch.equal(a[0], out) and a[1:] == (None,) * 4
    b = call(dim0=True, **{need: False})
    assert b[0] is None and torch.equal(b[1], q0) and torch.equal(b[2], s0) and b[3:] == (None, None)
    c = call(dim1=True, **{need: False})
    assert c[:3] == (None,) * 3 and torch.equal(c[3], q1) and torch.equal(c[4], s1)


def test_extremes(F):
    """Gates far out on both sides, zeros, zero padding rows (scale byte 0)."""
    h = torch.zeros(64, 128, dtype=torch.bfloat16)
    h[0, :64] = torch.linspace(-200, 200, 64).to(torch.bfloat16)
    h[0, 64:] = 1.0
    h[1, :64], h[1, 64:] = -3e38, 1.0
    h[2, :64], h[2, 64:] = 1e4, -1e4
    _check(F, h, None, None, F.NO_GROUPS, F.NO_GROUPS, True)
    _check(F, h, torch.ones(64, 64, dtype=torch.bfloat16), None, F.NO_GROUPS, F.NO_GROUPS, True)
    _, q0, s0, _, _ = F.fp8moe_swiglu_fwd(h.to(DEV), dim0=True, s0_layout=F.SCALES_ROWMAJOR)
    assert not q0[3:].any() and not s0[3:].any()


def test_invalid_offsets(F):
    """The status is set and nothing is written."""
    M, Fd = 96, 64
    h = _bf16((M, 2 * Fd), 1).to(DEV)
    for bad in ([32, 64, 64], [32, 0, 96], [16, 32, 96], [32, 128, 96], [-32, 32, 96]):
        offs = torch.tensor(bad, dtype=torch.int32, device=DEV)
        q0 = torch.full((M, Fd), 0xA5, dtype=torch.uint8, device=DEV)
        q1 = torch.full((Fd, M), 0xA5, dtype=torch.uint8, device=DEV)
        F.fp8moe_swiglu_fwd(h, offs, F.GROUP_ROWS, F.GROUP_COLS, need_out=False, dim0=True, dim1=True, q0=q0, q1=q1)
        assert F.fp8moe_get_device_status() == 5
        assert bool((q0 == 0xA5).all()) and bool((q1 == 0xA5).all())
    assert F.fp8moe_get_device_status() == 0


def test_feeds_the_grouped_products(F):
    """The outputs are the operands of the second product (forward), and of
    both products of the first one's backward, as they come."""
    sizes, Fd, K = [64, 0, 96, 32], 128, 64
    M, E = sum(sizes), len(sizes)
    offs = _offs(sizes)
    od = offs.to(DEV)
    h, dout = _bf16((M, 2 * Fd), 1), _bf16((M, Fd), 2)
    deq = lambda q, s: OQ.dequant_mx(q, s)
    v, _ = _ref(h, None)
    w2 = _bf16((E, K, Fd), 3, 0.1)
    _, q0, s0, q1, s1 = F.fp8moe_swiglu_fwd(h.to(DEV), od, F.GROUP_ROWS, F.GROUP_COLS, dim0=True, dim1=True)
    qw, sw, _, _ = F.fp8moe_mxfp8_quantize_dual(w2.to(DEV), None, F.NO_GROUPS, F.NO_GROUPS, dim1=False)
    y = F.fp8moe_scaled_grouped_mm_fwd(F.MXFP8, q0, s0, qw, sw, od)
    ref, bound = OG.grouped_mm_fwd(deq(*OQ.mxfp8_quantize_dim0(v)), deq(*OQ.mxfp8_quantize_dim0(_np(w2))), offs.numpy())
    # 2^-3 of a code may change where fp32 and float64 round apart: one in a few thousand values
    assert np.all(np.abs(_np(y) - ref) <= 8e-3 * np.abs(ref) + 2e-3 * bound)
    dy = _bf16((M, K), 4)
    _, _, qt, st = F.fp8moe_mxfp8_quantize_dual(dy.to(DEV), od, F.GROUP_ROWS, F.GROUP_COLS)
    dw2 = F.fp8moe_scaled_grouped_mm_wgrad(F.MXFP8, qt, st, q1, s1, od, M)
    ref, bound = OG.grouped_mm_wgrad(deq(*OQ.mxfp8_quantize_dim1(_np(dy))), deq(*OQ.mxfp8_quantize_dim1(v)), offs.numpy())
    assert np.all(np.abs(_np(dw2) - ref) <= 8e-3 * np.abs(ref) + 2e-3 * bound)
    g, _ = _ref(h, dout)
    w1 = _bf16((E, 2 * Fd, K), 5, 0.1)
    _, d0, t0, d1, t1 = F.fp8moe_swiglu_bwd(dout.to(DEV), h.to(DEV), od, F.GROUP_ROWS, F.GROUP_COLS, dim0=True, dim1=True)
    _, _, qwt, swt = F.fp8moe_mxfp8_quantize_dual(w1.to(DEV), None, F.NO_GROUPS, F.NO_GROUPS)
    dx = F.fp8moe_scaled_grouped_mm_dgrad(F.MXFP8, d0, t0, qwt, swt, od)
    ref, bound = OG.grouped_mm_dgrad(deq(*OQ.mxfp8_quantize_dim0(g)), deq(*OQ.mxfp8_quantize_dim1(_np(w1))), offs.numpy())
    assert np.all(np.abs(_np(dx) - ref) <= 8e-3 * np.abs(ref) + 2e-3 * bound)
    x = _bf16((M, K), 6)
    _, _, xt, xs = F.fp8moe_mxfp8_quantize_dual(x.to(DEV), od, F.GROUP_ROWS, F.GROUP_COLS)
    dw1 = F.fp8moe_scaled_grouped_mm_wgrad(F.MXFP8, d1, t1, xt, xs, od, M)
    ref, bound = OG.grouped_mm_wgrad(deq(*OQ.mxfp8_quantize_dim1(g)), deq(*OQ.mxfp8_quantize_dim1(_np(x))), offs.numpy())
    assert np.all(np.abs(_np(dw1) - ref) <= 8e-3 * np.abs(ref) + 2e-3 * bound)
    assert F.fp8moe_get_device_status() == 0


def test_gradient_against_differences(F):
    """<a(h + s d) - a(h - s d), dout> / 2s of the forward kernel's bf16 result
    against the backward kernel's, summed over a row.  The roundings to bf16 are
    2^-8 each at most, of both signs: half of that over a row; the third derivative of g sig(g) u along unit directions is
    below 2 (1 + |u|), so the quotient is off by at most s^2 / 3 (1 + |u|)."""
    M, Fd, step = 32, 64, 0.25
    g = torch.Generator().manual_seed(3)
    h = (torch.randint(-12, 13, (M, 2 * Fd), generator=g) / 4).to(torch.bfloat16)
    d = (torch.randint(0, 2, (M, 2 * Fd), generator=g) * 2 - 1).to(torch.bfloat16)
    dout = _bf16((M, Fd), 4)
    value = lambda t: _np(F.fp8moe_swiglu_fwd(t.to(DEV))[0])
    plus, minus = (h.float() + step * d.float()).to(torch.bfloat16), (h.float() - step * d.float()).to(torch.bfloat16)
    vp, vm = value(plus), value(minus)
    num = ((vp - vm) * _np(dout)).sum(1) / (2 * step)
    dh = _np(F.fp8moe_swiglu_bwd(dout.to(DEV), h.to(DEV))[0])
    got = (dh * _np(d)).sum(1)
    u = np.abs(_np(h)[:, Fd:])
    lim = (2.0 ** -9 * ((np.abs(vp) + np.abs(vm)) * np.abs(_np(dout))).sum(1) / (2 * step)
           + 2.0 ** -9 * np.abs(dh).sum(1) + step ** 2 / 3 * ((1 + u) * np.abs(_np(dout))).sum(1))
    assert np.all(np.abs(got - num) <= lim)


def test_no_rows(F):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    out, q0, s0, q1, s1 = F.fp8moe_swiglu_fwd(e, dim0=True, dim1=True)
    assert out.shape == (0, 32) and q0.shape == (0, 32) and q1.shape == (32, 0)


@pytest.mark.parametrize("bwd", [False, True])
def test_load_wait_timeout_sets_status(F, bwd):
    """A tile that never arrives: the bounded wait runs out, the status says so,
    and the next call in the same context is exact."""
    M, Fd = 8192, 512
    h, dout = _bf16((M, 2 * Fd), 1).to(DEV), _bf16((M, Fd), 2).to(DEV)
    call = (lambda: F.fp8moe_swiglu_bwd(dout, h, dim0=True, dim1=True)) if bwd else (
        lambda: F.fp8moe_swiglu_fwd(h, dim0=True, dim1=True))
    want = call()
    F.fp8moe_testing_stall_next_quant_ring()
    call()
    assert F.fp8moe_get_device_status() == 6
    got = call()
    assert F.fp8moe_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
