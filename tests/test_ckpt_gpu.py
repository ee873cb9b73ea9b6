"""Backward passes from activations kept as MXFP8, and the forward that writes them.

Three references: the definitions in 64 bits on the values that the codes stand
for; the calls on bf16 activations, given those values as bf16 (which hold them
exactly), with the same bits where the arithmetic is the same; and the quantizer,
for the checkpoint itself.

Tolerances as in the tests of the bf16 calls.  A weight gradient's sum of N
products is added by at most N / 16 and 8 joins a lane, each off by 2^-24 of the
magnitudes so far."""
import numpy as np
import pytest
import torch

from code_bounds import check_bf16, check_mx
from oracle import moe_ops as OM, quant as OQ, swizzle as OS

pytestmark = pytest.mark.gpu
DEV = "cuda"


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


def _pack(x):
    """(codes, scales) on the device and the values, as bf16, of x [R, C]."""
    q, s = OQ.mxfp8_quantize_dim0(_np(x))
    v = OQ.dequant_mx(q, s)
    b = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)
    assert np.array_equal(_np(b), v)
    return torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), b


def _same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def _offs(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device=DEV)


# --- gated activation, forward ----------------------------------------------------

@pytest.mark.parametrize("M,Fd,ld", [(1, 32, 0), (7, 96, 0), (33, 64, 40), (200, 160, 8), (9824, 416, 0), (20001, 160, 8)])
def test_forward_checkpoint(F, M, Fd, ld):
    """The checkpoint is the quantizer's, the other outputs the plain call's."""
    h = _bf16((M, 2 * Fd), M, 2.0)
    h[::7] *= 2.0 ** -20
    h[M // 2] = 0.0
    wide = torch.full((M, 2 * Fd + ld), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :2 * Fd] = h.to(DEV)
    hd = wide[:, :2 * Fd]
    rows = M % 32 == 0
    for kw in (dict(dim0=True, dim1=rows), dict(need_out=False, dim0=True, s0_layout=F.SCALES_ROWMAJOR), dict(need_out=False)):
        *out, hq, hs = F.fp8moe_swiglu_fwd_ckpt(hd, **kw)
        if kw != dict(need_out=False):
            _same(out, F.fp8moe_swiglu_fwd(hd, **kw))
        else:
            assert out == [None] * 5
        _same((hq, hs), F.fp8moe_mxfp8_quantize_dim0(h.to(DEV)))
        if M < 1000:
            q, s = OQ.mxfp8_quantize_dim0(_np(h))
            assert np.array_equal(hq.cpu().numpy(), q) and np.array_equal(hs.cpu().numpy(), s)
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.parametrize("M,Fd", [(64, 64), (8192, 512)])
def test_forward_groups_and_not_finite(F, M, Fd):
    h = _bf16((M, 2 * Fd), 3, 2.0)
    h[5, 3], h[6, Fd + 2], h[9, 40], h[11, 0] = float("nan"), float("inf"), -float("inf"), -300.0
    hd, offs = h.to(DEV), _offs([32, 0, M - 32])
    lay = (F.GROUP_ROWS, F.GROUP_COLS)
    *out, hq, hs = F.fp8moe_swiglu_fwd_ckpt(hd, offs, *lay, dim0=True, dim1=True)
    _same(out, F.fp8moe_swiglu_fwd(hd, offs, *lay, dim0=True, dim1=True))
    _same((hq, hs), F.fp8moe_mxfp8_quantize_dim0(hd))


# --- gated activation, backward ---------------------------------------------------

def _bwd_ref(dout, v):
    """(gradients, their tolerance, activation, its tolerance)."""
    g, u = np.split(v, 2, axis=1)
    d, s = np.abs(_np(dout)), OM._sig(g)
    size = np.concatenate([d * np.abs(u) * s * (1 + np.abs(g) * (1 - s)), d * np.abs(g) * s], axis=1)
    a = OM.swiglu(v)
    return OM.swiglu_grad(_np(dout), v), 1e-6 * size + 1e-37, a, 1e-6 * np.abs(a) + 1e-37


def _columns(F, s, layout, rows, cols, offs):
    s = s.cpu().numpy()
    if layout == F.SCALES_ROWMAJOR:
        return s.reshape(rows, cols)
    rp, cp = OS.swizzled_shape(rows, cols, 0 if offs is None else len(offs), layout)
    where = OS.swizzle(np.ones((rows, cols), np.uint8), offs, layout)
    assert s.size == rp * cp and not s[where == 0].any()
    return OS.unswizzle(s, rp, cp)[OS.unswizzle(where, rp, cp).astype(bool)].reshape(rows, cols)


@pytest.mark.parametrize("sizes,Fd", [([32], 32), ([0, 64, 0, 32], 96), ([128, 32, 0, 160, 96, 0], 64), ([96, 0] * 20, 160),
                                      ([4000, 0, 96, 5696 + 32], 416)])
def test_backward(F, sizes, Fd):
    M = sum(sizes)
    hq, hs, v = _pack(_bf16((M, 2 * Fd), M, 2.0))
    dout, offs = _bf16((M, Fd), M + 1), _offs(sizes)
    dd, vd = dout.to(DEV), v.to(DEV)
    on = offs.cpu().numpy()
    ref, tol, act, atol = _bwd_ref(dout, _np(v))
    for l0, l1, o in ((F.GROUP_ROWS, F.GROUP_COLS, offs), (F.NO_GROUPS, F.SCALES_ROWMAJOR, None), (F.SCALES_ROWMAJOR, F.NO_GROUPS, None)):
        *out, aq1, as1 = F.fp8moe_swiglu_bwd_ckpt(dd, hq, hs, o, l0, l1, dim0=True, dim1=True, act1=True)
        _same(out, F.fp8moe_swiglu_bwd(dd, vd, o, l0, l1, dim0=True, dim1=True))
        _same((aq1, as1), F.fp8moe_swiglu_fwd(vd, o, s1_layout=l1, need_out=False, dim1=True)[3:])
        check_bf16(out[0], ref, tol, "dh")
        check_mx(aq1.cpu().numpy(), _columns(F, as1, l1, Fd, M // 32, on if o is not None else None), act.T, atol.T, "act")
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.parametrize("M,Fd", [(1, 32), (7, 96), (33, 64), (200, 160), (20001, 160)])
def test_backward_any_rows(F, M, Fd):
    hq, hs, v = _pack(_bf16((M, 2 * Fd), M, 2.0))
    dout = _bf16((M, Fd), M + 1)
    for layout in (F.SCALES_ROWMAJOR, F.NO_GROUPS):
        out = F.fp8moe_swiglu_bwd_ckpt(dout.to(DEV), hq, hs, s0_layout=layout, dim0=True)
        _same(out[:5], F.fp8moe_swiglu_bwd(dout.to(DEV), v.to(DEV), s0_layout=layout, dim0=True))
    ref, tol, _, _ = _bwd_ref(dout, _np(v))
    check_bf16(out[0], ref, tol, "dh")


@pytest.mark.parametrize("M,Fd", [(160, 64), (9824, 416)])
def test_backward_each_output_alone(F, M, Fd):
    hq, hs, _ = _pack(_bf16((M, 2 * Fd), 1))
    dout = _bf16((M, Fd), 2).to(DEV)
    call = lambda **k: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, **k)
    full = call(dim0=True, dim1=True, act1=True)
    _same(call(), full[:1] + (None,) * 6)
    _same(call(need_dh=False, dim0=True), (None,) + full[1:3] + (None,) * 4)
    _same(call(need_dh=False, dim1=True), (None,) * 3 + full[3:5] + (None,) * 2)
    _same(call(need_dh=False, act1=True), (None,) * 5 + full[5:])


@pytest.mark.parametrize("M,Fd", [(64, 64), (8192, 320)])
def test_backward_far_and_not_finite(F, M, Fd):
    """Gates beyond fp32's exponential, products beyond fp32, NaN codes and
    scales, tiny blocks: the bf16 call's results on the same values."""
    h = _bf16((M, 2 * Fd), 3, 2.0)
    h[0, :32], h[1, Fd:Fd + 32], h[2, :64] = -300.0, 3e38, -2e38
    h[3] *= 2.0 ** -100
    hq, hs, v = _pack(h)
    hq[7, 5], hs[8, 1] = 0x7F, 255
    v[7, 5] = float("nan")
    v[8, 32:64] = float("nan")
    dout = _bf16((M, Fd), 4).to(DEV)
    dout[1] *= 1e4
    got = F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, dim0=True, dim1=True, act1=True)
    want = F.fp8moe_swiglu_bwd(dout, v.to(DEV), dim0=True, dim1=True) + F.fp8moe_swiglu_fwd(v.to(DEV), need_out=False, dim1=True)[3:]
    for a, b in zip(got, want):
        if a.dtype == torch.bfloat16:
            assert torch.equal(torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0))
        else:   # (a NaN's sign is not told)
            assert torch.equal(a, b) or torch.equal(a & 0x7F, b & 0x7F)


@pytest.mark.parametrize("M,Fd", [(96, 64), (20480, 256)])
def test_backward_invalid_offsets(F, M, Fd):
    hq, hs = torch.zeros(M, 2 * Fd, dtype=torch.uint8, device=DEV), torch.zeros(M, Fd // 16, dtype=torch.uint8, device=DEV)
    dout = torch.zeros(M, Fd, dtype=torch.bfloat16, device=DEV)
    for bad in ([32, 64, 64], [64, 32, M], [16, 32, M]):
        aq1 = torch.full((Fd, M), 0xA5, dtype=torch.uint8, device=DEV)
        F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, torch.tensor(bad, dtype=torch.int32, device=DEV), F.NO_GROUPS, F.GROUP_COLS,
                                 need_dh=False, act1=True, aq1=aq1)
        assert F.fp8moe_get_device_status() == 5 and bool((aq1 == 0xA5).all())
    assert F.fp8moe_get_device_status() == 0


def test_no_rows(F):
    e8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)
    e = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)
    out = F.fp8moe_swiglu_bwd_ckpt(e, e8(0, 64), e8(0, 2), dim0=True, dim1=True, act1=True)
    assert out[0].shape == (0, 64) and out[5].shape == (32, 0)
    out = F.fp8moe_swiglu_fwd_ckpt(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert out[5].shape == (0, 64) and out[6].shape == (0, 2)
    w = torch.ones(64, device=DEV)
    dx, dw = F.fp8moe_add_rmsnorm_bwd_ckpt(e.new_empty(0, 64), e8(0, 64), e8(0, 2), torch.empty(0, device=DEV), w)
    assert dx.shape == (0, 64) and not dw.any()
    z = F.fp8moe_route_weight_grad_ckpt(e, e8(4, 32), e8(4, 1), torch.empty(0, 3, dtype=torch.int32, device=DEV))
    assert z.shape == (0, 3)


@pytest.mark.parametrize("what", ["fwd", "norm", "decode"])
def test_wait_timeout_sets_status(F, what):
    """A tile that never arrives: the bounded waits run out, the status says so,
    and the next call in the same context is exact."""
    M, Fd = 8192, 512
    h = _bf16((M, 2 * Fd), 1).to(DEV)
    hq, hs = F.fp8moe_mxfp8_quantize_dim0(h)
    rstd, w = torch.ones(M, device=DEV), torch.ones(2 * Fd, device=DEV)
    wq, ws = hq[:2 * Fd].view(1, 2 * Fd, 2 * Fd), torch.full((4 * Fd * Fd // 32,), 120, dtype=torch.uint8, device=DEV)
    idx, one = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.ones(3, 1, device=DEV)
    call = {"fwd": lambda: F.fp8moe_swiglu_fwd_ckpt(h, dim0=True, dim1=True),
            "norm": lambda: F.fp8moe_add_rmsnorm_bwd_ckpt(h, hq, hs, rstd, w),
            "decode": lambda: (F.fp8moe_mxfp8_moe_decode(h[:3], idx, one, wq, ws, hq[:2 * Fd, :Fd].contiguous().view(1, 2 * Fd, Fd),
                                                         ws),)}[what]
    want = call()
    F.fp8moe_testing_stall_next_quant_ring()
    call()
    assert F.fp8moe_get_device_status() == 6
    got = call()
    assert F.fp8moe_get_device_status() == 0
    _same(got, want)


# --- norm backward ------------------------------------------------------------------

def _weight(H, seed, w32):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(H, generator=g) + 0.5
    return w if w32 else w.to(torch.bfloat16)


@pytest.mark.parametrize("T,H", [(1, 32), (3, 64), (5, 96), (301, 256), (700, 1056), (160, 2048), (33, 5120), (9, 7168), (17, 8224),
                                 (5, 16384), (4, 16416), (3001, 512)])
@pytest.mark.parametrize("stream,w32", [(False, False), (True, True), (True, False)])
def test_norm_backward(F, T, H, stream, w32):
    hq, hs, v = _pack(_bf16((T, H), T, 3.0))
    dy, w, dh = _bf16((T, H), T + 1), _weight(H, T, w32), _bf16((T, H), T + 2) if stream else None
    rstd = torch.from_numpy(OM.add_rmsnorm(_np(v), None, _np(w), 1e-5)[1].astype(np.float32))
    dd, rd, wd, sd = dy.to(DEV), rstd.to(DEV), w.to(DEV), None if dh is None else dh.to(DEV)
    dx, dw = F.fp8moe_add_rmsnorm_bwd_ckpt(dd, hq, hs, rd, wd, sd)
    rx, rw = OM.add_rmsnorm_grad(_np(dy), _np(v), _np(rstd), _np(w), None if dh is None else _np(dh))
    r = _np(rstd)[:, None]
    size = r * (np.abs(_np(dy) * _np(w)) + np.abs(_np(v) * r) * np.mean(np.abs(_np(dy) * _np(w) * _np(v) * r), axis=1, keepdims=True))
    check_bf16(dx, rx, 1e-6 * (size + (0 if dh is None else np.abs(_np(dh)))) + 1e-37, "dx")
    parts = np.abs(_np(dy) * _np(v) * r).sum(0)
    assert np.all(np.abs(_np(dw) - rw) <= (T / 8 + 32) * 2.0 ** -24 * parts + 1e-30)
    assert F.fp8moe_get_device_status() == 0


def test_norm_backward_in_place_any_workspace_same_bits(F):
    T, H = 700, 1024
    hq, hs, _ = _pack(_bf16((T, H), 1))
    dy, dh, w, rstd = _bf16((T, H), 2).to(DEV), _bf16((T, H), 3).to(DEV), _weight(H, 4, True).to(DEV), torch.rand(T, device=DEV) + 0.5
    want = F.fp8moe_add_rmsnorm_bwd_ckpt(dy, hq, hs, rstd, w, dh)
    ws = torch.full((F.fp8moe_add_rmsnorm_bwd_workspace_bytes(T, H) // 4,), float("nan"), device=DEV)
    d1, s1 = dy.clone(), dh.clone()
    _same(F.fp8moe_add_rmsnorm_bwd_ckpt(d1, hq, hs, rstd, w, dh, dx=d1, workspace=ws), want)
    _same(F.fp8moe_add_rmsnorm_bwd_ckpt(dy, hq, hs, rstd, w, s1, dx=s1), want)


# --- combine weight gradient ---------------------------------------------------------

@pytest.mark.parametrize("T,N,k", [(1, 32, 1), (3, 64, 2), (50, 7168, 8), (2503, 32, 3), (5000, 768, 5), (2503, 800, 6), (1301, 2048, 7),
                                   (1301, 2080, 1), (310, 8160, 4), (161, 8224, 8), (435, 480, 13), (77, 1280, 6)])
def test_weight_grad(F, T, N, k):
    """Missing rows, numbers past the last row, rows that no pair names hold NaN."""
    g = torch.Generator().manual_seed(N + T)
    rows = T * k + 9
    yq, ys, y = _pack(_bf16((rows, N), N))
    perm = torch.randperm(rows, generator=g)
    row_of = perm[:T * k].reshape(T, k).to(torch.int32)
    gone = torch.rand(T, k, generator=g) < 0.2
    yq[perm[T * k:].to(DEV)] = 0x7F
    yq[row_of[gone].long().to(DEV)], ys[row_of[gone].long().to(DEV)] = 0x7F, 255
    row_of[gone] = -1
    row_of[T // 2, k - 1] = rows
    dout = torch.randn(T, N, generator=g).to(torch.bfloat16)
    got = _np(F.fp8moe_route_weight_grad_ckpt(dout.to(DEV), yq, ys, row_of.to(DEV)))
    r = np.where(row_of.numpy() < rows, row_of.numpy(), -1)
    yn = _np(y)
    ref, size = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        rows_j = yn[np.maximum(r[:, j], 0)]
        ref[:, j] = (_np(dout) * rows_j).sum(1) * (r[:, j] >= 0)
        size[:, j] = np.abs(_np(dout) * rows_j).sum(1)
    assert np.all(np.abs(got - ref) <= (N / 16 + 16) * 2.0 ** -24 * size) and not got[r < 0].any()


def test_weight_grad_no_rows_and_no_columns(F):
    dout = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    e8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)
    row_of = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    assert not F.fp8moe_route_weight_grad_ckpt(dout, e8(0, 64), e8(0, 2), row_of).any()
    assert not F.fp8moe_route_weight_grad_ckpt(dout[:, :0].contiguous(), e8(3, 0), e8(3, 0), row_of).any()


# --- captured ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [96, 20480])
def test_replayed(F, M):
    """Captured, then replayed on other contents: the bits of plain calls."""
    Fd = 128
    hq, hs, v = _pack(_bf16((M, 2 * Fd), 1))
    hq2, hs2, v2 = _pack(_bf16((M, 2 * Fd), 2))
    h, h2 = v.to(DEV), v2.to(DEV)
    dout = _bf16((M, Fd), 3).to(DEV)
    rstd, w = torch.rand(M, device=DEV) + 0.5, torch.rand(2 * Fd, device=DEV)
    row_of = torch.randperm(M, device=DEV).to(torch.int32).view(-1, 2)
    do = _bf16((M // 2, 2 * Fd), 4).to(DEV)
    lay = dict(s0_layout=F.SCALES_ROWMAJOR, s1_layout=F.SCALES_ROWMAJOR, dim0=True, dim1=True)
    calls = [lambda: F.fp8moe_swiglu_fwd_ckpt(h, **lay), lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, act1=True, **lay),
             lambda: F.fp8moe_add_rmsnorm_bwd_ckpt(h, hq, hs, rstd, w),
             lambda: (F.fp8moe_route_weight_grad_ckpt(do, hq, hs, row_of),)]
    for call in calls:
        first = call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for a, b, c in ((h2, hq2, hs2), (v.to(DEV), *_pack(v)[:2])):
            keep = [t.clone() for t in (h, hq, hs)]
            for t, n in zip((h, hq, hs), (a, b, c)):
                t.copy_(n)
            want = [None if t is None else t.clone() for t in call()]
            for t in out:
                if t is not None:
                    t.view(torch.uint8).fill_(0xA5)
            graph.replay()
            torch.cuda.synchronize()
            _same(out, want)
            for t, n in zip((h, hq, hs), keep):
                t.copy_(n)
        del first
