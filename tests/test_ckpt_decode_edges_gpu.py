"""The calls on MXFP8 checkpoints and the few tokens' expert layer at their edges:
they write inside their outputs and workspaces only, refuse tensors of the wrong
kind, run from two host threads and on other streams, and reach more row tiles
than a grid's second dimension holds."""
import threading

import pytest
import torch

from test_canaries_gpu import DEV, Guarded, _bf16

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _ckpt(R, C, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(0, 256, (R, C), generator=g, dtype=U8, device=DEV)
    q.masked_fill_((q & 0x7F) == 0x7F, 0)
    return q, torch.randint(115, 120, (R, C // 32), generator=g, dtype=U8, device=DEV)


def _layer(F, T, H, Fd, E, k, seed=0):
    """Arguments of the few tokens' layer."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF16)
    idx = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=I32)
    w = torch.rand(T, k, generator=g, device=DEV)
    out = [x, idx, w]
    for R, K in ((2 * Fd, H), (H, Fd)):
        q, _ = _ckpt(E * R, K, seed)
        n = F.fp8moe_swizzled_scales_bytes(E, R, K // 32, 0, F.NO_GROUPS)
        out += [q.view(E, R, K), torch.full((n,), 118, dtype=U8, device=DEV)]
    return out


# --- inside their outputs ---------------------------------------------------------

@pytest.mark.parametrize("M,Fd", [(32, 32), (160, 96), (9824, 416)])
def test_activation_canaries(F, M, Fd):
    g = Guarded()
    h, dout = _bf16((M, 2 * Fd), 1), _bf16((M, Fd), 2)
    hq, hs = _ckpt(M, 2 * Fd)
    offs = torch.tensor([0, 32, 32, M], dtype=I32, device=DEV)
    size = F.fp8moe_swizzled_scales_bytes
    lay = (F.GROUP_ROWS, F.GROUP_COLS)
    outs = lambda W: dict(out=g((M, W), BF16), q0=g((M, W), U8), q1=g((W, M), U8),
                          s0=g((size(1, M, W // 32, 4, F.GROUP_ROWS),), U8), s1=g((size(1, W, M // 32, 4, F.GROUP_COLS),), U8))
    F.fp8moe_swiglu_fwd_ckpt(h, offs, *lay, dim0=True, dim1=True, hq=g((M, 2 * Fd), U8), hs=g((M, Fd // 16), U8), **outs(Fd))
    F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, offs, *lay, dim0=True, dim1=True, act1=True, aq1=g((Fd, M), U8),
                             as1=g((size(1, Fd, M // 32, 4, F.GROUP_COLS),), U8), **outs(2 * Fd))
    n = M - 5   # a ragged last row block, rows alone
    F.fp8moe_swiglu_fwd_ckpt(h[:n], None, F.SCALES_ROWMAJOR, need_out=False, hq=g((n, 2 * Fd), U8), hs=g((n, Fd // 16), U8))
    F.fp8moe_swiglu_bwd_ckpt(dout[:n], hq[:n], hs[:n], None, F.SCALES_ROWMAJOR, dim0=True, out=g((n, 2 * Fd), BF16),
                             q0=g((n, 2 * Fd), U8), s0=g((n, Fd // 16), U8))
    g.check("gated activation with its checkpoint")
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.parametrize("T,H", [(1, 160), (77, 96), (700, 512), (130, 1056), (3, 2080), (5, 16416)])
def test_norm_and_weight_grad_canaries(F, T, H):
    g = Guarded()
    dy, dh = _bf16((T, H), 3), _bf16((T, H), 2)
    hq, hs = _ckpt(T, H)
    rstd, nws = torch.ones(T, device=DEV), F.fp8moe_add_rmsnorm_bwd_workspace_bytes(T, H)
    for w in (torch.ones(H, device=DEV), torch.ones(H, device=DEV, dtype=BF16)):
        for d in (None, dh):
            F.fp8moe_add_rmsnorm_bwd_ckpt(dy, hq, hs, rstd, w, d, dx=g((T, H), BF16), dweight=g((H,), F32),
                                          workspace=g((nws,), U8))
    for k in (1, 3, 8):
        F.fp8moe_route_weight_grad_ckpt(dy, hq, hs, torch.arange(T * k, device=DEV, dtype=I32).reshape(T, k) - 1,
                                        dw=g((T, k), F32))
    g.check("backward")


@pytest.mark.parametrize("T,H,Fd,E,k", [(1, 96, 160, 4, 3), (1, 32, 32, 1, 1), (3, 160, 96, 7, 2), (40, 352, 416, 9, 3)])
def test_decode_canaries(F, T, H, Fd, E, k):
    g = Guarded()
    n = F.fp8moe_mxfp8_moe_decode_workspace_bytes(T, k, E, H, Fd)
    F.fp8moe_mxfp8_moe_decode(*_layer(F, T, H, Fd, E, k), out=g((T, H), BF16), workspace=g((n,), U8))
    g.check("few tokens")
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.parametrize("M", [32, 3200])
def test_new_results_are_apart(F, M):
    h, dout = _bf16((M, 512), 1), _bf16((M, 256), 2)
    hq, hs = _ckpt(M, 512)
    for call in (lambda: F.fp8moe_swiglu_fwd_ckpt(h, dim0=True, dim1=True),
                 lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, dim0=True, dim1=True, act1=True)):
        got = call()
        assert len(got) == 7 and all(t is not None for t in got)
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in got)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in got)


# --- refused ----------------------------------------------------------------------------

def test_refusals(F):
    M, Fd, H = 64, 64, 128
    h, dout = _bf16((M, 2 * Fd), 1), _bf16((M, Fd), 2)
    hq, hs = _ckpt(M, 2 * Fd)
    rstd, w = torch.ones(M, device=DEV), torch.ones(H, device=DEV)
    row_of = torch.zeros(M, 2, dtype=I32, device=DEV)
    x, idx, tw, w1, s1, w2, s2 = _layer(F, 4, 64, 96, 5, 2)
    offs = torch.tensor([32, M], dtype=I32, device=DEV)
    bad = [
        lambda: F.fp8moe_swiglu_fwd_ckpt(h.float()),
        lambda: F.fp8moe_swiglu_fwd_ckpt(h[:, :96]),
        lambda: F.fp8moe_swiglu_fwd_ckpt(h.cpu()),
        lambda: F.fp8moe_swiglu_fwd_ckpt(h, hq=hq[:32]),
        lambda: F.fp8moe_swiglu_fwd_ckpt(h, hs=hs.to(torch.int8)),
        lambda: F.fp8moe_swiglu_fwd_ckpt(h, offs, F.GROUP_COLS, dim0=True),
        lambda: F.fp8moe_swiglu_fwd_ckpt(h[:40], dim1=True),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq.to(torch.int8), hs),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs[:, :2]),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs.cpu()),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq.t().contiguous().t(), hs),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout.float(), hq, hs),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, need_dh=False),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout[:40], hq[:40], hs[:40], act1=True),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, act1=True, aq1=hq),
        lambda: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, None, F.GROUP_ROWS, dim0=True),
        lambda: F.fp8moe_add_rmsnorm_bwd_ckpt(h, hq, None, rstd, w),
        lambda: F.fp8moe_add_rmsnorm_bwd_ckpt(h, h, hs, rstd, w),
        lambda: F.fp8moe_add_rmsnorm_bwd_ckpt(h, hq, hs[:, :3], rstd, w),
        lambda: F.fp8moe_add_rmsnorm_bwd_ckpt(h[:, :120].contiguous(), hq[:, :120].contiguous(), hs[:, :3].contiguous(), rstd,
                                              w[:120]),
        lambda: F.fp8moe_add_rmsnorm_bwd_ckpt(h, hq, hs, rstd, w, workspace=torch.empty(16, dtype=U8, device=DEV)),
        lambda: F.fp8moe_route_weight_grad_ckpt(h, hq, None, row_of),
        lambda: F.fp8moe_route_weight_grad_ckpt(h, h, hs, row_of),
        lambda: F.fp8moe_route_weight_grad_ckpt(h, hq, hs[:32], row_of),
        lambda: F.fp8moe_route_weight_grad_ckpt(h, hq, hs, row_of.long()),
        lambda: F.fp8moe_mxfp8_moe_decode(x.float(), idx, tw, w1, s1, w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx.long(), tw, w1, s1, w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx, tw[:, :1], w1, s1, w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx, tw, w1[:4], s1, w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx, tw, w1, s1[:-1], w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx, tw, w1, s1, w2, s2[:-1]),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx, tw, w1, s1, w2.transpose(1, 2), s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx, tw, w1, s1, w2, s2, out=torch.empty_like(x).float()),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx, tw, w1, s1, w2, s2, workspace=torch.empty(1024, dtype=U8, device=DEV)),
        lambda: F.fp8moe_mxfp8_moe_decode(x.t().contiguous().t(), idx, tw, w1, s1, w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x[:, :0], idx, tw, w1, s1, w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x, idx[:, :0], tw[:, :0], w1, s1, w2, s2),
        lambda: F.fp8moe_mxfp8_moe_decode(x.expand(4, 64)[:1].expand(4, 64), idx, tw, w1, s1, w2, s2),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(F.Fp8MoeError):
            call()
            pytest.fail(f"call {i} is not refused")
    assert F.fp8moe_get_device_status() == 0
    F.fp8moe_mxfp8_moe_decode(x, idx, tw, w1, s1, w2, s2)
    assert F.fp8moe_get_device_status() == 0


# --- threads and streams --------------------------------------------------------------

def test_two_host_threads(F):
    """Both forms of the few tokens' kernel and a checkpointed backward from threads
    of their own, each on its stream: the bits of calls alone."""
    one, few = _layer(F, 1, 512, 256, 6, 4), _layer(F, 20, 256, 512, 6, 2)
    dout = _bf16((640, 256), 2)
    hq, hs = _ckpt(640, 512)
    calls = [lambda s: (F.fp8moe_mxfp8_moe_decode(*one, stream=s),), lambda s: (F.fp8moe_mxfp8_moe_decode(*few, stream=s),),
             lambda s: F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, need_dh=False, dim1=True, act1=True, s1_layout=F.SCALES_ROWMAJOR,
                                                stream=s)]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    fails = []

    def work(call, ref):
        s = torch.cuda.Stream()
        for _ in range(40):
            got = call(s)
            s.synchronize()
            if not all(a is None or torch.equal(a, b) for a, b in zip(got, ref)):
                fails.append(1)

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fails and F.fp8moe_get_device_status() == 0


# --- many rows ------------------------------------------------------------------------

def test_more_row_tiles_than_a_grid_dimension(F):
    """65540 tiles of 64 rows: the last rows have the bits of a call on them alone."""
    M, Fd, n = 65540 * 64, 32, 256
    dout = _bf16((4096, Fd), 2).repeat(M // 4096 + 1, 1)[:M]
    hq, hs = _ckpt(M, 2 * Fd)
    lay = dict(s0_layout=F.SCALES_ROWMAJOR, s1_layout=F.SCALES_ROWMAJOR, dim0=True, dim1=True, act1=True)
    big = F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, **lay)
    for cut in (slice(M - n, M), slice(32768 * 64 - 128, 32768 * 64 + 128), slice(0, n)):
        small = F.fp8moe_swiglu_bwd_ckpt(dout[cut], hq[cut], hs[cut], **lay)
        blocks = slice(cut.start // 32, cut.stop // 32)
        parts = [big[0][cut], big[1][cut], big[2][cut], big[3][:, cut], big[4][:, blocks], big[5][:, cut], big[6][:, blocks]]
        for i, (a, b) in enumerate(zip(parts, small)):
            assert torch.equal(a, b), i
    # tiled scales: a row's place among them
    tiled = F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, need_dh=False, act1=True)
    rows = tiled[6].view(-1)[:M // 128 * 512].view(M // 128, 32, 16)[:, :, :4].permute(1, 0, 2).reshape(32, M // 32)
    assert torch.equal(tiled[5], big[5]) and torch.equal(rows, big[6])
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.slow
def test_large_activation(F):
    """2.3e9 gate and up values."""
    M, Fd, n = 280000 // 128 * 128, 4096, 256
    dout = _bf16((4096, Fd), 2).repeat(M // 4096 + 1, 1)[:M]
    h = _bf16((4096, 2 * Fd), 3).repeat(M // 4096 + 1, 1)[:M]
    cut, blocks = slice(M - n, M), slice((M - n) // 32, M // 32)
    lay = dict(s0_layout=F.SCALES_ROWMAJOR, s1_layout=F.SCALES_ROWMAJOR, dim0=True, dim1=True)
    _, q0, s0, q1, s1, hq, hs = F.fp8moe_swiglu_fwd_ckpt(h, need_out=False, **lay)
    small = F.fp8moe_swiglu_fwd_ckpt(h[cut], need_out=False, **lay)
    for a, b in zip((q0[cut], s0[cut], q1[:, cut], s1[:, blocks], hq[cut], hs[cut]), small[1:]):
        assert torch.equal(a, b)
    del h, q0, s0, q1, s1
    big = F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, need_dh=False, act1=True, **lay)
    small = F.fp8moe_swiglu_bwd_ckpt(dout[cut], hq[cut], hs[cut], need_dh=False, act1=True, **lay)
    parts = (big[1][cut], big[2][cut], big[3][:, cut], big[4][:, blocks], big[5][:, cut], big[6][:, blocks])
    for i, (a, b) in enumerate(zip(parts, small[1:])):
        assert torch.equal(a, b), i
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.slow
def test_large_norm_and_weight_grad(F):
    T, H, n = 270000, 8192, 1024    # 2.2e9 elements
    hq, hs = _ckpt(T, H)
    dy = _bf16((4096, H), 2).repeat(T // 4096 + 1, 1)[:T]
    rstd, w = torch.rand(T, device=DEV) + 0.5, torch.ones(H, device=DEV)
    cut = slice(T - n, T)
    dx, dw = F.fp8moe_add_rmsnorm_bwd_ckpt(dy, hq, hs, rstd, w)
    small, _ = F.fp8moe_add_rmsnorm_bwd_ckpt(dy[cut], hq[cut], hs[cut], rstd[cut], w)
    assert torch.equal(dx[cut], small) and bool(torch.isfinite(dw).all())
    del dx
    row_of = torch.arange(T, device=DEV, dtype=I32).flip(0).reshape(T // 2, 2)
    d = F.fp8moe_route_weight_grad_ckpt(dy[:T // 2], hq, hs, row_of)
    assert torch.equal(d[:n // 2], F.fp8moe_route_weight_grad_ckpt(dy[:n // 2], hq[cut], hs[cut], row_of[:n // 2] - (T - n)))


@pytest.mark.slow
def test_large_experts(F):
    """W1 of 2.4e9 codes: the last experts' pieces lie past 2^31 bytes."""
    T, H, Fd, E, k = 1, 4096, 2048, 144, 2
    x, idx, w, w1, s1, w2, s2 = _layer(F, T, H, Fd, E, k)
    idx[0, 0], idx[0, 1] = E - 1, 3
    out = F.fp8moe_mxfp8_moe_decode(x, idx, w, w1, s1, w2, s2)
    pick = torch.tensor([3, E - 1], device=DEV)
    per = lambda s: s.view(E, -1)[pick].contiguous().view(-1)
    small = F.fp8moe_mxfp8_moe_decode(x, torch.tensor([[1, 0]], dtype=I32, device=DEV), w, w1[pick], per(s1), w2[pick], per(s2))
    assert torch.equal(out, small) and bool(out.float().abs().max() > 0)
    assert F.fp8moe_get_device_status() == 0


# --- long runs of tiles, odd addresses ---------------------------------------------------

def _values(q, s):
    v = q.view(torch.float8_e4m3fn).float().view(q.shape[0], -1, 32) * torch.exp2(s.float() - 127)[..., None]
    return v.view(q.shape).to(BF16)


def _at_odd(t):
    """The same bytes one byte further."""
    raw = torch.empty(t.numel() + 1, dtype=U8, device=DEV)
    raw[1:].copy_(t.reshape(-1))
    return raw[1:].view(t.shape)


@pytest.mark.parametrize("M,Fd", [(60032, 128), (60000, 160), (40000, 416), (80000, 512), (30016, 608)])
@pytest.mark.parametrize("grouped", [False, True])
def test_backward_long_runs(F, M, Fd, grouped):
    """Many tiles: a warp has several, and row scales go out as words, of gate and up in
    step or not (F a multiple of 128 or not)."""
    hq, hs = _ckpt(M, 2 * Fd)
    v, dout = _values(hq, hs), _bf16((4096, Fd), 2).repeat(M // 4096 + 1, 1)[:M].contiguous()
    ends = sorted({32 * i for i in (1, 7, 7, 300, M // 64)}) + [M]
    offs = torch.tensor(ends, dtype=I32, device=DEV) if grouped else None
    lay = (F.GROUP_ROWS, F.GROUP_COLS) if grouped else (F.NO_GROUPS, F.NO_GROUPS)
    kw = dict(need_dh=False, dim0=True, dim1=True)
    want = F.fp8moe_swiglu_bwd(dout, v, offs, *lay, **kw)
    act = F.fp8moe_swiglu_fwd(v, offs, *lay, need_out=False, dim1=True)
    for odd in (False, True):
        more, scales = {}, hs
        if odd:
            scales = _at_odd(hs)
            more = dict(s0=_at_odd(torch.zeros_like(want[2])), s1=_at_odd(torch.zeros_like(want[4])), q0=torch.empty_like(want[1]),
                        q1=torch.empty_like(want[3]), aq1=torch.empty_like(act[3]), as1=_at_odd(torch.zeros_like(act[4])))
        got = F.fp8moe_swiglu_bwd_ckpt(dout, hq, scales, offs, *lay, act1=True, **kw, **more)
        for a, b in zip(got[1:], (*want[1:], act[3], act[4])):
            assert torch.equal(a, b)
        # rows alone, as the last rows are not whole
        n = M - 5
        if not grouped:
            few = F.fp8moe_swiglu_bwd_ckpt(dout[:n], hq[:n], scales[:n] if odd else hs[:n], None, F.SCALES_ROWMAJOR, dim0=True)
            ref = F.fp8moe_swiglu_bwd(dout[:n], v[:n], None, F.SCALES_ROWMAJOR, dim0=True)
            assert all(torch.equal(a, b) for a, b in zip(few[:3], ref[:3]))
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.parametrize("M,Fd", [(77, 96), (20001, 160)])
def test_forward_scales_at_odd_addresses(F, M, Fd):
    h = _bf16((M, 2 * Fd), 1)
    want = F.fp8moe_swiglu_fwd_ckpt(h, need_out=False)
    hs = _at_odd(torch.zeros_like(want[6]))
    got = F.fp8moe_swiglu_fwd_ckpt(h, need_out=False, hs=hs)
    assert torch.equal(got[5], want[5]) and torch.equal(hs, want[6])


@pytest.mark.parametrize("T,H,w32", [(1301, 7168, False), (1300, 7168, True), (700, 8192, False), (2001, 4096, True), (2003, 1376, False)])
@pytest.mark.parametrize("stream", [False, True])
def test_norm_several_rows_a_thread(F, T, H, w32, stream):
    """Rings that turn several times: against float64 on the device."""
    hq, hs = _ckpt(T, H)
    v, dy, dh = _values(hq, hs).double(), _bf16((T, H), 3), _bf16((T, H), 4) if stream else None
    w = (torch.rand(H, device=DEV) + 0.5).to(F32 if w32 else BF16)
    rstd = torch.rsqrt(v.square().mean(1)).float()
    dx, dw = F.fp8moe_add_rmsnorm_bwd_ckpt(dy, hq, _at_odd(hs), rstd, w, dh)
    r, g, xh = rstd.double()[:, None], dy.double() * w.double(), v * rstd.double()[:, None]
    mean = (g * xh).mean(1, keepdim=True)
    ref = r * (g - xh * mean) + (dh.double() if stream else 0)
    size = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + (dh.double().abs() if stream else 0)
    assert bool(((dx.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2e-6 * size).all())
    ref, parts = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    assert bool(((dw.double() - ref).abs() <= (T / 8 + 32) * 2.0 ** -24 * parts).all())
    assert F.fp8moe_get_device_status() == 0


# --- few tokens with many choices ----------------------------------------------------------

def _decode_ok(F, args):
    """The sums in float64; the tolerances are those of the other tests of this call."""
    x, idx, w, w1, s1, w2, s2 = args
    (T, H), (E, _, Fd), k = x.shape, w2.shape, idx.shape[1]
    out = F.fp8moe_mxfp8_moe_decode(x, idx, w, w1, s1, w2, s2).double()
    f = 2.0 ** (118 - 127)
    a1, a2 = (m.view(torch.float8_e4m3fn).float().double() * f for m in (w1, w2))
    gu = torch.einsum("enh,th->ten", a1, x.double())
    size = torch.einsum("enh,th->ten", a1.abs(), x.double().abs())
    g, u = gu.chunk(2, 2)
    dg, du = ((max(H, Fd) / 32 + 64) * 2.0 ** -22 * size).chunk(2, 2)
    s = g * torch.sigmoid(g)
    act = s * u
    dact = 1.1 * dg * (u.abs() + du) + s.abs() * du + (2.0 ** -12 + 2.0 ** -20) * act.abs()
    y = torch.einsum("ehf,tef->teh", a2, act)
    dy = torch.einsum("ehf,tef->teh", a2.abs(), dact + (max(H, Fd) / 32 + 64) * 2.0 ** -22 * act.abs())
    share = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_add_(1, idx.long(), w.double())
    ref = torch.einsum("te,teh->th", share, y)
    # k products added in fp32, each sum off by half a step
    tol = torch.einsum("te,teh->th", share, dy + (k + 1) * 2.0 ** -24 * y.abs()) + 2.0 ** -8 * ref.abs() + 1e-30
    assert bool(((out - ref).abs() <= tol).all())
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.parametrize("T,H,Fd,E,k", [(1, 64, 64, 64, 40), (1, 96, 32, 3, 1024), (2, 96, 64, 48, 30), (2, 32, 160, 1024, 512),
                                        (24, 64, 96, 5, 4), (25, 64, 96, 5, 4)])
def test_decode_many_choices(F, T, H, Fd, E, k):
    """More than 32 pairs of one or two tokens, the same expert often; both sides of the
    entries' rule."""
    _decode_ok(F, _layer(F, T, H, Fd, E, k, seed=k))


@pytest.mark.parametrize("T,H,Fd,E,k,hot", [(8, 160, 96, 8, 2, 8), (5, 96, 64, 6, 2, 5), (3, 4128, 64, 3, 2, 3), (8, 96, 4128, 16, 4, 7),
                                            (7, 512, 256, 7, 2, 0), (20, 256, 96, 40, 4, 0), (23, 96, 160, 64, 3, 8),
                                            (23, 96, 160, 64, 3, 9), (60, 64, 512, 128, 2, 5), (100, 32, 64, 200, 4, 8)])
def test_decode_entries_of_several(F, T, H, Fd, E, k, hot):
    """Entries of up to eight pairs whose terms are made on the way, and one pair more."""
    args = _layer(F, T, H, Fd, E, k, seed=T)
    # distinct choices, the first of `hot` tokens the same
    args[1] = torch.rand(T, E, device=DEV)[:, 1:].topk(k, 1)[1].to(I32) + 1
    args[1][:hot, 0] = 0
    _decode_ok(F, args)
    x, idx, w = args[0].clone(), args[1].clone(), args[2].clone()
    w[T // 2] = 0          # and with a token that takes no part, whatever it holds
    x[T // 2] = float("nan")
    out = F.fp8moe_mxfp8_moe_decode(x, idx, w, *args[3:])
    assert not out[T // 2].any() and bool(torch.isfinite(out.float()).all())
    same = F.fp8moe_mxfp8_moe_decode(x, idx, w, *args[3:])
    assert torch.equal(out, same)
    x[T // 2] = 0
    _decode_ok(F, [x, idx, w, *args[3:]])
