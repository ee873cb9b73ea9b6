"""The expert layer of a few tokens against its definition in 64 bits.

Tolerances: x is taken exactly but for values below 2^-22 of their block's
largest, the activation to 2^-12 of itself (three e4m3 terms) and 2^-20 for exp
and the divisions.  A sum of K products is added in fp32 in K / 32 steps, each
off by at most 2^-22 of the magnitudes so far (truncated or rounded), and up to
64 partial sums: (K / 32 + 64) 2^-22.  The output is rounded once."""
import numpy as np
import pytest
import torch

from code_bounds import check_bf16
from oracle import formats as OF, moe_ops as OM, swizzle as OS

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _weights(g, E, N, K, pad=255):
    """(codes, tiled scales with ``pad`` in the padding, float64 values) of MXFP8 weights."""
    q = torch.randint(0, 256, (E, N, K), generator=g, dtype=torch.uint8)
    q[(q & 0x7F) == 0x7F] = 0
    s = torch.randint(117, 122, (E, N, K // 32), generator=g, dtype=torch.uint8)
    v = OF.decode(q.numpy(), OF.FN).reshape(E, N, K // 32, 32) * np.ldexp(1.0, s.numpy().astype(np.int32) - 127 - 6)[..., None]
    s = s - 6
    rp, cp = OS.swizzled_shape(N, K // 32, 0, -1)
    tiled = np.stack([np.where(OS.swizzle(np.ones_like(m), None, -1) != 0, OS.swizzle(m, None, -1), pad)
                      for m in s.numpy()]).astype(np.uint8)
    assert tiled.size == E * rp * cp
    return q, torch.from_numpy(tiled.reshape(-1)), v.reshape(E, N, K)


def _case(T, H, Fd, E, k, seed=0, distinct=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    if distinct:
        idx = torch.rand(T, E, generator=g).topk(k, dim=1)[1].to(torch.int32)
    else:
        idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    w = torch.rand(T, k, generator=g) + 0.05
    return x, idx, w, _weights(g, E, 2 * Fd, H), _weights(g, E, H, Fd)


def _gamma(H, Fd):
    return (max(H, Fd) / 32 + 64) * 2.0 ** -22


def _run(F, x, idx, w, w1, w2, **kw):
    d = lambda t: t.to(DEV)
    return F.fp8moe_mxfp8_moe_decode(d(x), d(idx), d(w), d(w1[0]), d(w1[1]), d(w2[0]), d(w2[1]), **kw)


def _check(F, x, idx, w, w1, w2, out=None, rows=None):
    out = _run(F, x, idx, w, w1, w2) if out is None else out
    assert F.fp8moe_get_device_status() == 0
    H, Fd = w2[2].shape[1:]
    ref, bound = OM.moe_decode(x.double().numpy(), idx.numpy(), w.numpy(), w1[2], w2[2], _gamma(H, Fd), 2.0 ** -12 + 2.0 ** -20)
    rows = slice(None) if rows is None else rows
    check_bf16(out.cpu()[rows], ref[rows], bound[rows] + 1e-30, "out")
    return out


SIZES = [  # T, H, F, E, k
    (1, 32, 32, 1, 1), (1, 64, 32, 3, 2), (1, 256, 512, 4, 1), (2, 96, 160, 5, 3), (1, 2048, 1408, 16, 6), (7, 1056, 352, 9, 4),
    (3, 128, 4096, 2, 2), (5, 4128, 64, 2, 1), (32, 288, 224, 60, 1), (33, 160, 96, 7, 1), (23, 512, 256, 256, 8),
    (64, 384, 160, 2, 1), (130, 224, 128, 1, 1), (200, 160, 224, 3, 2), (128, 256, 128, 16, 8), (1024, 64, 64, 5, 1),
    (32, 128, 128, 1024, 32)]


@pytest.mark.parametrize("T,H,Fd,E,k", SIZES)
def test_sizes(F, T, H, Fd, E, k):
    _check(F, *_case(T, H, Fd, E, k, seed=T + H))


def test_no_tokens(F):
    x, idx, w, w1, w2 = _case(1, 64, 64, 2, 1)
    out = _run(F, x[:0], idx[:0], w[:0], w1, w2)
    assert out.shape == (0, 64)


def test_nobody_is_live(F):
    """Masked tokens and experts of other devices: zeros, whatever stands in x."""
    x, idx, w, w1, w2 = _case(6, 128, 96, 4, 2)
    x[:] = float("nan")
    w[:3] = 0.0
    idx[3:] = torch.tensor([[-1, 4], [2 ** 31 - 1, -2 ** 31], [5, 1000]], dtype=torch.int32)
    out = _run(F, x, idx, w, w1, w2)
    assert torch.equal(out.view(torch.uint8), torch.zeros_like(out).view(torch.uint8))


@pytest.mark.parametrize("T", [6, 40])
def test_some_are_not_live(F, T):
    x, idx, w, w1, w2 = _case(T, 256, 160, 8, 3, seed=T)
    w[1] = 0.0
    w[4, 0] = -0.0
    w[2] = -w[2]
    idx[0, 1], idx[3, 0], idx[5] = -1, 8, torch.tensor([-7, 3, 9], dtype=torch.int32)
    _check(F, x, idx, w, w1, w2)


@pytest.mark.parametrize("T", [5, 90])
def test_an_expert_twice(F, T):
    """The same choice several times in a row counts as often."""
    x, idx, w, w1, w2 = _case(T, 160, 128, 3, 4, seed=T, distinct=False)
    idx[0] = 1
    _check(F, x, idx, w, w1, w2)


def test_strided_rows(F):
    x, idx, w, w1, w2 = _case(9, 192, 64, 4, 2)
    wide = torch.full((9, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :192] = x.to(DEV)
    d = lambda t: t.to(DEV)
    out = F.fp8moe_mxfp8_moe_decode(wide[:, :192], d(idx), d(w), d(w1[0]), d(w1[1]), d(w2[0]), d(w2[1]))
    _check(F, x, idx, w, w1, w2, out=out)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_stays_in_its_token(F, bad):
    x, idx, w, w1, w2 = _case(12, 160, 96, 3, 2, seed=5)
    x[4, 37] = bad
    out = _run(F, x, idx, w, w1, w2)
    assert out[4].isnan().all()
    rows = [t for t in range(12) if t != 4]
    x[4] = 0.0
    _check(F, x, idx, w, w1, w2, out=out, rows=rows)


def test_a_broken_expert_stays_with_its_tokens(F):
    x, idx, w, w1, w2 = _case(16, 128, 128, 6, 2, seed=9)
    idx[:8] = torch.where(idx[:8] == 2, torch.full_like(idx[:8], 3), idx[:8])
    idx[8:, 0] = 2
    ref = _run(F, x, idx, w, w1, w2)
    w1[0][2], w2[0][2] = 0x7F, 0xFF
    out = _run(F, x, idx, w, w1, w2)
    assert out[8:].isnan().all() and torch.equal(out[:8], ref[:8])


def test_wide_range(F):
    """Blocks of very different sizes, down to zeros and subnormals, up to 2^50."""
    x, idx, w, w1, w2 = _case(8, 256, 128, 4, 2, seed=3)
    x[0] = 0.0
    x[1, :32] *= 2.0 ** 50
    x[2] *= 2.0 ** -40
    x[3, 32:64] = 2.0 ** -133
    x[4] *= torch.exp2(torch.arange(256, dtype=torch.float32) % 32 - 20).to(torch.bfloat16)
    x[5, ::2] = 0.0
    out = _run(F, x, idx, w, w1, w2)
    assert not out[0].any()
    H, Fd = 256, 128
    ref, bound = OM.moe_decode(x.double().numpy(), idx.numpy(), w.numpy(), w1[2], w2[2], _gamma(H, Fd) + 2.0 ** -18, 2.0 ** -12 + 2.0 ** -20)
    check_bf16(out, ref, bound + 1e-30, "out")


def test_any_workspace_and_the_same_bits(F):
    x, idx, w, w1, w2 = _case(24, 512, 384, 8, 4, seed=11)
    n = F.fp8moe_mxfp8_moe_decode_workspace_bytes(24, 4, 8, 512, 384)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device=DEV)
        out = torch.full((26, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        r = _run(F, x, idx, w, w1, w2, out=out[1:25], workspace=ws[:n])
        assert r.data_ptr() == out[1].data_ptr() and (out[0] == 7).all() and (out[25] == 7).all()
        assert (ws[n:] == fill).all()
        first = r.clone() if first is None else first
        assert torch.equal(r, first)
    _check(F, x, idx, w, w1, w2, out=first)


@pytest.mark.parametrize("T", [3, 50])
def test_graph_and_streams(F, T):
    """Captured and replayed with other routing; two graphs that share a workspace;
    calls on two streams at once."""
    x, idx, w, w1, w2 = _case(T, 320, 160, 6, 2, seed=T)
    x2, idx2, w_2, _, _ = _case(T, 320, 160, 6, 2, seed=T + 1)
    d = lambda t: t.to(DEV)
    args = [d(x), d(idx), d(w)]
    rest = [d(w1[0]), d(w1[1]), d(w2[0]), d(w2[1])]
    ws = torch.empty(F.fp8moe_mxfp8_moe_decode_workspace_bytes(T, 2, 6, 320, 160), dtype=torch.uint8, device=DEV)
    want = [F.fp8moe_mxfp8_moe_decode(*args, *rest), F.fp8moe_mxfp8_moe_decode(d(x2), d(idx2), d(w_2), *rest)]
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(F.fp8moe_mxfp8_moe_decode(*args, *rest, workspace=ws))
        graphs.append(g)
    for i, new in enumerate([(x, idx, w), (x2, idx2, w_2), (x, idx, w)]):
        for a, b in zip(args, new):
            a.copy_(d(b))
        for g, o in zip(graphs, outs):
            o.fill_(3.0)
            g.replay()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want[i % 2])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(8):
        s = streams[i % 2]
        got.append(F.fp8moe_mxfp8_moe_decode(*args, *rest, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) for o in got)
    assert F.fp8moe_get_device_status() == 0


def test_as_the_quantizer_lays_weights_out(F):
    """Weights from fp8moe_mxfp8_quantize_dual, choices from the router, on a
    block of the trained layer's form."""
    g = torch.Generator().manual_seed(2)
    T, H, Fd, E, k = 4, 256, 160, 8, 2
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    b1 = (torch.randn(E, 2 * Fd, H, generator=g) * H ** -0.5).to(torch.bfloat16).to(DEV)
    b2 = (torch.randn(E, H, Fd, generator=g) * Fd ** -0.5).to(torch.bfloat16).to(DEV)
    idx, w, _, _, _ = F.fp8moe_router_fwd(torch.randn(T, E, generator=g).to(DEV), k)
    q1, s1, _, _ = F.fp8moe_mxfp8_quantize_dual(b1, dim1=False)
    q2, s2, _, _ = F.fp8moe_mxfp8_quantize_dual(b2, dim1=False)
    out = F.fp8moe_mxfp8_moe_decode(x, idx, w, q1, s1, q2, s2)

    def value(q, s):
        E, N, K = q.shape
        rp, cp = OS.swizzled_shape(N, K // 32, 0, -1)
        byte = np.stack([OS.unswizzle(m, rp, cp)[:N, :K // 32] for m in s.cpu().numpy().reshape(E, -1)])
        return (OF.decode(q.cpu().numpy(), OF.FN).reshape(E, N, K // 32, 32) *
                np.ldexp(1.0, byte.astype(np.int32) - 127)[..., None]).reshape(E, N, K)

    ref, bound = OM.moe_decode(x.double().cpu().numpy(), idx.cpu().numpy(), w.cpu().numpy(), value(q1, s1), value(q2, s2),
                               _gamma(H, Fd), 2.0 ** -12 + 2.0 ** -20)
    check_bf16(out, ref, bound + 1e-30, "out")


@pytest.mark.parametrize("T", [7, 8, 11, 17, 21, 24, 31])
def test_one_expert_for_all(F, T):
    """Every token's choice is the same expert, and a CTA's run has several row tiles:
    both accumulators in use with as many columns as an entry has."""
    x, idx, w, w1, w2 = _case(T, 65536, 64, 2, 1, seed=T)
    _check(F, x, torch.ones_like(idx), w, w1, w2)
