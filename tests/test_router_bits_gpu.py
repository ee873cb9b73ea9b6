"""What the router's results hang on to the last bit: the size of the batch, the
division by the scores' sum, and the sigmoid's slope where it is nearly one."""
import numpy as np
import pytest
import torch

from code_bounds import check_bf16
from oracle import moe_ops as OM

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 1e-5   # see test_router_gpu


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("E,k", [(3, 2), (8, 2), (8, 8), (16, 4), (20, 8), (31, 5), (33, 4), (64, 6), (64, 8), (100, 9),
                                 (128, 16), (256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
def test_a_token_does_not_depend_on_its_batch(F, E, k, score, bf16):
    """A token's choice and weights have the same bits alone, among a few and
    among many tokens."""
    T = 5003
    g = torch.Generator().manual_seed(E + k)
    x = (torch.randn(T, E, generator=g) * 2).to(torch.bfloat16 if bf16 else torch.float32).to(DEV)
    b = (torch.randn(E, generator=g) * 0.1).to(DEV)
    sc = F.SCORE_SOFTMAX if score == "softmax" else F.SCORE_SIGMOID
    for bias in (None, b):
        for renorm in (False, True):
            kw = dict(score=sc, renormalize=renorm, bias=bias, need_balance=False)
            idx, w = F.fp8moe_router_fwd(x, k, **kw)[:2]
            for n in (1, 37, 1250):
                for at in range(0, T, n) if n > 1 else range(0, T, 101):
                    i, v = F.fp8moe_router_fwd(x[at:at + n], k, **kw)[:2]
                    assert torch.equal(i, idx[at:at + n]) and torch.equal(v, w[at:at + n])


@pytest.mark.parametrize("E,T", [(1, 9), (1, 4096), (7, 2000), (64, 4096), (100, 6000), (256, 300)])
def test_the_only_live_expert_has_probability_one(F, E, T):
    """s / s = 1 whatever s is: the sum over the tokens is their number, the
    loss E N N / N^2, and its gradient p (c - p c) is zero."""
    g = torch.Generator().manual_seed(E)
    x = torch.full((T, E), -float("inf"))
    x[:, E // 2] = torch.randn(T, generator=g) * 3
    x = x.to(DEV)
    idx, w, counts, psum, loss = F.fp8moe_router_fwd(x, 1, score=F.SCORE_SIGMOID)
    assert bool((idx == E // 2).all()) and float(psum[E // 2]) == T and float(psum.sum()) == T and float(loss) == E
    for xs in (x, x.to(torch.bfloat16)):
        d = F.fp8moe_router_bwd(xs, idx, counts, None, torch.ones(1, device=DEV), score=F.SCORE_SIGMOID)
        assert not d.any()


@pytest.mark.parametrize("T,E,k", [(5, 8, 2), (64, 64, 6), (300, 256, 8), (1400, 33, 4), (5000, 100, 9), (40, 700, 8)])
@pytest.mark.parametrize("renorm,bf16", [(False, False), (True, False), (False, True)])
def test_slope_of_confident_experts(F, T, E, k, renorm, bf16):
    """The gradient carries the factor 1 - s, which is e^-x and not the
    difference of two numbers near one: bounds on the terms with that factor."""
    g = torch.Generator().manual_seed(T)
    x = torch.rand(T, E, generator=g) * 16 + 4
    far = torch.rand(T, E, generator=g)
    x = torch.where(far < 0.2, -x, x)
    x[torch.rand(T, E, generator=g) < 0.02] = 60.0
    x[torch.rand(T, E, generator=g) < 0.02] = -95.0
    x[0], x[1] = 18.0, torch.linspace(-90, 90, E)
    x = x.to(torch.bfloat16) if bf16 else x
    kw = dict(score=F.SCORE_SIGMOID, renormalize=renorm, route_scale=2.5)
    idx, _, counts, _, _ = F.fp8moe_router_fwd(x.to(DEV), k, **kw)
    dw = torch.randn(T, k, generator=g)
    got = F.fp8moe_router_bwd(x.to(DEV), idx, counts, dw.to(DEV), torch.full((1,), 3.0, device=DEV), **kw)
    ii, cc = idx.cpu().numpy().astype(np.int64), counts.cpu().numpy()[:E]
    # 1 - s of the sigmoid in 64 bits is s of -x
    s, p = OM.scores(_np(x), "sigmoid")
    rest = OM.scores(-_np(x), "sigmoid")[0]
    c = 3.0 * E / (k * T ** 2) * cc
    r, size = p * (c - (p * c).sum(1, keepdims=True)), p * (c + (p * c).sum(1, keepdims=True))
    sel, d = np.take_along_axis(s, ii, 1), _np(dw)
    if renorm:
        sel = sel / sel.sum(1, keepdims=True)
    u = 2.5 * sel * (d - ((d * sel).sum(1, keepdims=True) if renorm else 0))
    au = 2.5 * sel * (np.abs(d) + ((np.abs(d) * sel).sum(1, keepdims=True) if renorm else 0))
    full, afull = np.zeros_like(s), np.zeros_like(s)
    np.put_along_axis(full, ii, u, 1)
    np.put_along_axis(afull, ii, au, 1)
    ref, lim = rest * (r + full), 4 * REL * rest * (size + afull) + 1e-37
    if bf16:
        check_bf16(got, ref, lim, "dlogits")
    else:
        assert np.all(np.abs(_np(got) - ref) <= lim)
