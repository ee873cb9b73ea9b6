"""The router, its gradient and the combine's weight gradient against the
float64 definitions.

Tolerances.  A score: exp of an argument that is off by 2^-24 of itself (at
most 100 here: 6e-6), two ulp of exp, and a division: 1e-5 relative covers it
and the sums of up to 1024 positive terms; weights, probabilities and sums
take twice that, the loss three times.  Gradients: the same on the sizes of
the terms that are added.  bf16 logit gradients lie between the roundings of
the two ends."""
import numpy as np
import pytest
import torch

from code_bounds import check_bf16
from oracle import moe_ops as OM, routing as RT

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 1e-5


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _np(t):
    return t.double().cpu().numpy()


def _logits(T, E, seed, bf16, dead=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * 2
    if dead:
        x[:, torch.randperm(E, generator=g)[:dead]] = -float("inf")
    return x.to(torch.bfloat16) if bf16 else x


def _score(F, name):
    return F.SCORE_SOFTMAX if name == "softmax" else F.SCORE_SIGMOID


def _check(F, x, k, score, renorm, scale, bias=None, mask=None, ld=None):
    """One forward against the definition on the kernel's own choice, and the
    choice against the keys."""
    T, E = x.shape
    d = lambda t: None if t is None else t.to(DEV)
    xd = d(x)
    if ld is not None:
        wide = torch.full((T, ld), float("nan"), dtype=x.dtype, device=DEV)
        wide[:, :E] = xd
        xd = wide[:, :E]
    out = F.fp8moe_router_fwd(xd, k, score=_score(F, score), renormalize=renorm, route_scale=scale, bias=d(bias),
                              token_mask=d(mask))
    idx, w, counts, psum, loss = (t.cpu() for t in out)
    idx = idx.numpy().astype(np.int64)
    m = None if mask is None else mask.numpy()
    ref = OM.router(_np(x), k, score, renorm, scale, None if bias is None else _np(bias), m, idx=idx)
    assert np.all((idx >= 0) & (idx < E)) and all(len(set(r)) == k for r in idx.tolist())
    live = OM._live(_np(x), m)
    key = live if bias is None else np.where(live == -np.inf, -np.inf, ref["s"] + _np(bias))
    if bias is None:
        assert np.array_equal(idx, OM.choose(key, k))
    else:
        best = np.take_along_axis(key, OM.choose(key, k), 1)
        mine = np.take_along_axis(key, idx, 1)
        dead = best == -np.inf
        assert np.array_equal(dead, mine == -np.inf)
        assert np.all(np.where(dead, 0.0, np.abs(np.where(dead, 0.0, best) - np.where(dead, 0.0, mine))) <= 4e-7)
    assert np.all(np.abs(_np(w) - ref["w"]) <= 2 * REL * np.abs(ref["w"]) + 1e-37)
    assert np.array_equal(counts.numpy()[:E], ref["counts"]) and int(counts[E]) == ref["tokens"]
    assert np.all(np.abs(_np(psum) - ref["prob_sum"]) <= 2 * REL * ref["prob_sum"] + 1e-37)
    assert abs(float(loss) - ref["loss"]) <= 3 * REL * ref["loss"]
    # without the sums the choice is the same
    i2, w2, *none = F.fp8moe_router_fwd(xd, k, score=_score(F, score), renormalize=renorm, route_scale=scale,
                                        bias=d(bias), token_mask=d(mask), need_balance=False)
    assert none == [None] * 3 and torch.equal(i2, out[0]) and torch.equal(w2, out[1])
    return out


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 256, 8), (16, 64, 6), (17, 33, 32), (300, 100, 4),
                                   (2500, 256, 8), (5, 1024, 10), (70, 1000, 32), (1300, 5, 5)])
@pytest.mark.parametrize("score,renorm,bf16", [("softmax", False, True), ("softmax", True, False),
                                               ("sigmoid", True, False), ("sigmoid", False, True)])
def test_forward(F, T, E, k, score, renorm, bf16):
    x = _logits(T, E, T + E, bf16, dead=min(3, E - 1))
    bias = torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.1
    _check(F, x, k, score, renorm, 2.5)
    _check(F, x, k, score, renorm, 1.0, bias=bias, ld=E + 5)


@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks(F, T, score):
    """Padding tokens (whose logits hold anything), rows of nothing but -inf,
    the type's lowest value, and fewer experts left than k."""
    E, k = 40, 6
    for bf16 in (False, True):
        x = _logits(T, E, 5, bf16)
        lowest = torch.finfo(x.dtype).min
        x[0] = -float("inf")
        x[1] = lowest
        x[2, 3:] = -float("inf")
        x[3, ::2] = lowest
        mask = torch.ones(T, dtype=torch.uint8)
        if T > 4:
            mask[10:60:3] = 0
        _check(F, x, k, score, True, 1.5, mask=mask)
        bias = torch.linspace(-0.5, 0.5, E)
        clean = _check(F, x, k, score, False, 1.0, bias=bias, mask=mask)
        y = x.clone()
        y[mask == 0] = float("nan")
        got = F.fp8moe_router_fwd(y.to(DEV), k, score=_score(F, score), renormalize=False, bias=bias.to(DEV),
                                  token_mask=mask.bool().to(DEV))
        for a, b in zip(got, clean):
            assert torch.equal(a, b)


# many tokens over few experts: eight or sixteen lanes a token, ragged tokens
# per warp, k up to the lanes and (the last two) past them
MANY = [(1301, 8, 8), (1250, 16, 2), (2431, 31, 5), (1999, 64, 6), (4999, 100, 9), (5003, 128, 16), (1301, 64, 9),
        (4999, 128, 17)]


@pytest.mark.parametrize("T,E,k", MANY)
@pytest.mark.parametrize("score,bf16", [("softmax", False), ("sigmoid", True)])
def test_many_tokens(F, T, E, k, score, bf16):
    x = _logits(T, E, T + E, bf16, dead=1)
    x[5] = -float("inf")
    mask = torch.ones(T, dtype=torch.uint8)
    mask[::7] = 0
    bias = torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.1
    _check(F, x, k, score, True, 2.5, mask=mask)
    _check(F, x, k, score, False, 1.0, bias=bias, ld=E + 3)


def test_ties_and_signed_zero(F):
    """Equal keys go to the lowest id; 0 and -0 are equal."""
    x = torch.zeros(40, 96)
    x[1:, ::2] = -0.0
    x[2, 70] = x[2, 5] = 1.0
    for score in ("softmax", "sigmoid"):
        idx = F.fp8moe_router_fwd(x.to(DEV), 4, score=_score(F, score))[0].cpu()
        assert idx[0].tolist() == idx[1].tolist() == [0, 1, 2, 3] and idx[2].tolist() == [5, 70, 0, 1]
        idx = F.fp8moe_router_fwd(x.to(DEV), 4, score=_score(F, score), bias=torch.zeros(96, device=DEV))[0].cpu()
        assert idx[0].tolist() == [0, 1, 2, 3] and idx[2].tolist() == [5, 70, 0, 1]


@pytest.mark.parametrize("E,k", [(130, 6), (256, 8), (384, 12), (1000, 32), (1024, 20)])
@pytest.mark.parametrize("T", [37, 9999])
def test_one_lane_has_the_best(F, T, E, k):
    """Runs of equal or falling keys within one lane's experts, which lose more
    of them than a lane keeps at hand."""
    g = torch.Generator().manual_seed(E)
    x = (torch.randint(-2, 3, (T, E), generator=g) * 0.5).float()
    x[1] = 0.0
    x[2] = -torch.arange(E, dtype=torch.float32)
    x[3] = torch.arange(E, dtype=torch.float32) / E
    for piece in range(min(E // 128, 8)):      # the four neighbours of one lane in every piece
        x[4, 128 * piece + 8:128 * piece + 12] = 9.0 - piece
        x[5, 128 * piece + 8:128 * piece + 12] = 9.0
    x[6, 3:] = -float("inf")
    _check(F, x, k, "softmax", True, 2.5)
    _check(F, x.to(torch.bfloat16), k, "sigmoid", False, 1.0)
    bias = (torch.randint(-1, 2, (E,), generator=g) * 0.25).float()
    _check(F, x, k, "sigmoid", True, 1.0, bias=bias)


@pytest.mark.parametrize("E,k", [(4, 3), (15, 5), (20, 8), (60, 6), (96, 8), (256, 8), (384, 12), (1024, 8)])
@pytest.mark.parametrize("T", [37, 1301])
def test_bf16_ties(F, T, E, k):
    """Rows of few different values, signed zeros and NaN: the lowest ids of
    equal logits win, in any layout of lanes."""
    g = torch.Generator().manual_seed(E)
    x = (torch.randint(-3, 4, (T, E), generator=g) * 0.25).to(torch.bfloat16)
    x[1] = -0.0
    x[2, ::2] = -float("inf")
    x[3] = torch.finfo(torch.bfloat16).min
    _check(F, x, k, "softmax", True, 2.5)
    x[5, 1] = float("nan")
    x[6] = float("nan")
    idx = F.fp8moe_router_fwd(x.to(DEV), k, score=F.SCORE_SIGMOID)[0].cpu()
    live = _np(x).copy()
    live[np.isnan(live)] = -np.inf
    assert np.array_equal(idx.numpy(), OM.choose(live, k))


@pytest.mark.parametrize("E", [4, 8, 12, 28, 64, 100, 128, 256, 384, 1024])
@pytest.mark.parametrize("bf16", [False, True])
def test_row_strides_and_offsets(F, E, bf16):
    """Rows that start anywhere give the bits of aligned rows, forward and
    backward."""
    k, score = min(E, 6), F.SCORE_SOFTMAX
    for T in (41, 1303):
        x = _logits(T, E, E, bf16).to(DEV)
        mask = torch.ones(T, dtype=torch.uint8, device=DEV)
        mask[3::5] = 0
        base = F.fp8moe_router_fwd(x, k, score=score, token_mask=mask)
        dw, dl = torch.randn(T, k, device=DEV), torch.full((1,), 0.5, device=DEV)
        grad = F.fp8moe_router_bwd(x, base[0], base[2], dw, dl, score=score, token_mask=mask)
        for ld, at in ((E + 1, 0), (E + 4, 2), (E + 4, 4), (E + 2, 1), (E + 8, 8)):
            buf = torch.full((T * ld + at,), float("nan"), dtype=x.dtype, device=DEV)
            v = buf[at:].view(T, ld)[:, :E]
            v.copy_(x)
            for a, b in zip(F.fp8moe_router_fwd(v, k, score=score, token_mask=mask), base):
                assert torch.equal(a, b)
            assert torch.equal(F.fp8moe_router_bwd(v, base[0], base[2], dw, dl, score=score, token_mask=mask), grad)
            out = torch.empty(T * E + 1, dtype=x.dtype, device=DEV)[1:].view(T, E)
            F.fp8moe_router_bwd(v, base[0], base[2], dw, dl, score=score, token_mask=mask, dlogits=out)
            assert torch.equal(out, grad)


def test_nan_logits_keep_the_ids_valid(F):
    x = _logits(64, 64, 1, False)
    x[7, 3] = x[7, 9] = float("nan")
    x[8] = float("nan")
    for score in ("softmax", "sigmoid"):
        idx, w, *_ = F.fp8moe_router_fwd(x.to(DEV), 6, score=_score(F, score))
        i = idx.cpu()
        assert bool(((i >= 0) & (i < 64)).all()) and all(len(set(r)) == 6 for r in i.tolist())
        assert 3 not in i[7].tolist() and 9 not in i[7].tolist() and i[8].tolist() == [0, 1, 2, 3, 4, 5]
        assert bool(torch.isfinite(w[:7]).all()) and bool(torch.isnan(w[8]).all())


def test_no_tokens(F):
    x = torch.empty(0, 16, device=DEV)
    idx, w, counts, psum, loss = F.fp8moe_router_fwd(x, 2)
    assert idx.shape == w.shape == (0, 2) and not counts.any() and not psum.any() and float(loss) == 0.0
    assert F.fp8moe_router_bwd(x, idx, counts, w, loss).shape == (0, 16)


def test_same_bits_every_time(F):
    """Large enough for many CTAs; a dirty workspace does not matter."""
    T, E = 20000, 128
    x = _logits(T, E, 3, False).to(DEV)
    ws = torch.full((F.fp8moe_router_workspace_bytes(T, E) // 4,), float("nan"), device=DEV)
    a = F.fp8moe_router_fwd(x, 8)
    b = F.fp8moe_router_fwd(x, 8, workspace=ws)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (2, 8, 2), (33, 256, 8), (257, 100, 4), (9, 1024, 10), (40, 40, 32)] + MANY)
@pytest.mark.parametrize("score,renorm,bf16", [("softmax", False, False), ("softmax", True, True),
                                               ("sigmoid", True, False), ("sigmoid", False, True)])
def test_backward(F, T, E, k, score, renorm, bf16):
    x = _logits(T, E, T + E, bf16, dead=min(2, E - 1))
    mask = torch.ones(T, dtype=torch.uint8)
    if T > 8:
        mask[::5] = 0
        x[1] = -float("inf")
    xd, md = x.to(DEV), mask.to(DEV)
    kw = dict(score=_score(F, score), renormalize=renorm, route_scale=2.5, token_mask=md)
    idx, _, counts, _, _ = F.fp8moe_router_fwd(xd, k, **kw)
    g = torch.Generator().manual_seed(1)
    dw, dloss = torch.randn(T, k, generator=g), torch.tensor([3.0])
    ii, cc, n = idx.cpu().numpy().astype(np.int64), counts.cpu().numpy()[:E], int(counts[E])
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        got = F.fp8moe_router_bwd(xd, idx, counts if use_l else None, dw.to(DEV) if use_w else None,
                                  dloss.to(DEV) if use_l else None, **kw)
        args = (_np(x), ii, cc, n, _np(dw) if use_w else None, 3.0 if use_l else 0.0, score, renorm, 2.5, mask.numpy())
        ref = OM.router_grad(*args)
        # the size of what is added: the same formula on absolute values
        s, p = OM.scores(OM._live(_np(x), mask.numpy()), score)
        c = (3.0 if use_l else 0.0) * E / (k * max(n, 1) ** 2) * cc
        size = p * (c + (p * c).sum(1, keepdims=True))
        if use_w:
            sel = np.take_along_axis(s, ii, 1)
            if renorm:
                z = sel.sum(1, keepdims=True)
                sel = sel / np.where(z == 0, 1, z)
            ad = np.abs(_np(dw))
            u = 2.5 * sel * (ad + ((ad * sel).sum(1, keepdims=True) if renorm else 0))
            full = np.zeros_like(s)
            np.put_along_axis(full, ii, u, 1)
            size = size + full + (p * u.sum(1, keepdims=True) if score == "softmax" else 0)
        lim = 4 * REL * size + 1e-37
        if bf16:
            check_bf16(got, ref, lim, "dlogits")
        else:
            assert got.dtype == x.dtype and np.all(np.abs(_np(got) - ref) <= lim)
        assert not got[mask.to(DEV) == 0].any()


def test_backward_skips_foreign_ids_and_masked_garbage(F):
    x = _logits(16, 24, 2, False)
    idx = F.fp8moe_router_fwd(x.to(DEV), 3)[0]
    dw = torch.ones(16, 3)
    mask = torch.ones(16, dtype=torch.uint8)
    mask[4] = 0
    bad = idx.clone()
    bad[2, 1], bad[3, 0] = -1, 24
    x2, dw2 = x.clone(), dw.clone()
    x2[4], dw2[4] = float("nan"), float("nan")
    got = F.fp8moe_router_bwd(x2.to(DEV), bad, None, dw2.to(DEV), renormalize=False, token_mask=mask.to(DEV))
    want = F.fp8moe_router_bwd(x.to(DEV), idx, None, dw.to(DEV), renormalize=False, token_mask=mask.to(DEV))
    keep = [t for t in range(16) if t not in (2, 3)]
    assert torch.equal(got[keep], want[keep]) and bool(torch.isfinite(got).all()) and not got[4].any()


@pytest.mark.parametrize("T,N,k", [(1, 8, 1), (3, 264, 2), (50, 1032, 4), (7, 7168, 8), (3000, 256, 3), (9, 520, 11),
                                   (2600, 64, 8)])
def test_weight_grad(F, T, N, k):
    """fp32 sums of N products: at most N / 32 terms in a row and 8 joins."""
    g = torch.Generator().manual_seed(T)
    rows = T * k + 5
    y, dout = torch.randn(rows, N, generator=g).to(torch.bfloat16), torch.randn(T, N, generator=g).to(torch.bfloat16)
    row_of = torch.randperm(rows, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    row_of[0, 0] = -1
    got = F.fp8moe_route_weight_grad(dout.to(DEV), y.to(DEV), row_of.to(DEV))
    r = row_of.numpy()
    ref = np.einsum("tn,tkn->tk", _np(dout), _np(y)[np.maximum(r, 0)]) * (r >= 0)
    size = np.einsum("tn,tkn->tk", np.abs(_np(dout)), np.abs(_np(y))[np.maximum(r, 0)])
    assert np.all(np.abs(_np(got) - ref) <= (N / 32 + 16) * 2.0 ** -24 * size)
    if T <= 50:
        assert np.allclose(ref, OM.weight_grad(_np(dout), _np(y), r), rtol=1e-12, atol=1e-9)


@pytest.mark.parametrize("T,N,k", [(2503, 8, 3), (5000, 376, 5), (2503, 392, 6), (1301, 968, 7), (1301, 1032, 1),
                                   (1301, 2048, 2), (310, 4088, 4), (161, 8200, 8), (2435, 248, 13), (77, 640, 6)])
def test_weight_grad_lane_counts(F, T, N, k):
    """Sizes on both sides of each choice of lanes per token: many and few
    tokens, short and long rows; missing rows anywhere, and rows of y that no
    pair names hold NaN.  The bound is test_weight_grad's."""
    g = torch.Generator().manual_seed(N)
    rows = T * k + 9
    y, dout = torch.randn(rows, N, generator=g).to(torch.bfloat16), torch.randn(T, N, generator=g).to(torch.bfloat16)
    perm = torch.randperm(rows, generator=g)
    row_of = perm[:T * k].reshape(T, k).to(torch.int32)
    y[perm[T * k:]] = float("nan")
    gone = torch.rand(T, k, generator=g) < 0.2
    y[row_of[gone].long()] = float("nan")
    row_of[gone] = -1
    got = _np(F.fp8moe_route_weight_grad(dout.to(DEV), y.to(DEV), row_of.to(DEV)))
    r, yn = row_of.numpy(), _np(torch.nan_to_num(y))
    ref = np.einsum("tn,tkn->tk", _np(dout), yn[np.maximum(r, 0)]) * (r >= 0)
    size = np.einsum("tn,tkn->tk", np.abs(_np(dout)), np.abs(yn)[np.maximum(r, 0)])
    assert np.all(np.abs(got - ref) <= (N / 32 + 16) * 2.0 ** -24 * size) and not got[r < 0].any()


def test_weight_grad_is_the_difference_of_the_combine(F):
    """<unpermute(y, w + s e) - unpermute(y, w - s e), dout> / 2s, exact in w up
    to the combine's bf16 output: values chosen so that it rounds nothing."""
    T, N, k, E = 20, 64, 3, 7
    g = torch.Generator().manual_seed(4)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    _, _, rrow = RT.route_permute(np.zeros((T, 8), np.float32), idx.numpy(), E)
    row_of = torch.from_numpy(rrow.astype(np.int32)).to(DEV)
    y = torch.randint(-2, 3, (RT.route_rows(T, k, E), N), generator=g).to(torch.bfloat16).to(DEV)
    dout = torch.randint(-4, 5, (T, N), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.full((T, k), 1.0, device=DEV)
    got = F.fp8moe_route_weight_grad(dout, y, row_of)
    for j in range(k):
        step = torch.zeros(T, k, device=DEV)
        step[:, j] = 1.0
        d = F.fp8moe_route_unpermute(y, row_of, w + step).double() - F.fp8moe_route_unpermute(y, row_of, w - step).double()
        assert torch.equal((d * dout.double()).sum(1) / 2, got[:, j].double())
