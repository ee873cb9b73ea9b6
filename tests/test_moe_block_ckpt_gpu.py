"""The block that trains with its activations kept in MXFP8 and answers a few
tokens at a time: gradients against float32 autograd with the same choice of
experts, the few-token call against the definition on the weights it reads, and
both in one program.

MXFP8 noise as in the block's other test; a checkpoint adds an e4m3 rounding, 3%
rms, to factors of products that have 7%: a cosine of 0.99 keeps its room."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from code_bounds import check_bf16
from oracle import formats as OF, moe_ops as OM, swizzle as OS

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from mxfp8_moe_quantization_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients(B, score):
    F = B.F
    T, H, N, E, k = 384, 256, 128, 6, 2
    s = F.SCORE_SOFTMAX if score == "softmax" else F.SCORE_SIGMOID
    blk = B.MoeBlock(H, N, E, k, score=s, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=g)
    x, r, dout, dh = (rand(T, H).to(torch.bfloat16) for _ in range(4))
    dbal = torch.full((1,), 3.0, device="cuda")
    h, out, balance, saved = blk.forward(x, r, checkpoint=True)
    dx, grads = blk.backward(dout, dh, dbal, saved)
    h0, out0, balance0, _ = blk.forward(x, r)
    assert torch.equal(h, h0) and torch.equal(out, out0) and torch.equal(balance, balance0)
    assert F.fp8moe_get_device_status() == 0
    idx, counts = saved[4].long(), saved[6][:E].float()

    p = {n: getattr(blk, n).float().requires_grad_() for n in ("norm", "router", "w1", "w2")}
    xa = x.float().requires_grad_()
    ha = xa + r.float()
    y = ha * torch.rsqrt(ha.square().mean(1, keepdim=True) + blk.eps) * p["norm"]
    logits = y @ p["router"].t()
    sc = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    prob = sc / sc.sum(1, keepdim=True)
    w = sc.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    ref = 0
    for j in range(k):
        w1, w2 = p["w1"][idx[:, j]], p["w2"][idx[:, j]]
        ga, up = torch.einsum("tnh,th->tn", w1, y).chunk(2, 1)
        ref = ref + w[:, j:j + 1] * torch.einsum("thn,tn->th", w2, torch.nn.functional.silu(ga) * up)
    bal = E / (k * T * T) * (counts * prob.sum(0)).sum()
    ((ref * dout.float()).sum() + (ha * dh.float()).sum() + 3.0 * bal).backward()
    cosine = lambda a, b: float(torch.nn.functional.cosine_similarity(a.detach().float().flatten(), b.float().flatten(), dim=0))
    assert cosine(dx, xa.grad) > 0.99
    for n, t in p.items():
        assert grads[n].shape == t.shape and cosine(grads[n], t.grad) > 0.99, n


def _value(q, s):
    E, N, K = q.shape
    rp, cp = OS.swizzled_shape(N, K // 32, 0, -1)
    byte = np.stack([OS.unswizzle(m, rp, cp)[:N, :K // 32] for m in s.cpu().numpy().reshape(E, -1)])
    return (OF.decode(q.cpu().numpy(), OF.FN).reshape(E, N, K // 32, 32) *
            np.ldexp(1.0, byte.astype(np.int32) - 127)[..., None]).reshape(E, N, K)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_decode(B, T):
    """The layer's definition on the norm's and the router's own outputs; a masked
    row is zero whatever it holds."""
    F = B.F
    H, N, E, k = 256, 160, 12, 3
    blk = B.MoeBlock(H, N, E, k, seed=8)
    g = torch.Generator(device="cuda").manual_seed(T)
    x, r = (torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    if T > 1:
        mask[T // 2] = 0
        x[T // 2] = float("nan")
    weights = blk.serving_weights()
    _, out = blk.decode(x, r, weights, mask)
    assert F.fp8moe_get_device_status() == 0
    _, y, _, _, _ = F.fp8moe_add_rmsnorm_fwd(x, blk.norm, r, eps=blk.eps)
    idx, w, _, _, _ = F.fp8moe_router_fwd(y.float() @ blk.router.t(), k, score=blk.score, token_mask=mask, need_balance=False)
    ref, bound = OM.moe_decode(torch.nan_to_num(y).double().cpu().numpy(), idx.cpu().numpy(), w.cpu().numpy(),
                               _value(*weights[:2]), _value(*weights[2:]), (256 / 32 + 64) * 2.0 ** -22, 2.0 ** -12 + 2.0 ** -20)
    check_bf16(out, ref, bound + 1e-30, "out")
    assert T == 1 or not out[T // 2].any()


def test_it_runs_with_checkpoints(B):
    losses = B.main(3, checkpoint=True)
    assert len(losses) == 3 and all(np.isfinite(losses))
