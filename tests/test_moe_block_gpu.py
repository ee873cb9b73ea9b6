"""The block that runs the norm, the router, the grouped products and the gated
activation together: gradients against float32 autograd of the same map with
the same choice of experts, and a few training steps.

MXFP8 noise: an e4m3 value is off by 2^-4 at most, 3% rms; a product of two
quantized operands 4%; three of them in a row 7%, so a gradient's direction
keeps a cosine of 0.99 with room."""
import importlib.util
import os

import pytest
import torch

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
    h, out, balance, saved = blk.forward(x, r)
    dx, grads = blk.backward(dout, dh, dbal, saved)
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
    loss = (ref * dout.float()).sum() + (ha * dh.float()).sum() + 3.0 * bal
    loss.backward()
    assert float(balance) == pytest.approx(float(bal.detach()), rel=1e-2)

    def cosine(a, b):
        return float(torch.nn.functional.cosine_similarity(a.detach().float().flatten(), b.detach().float().flatten(), dim=0))

    assert cosine(out, ref) > 0.99 and torch.equal(h, (x.float() + r.float()).to(torch.bfloat16))
    assert cosine(dx, xa.grad) > 0.99
    for n, t in p.items():
        assert grads[n].shape == t.shape and cosine(grads[n], t.grad) > 0.99, n


def test_it_learns(B):
    losses = B.main(30)
    assert losses[-1] < 0.8 * losses[0] and all(b < 1.05 * a for a, b in zip(losses, losses[1:]))
