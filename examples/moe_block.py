"""A trained MoE block on MXFP8 products, forward and backward, from this
package's calls alone (PyTorch holds the memory and computes the router's
small linear layer).

    h = x + residual;  y = rmsnorm(h) * g
    logits = y Wr^T;   ids, weights, balance loss = router(logits)
    rows = y, permuted to the experts;  out = sum_j weights_j W2_e (swiglu(W1_e rows))

    python examples/moe_block.py          # a few SGD steps on a small task
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mxfp8_moe_quantization_gb300 as F  # noqa: E402


class MoeBlock:
    """Parameters and one step of the block: H features, E experts of width
    N (gate and up: 2N rows of W1), k experts a token."""

    def __init__(self, H: int, N: int, E: int, k: int, score: int = F.SCORE_SIGMOID, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device=device, generator=g)
        self.E, self.k, self.score, self.eps = E, k, score, 1e-5
        self.norm = torch.ones(H, device=device)
        self.router = rand(E, H) * H ** -0.5
        self.w1 = (rand(E, 2 * N, H) * H ** -0.5).to(torch.bfloat16)
        self.w2 = (rand(E, H, N) * N ** -0.5).to(torch.bfloat16)

    def forward(self, x, residual):
        """x, residual [T, H] bf16 -> (h, out, balance loss, saved)."""
        h, y, rstd, _, _ = F.fp8moe_add_rmsnorm_fwd(x, self.norm, residual, eps=self.eps)
        logits = y.float() @ self.router.t()
        idx, w, counts, _, balance = F.fp8moe_router_fwd(logits, self.k, score=self.score)
        rows, offs, row_of = F.fp8moe_route_permute(y, idx, self.E)
        qa, sa, qat, sat = F.fp8moe_mxfp8_quantize_dual(rows, offs, F.GROUP_ROWS, F.GROUP_COLS)
        qw1, sw1, qw1t, sw1t = F.fp8moe_mxfp8_quantize_dual(self.w1)
        qw2, sw2, qw2t, sw2t = F.fp8moe_mxfp8_quantize_dual(self.w2)
        gu = F.fp8moe_scaled_grouped_mm_fwd(F.MXFP8, qa, sa, qw1, sw1, offs)
        _, qh, sh, qht, sht = F.fp8moe_swiglu_fwd(gu, offs, F.GROUP_ROWS, F.GROUP_COLS, need_out=False, dim0=True,
                                                  dim1=True)
        rows2 = F.fp8moe_scaled_grouped_mm_fwd(F.MXFP8, qh, sh, qw2, sw2, offs)
        out = F.fp8moe_route_unpermute(rows2, row_of, w)
        saved = (h, y, rstd, logits, idx, w, counts, offs, row_of, qat, sat, qw1t, sw1t, qw2t, sw2t, gu, qht, sht, rows2)
        return h, out, balance, saved

    def backward(self, dout, dh, dbalance, saved):
        """Gradients of out, of h and of the balance loss ([1] fp32) -> (gradient
        of x and of residual, {parameter: gradient})."""
        (h, y, rstd, logits, idx, w, counts, offs, row_of, qat, sat, qw1t, sw1t, qw2t, sw2t, gu, qht, sht, rows2) = saved
        M = rows2.shape[0]
        dw = F.fp8moe_route_weight_grad(dout, rows2, row_of)
        dlogits = F.fp8moe_router_bwd(logits, idx, counts, dw, dbalance, score=self.score)
        drows2, _, _ = F.fp8moe_route_permute(dout, idx, self.E, w)
        qd, sd, qdt, sdt = F.fp8moe_mxfp8_quantize_dual(drows2, offs, F.GROUP_ROWS, F.GROUP_COLS)
        dact = F.fp8moe_scaled_grouped_mm_dgrad(F.MXFP8, qd, sd, qw2t, sw2t, offs)
        dw2 = F.fp8moe_scaled_grouped_mm_wgrad(F.MXFP8, qdt, sdt, qht, sht, offs, M)
        _, qg, sg, qgt, sgt = F.fp8moe_swiglu_bwd(dact, gu, offs, F.GROUP_ROWS, F.GROUP_COLS, need_dh=False, dim0=True,
                                                  dim1=True)
        drows = F.fp8moe_scaled_grouped_mm_dgrad(F.MXFP8, qg, sg, qw1t, sw1t, offs)
        dw1 = F.fp8moe_scaled_grouped_mm_wgrad(F.MXFP8, qgt, sgt, qat, sat, offs, M)
        dy = F.fp8moe_route_unpermute(drows, row_of).float() + dlogits @ self.router
        dx, dnorm = F.fp8moe_add_rmsnorm_bwd(dy.to(torch.bfloat16), h, rstd, self.norm, dh)
        return dx, {"norm": dnorm, "router": dlogits.t() @ y.float(), "w1": dw1, "w2": dw2}


def main(steps: int = 30) -> list:
    """The block learns another block's map; returns the losses."""
    T, H, N, E, k = 1024, 256, 128, 8, 2
    teacher, block = MoeBlock(H, N, E, k, seed=1), MoeBlock(H, N, E, k, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    r = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    want = teacher.forward(x, r)[1].float()
    alpha = torch.full((1,), 0.01, device="cuda")   # weight of the balance loss
    scale = 1024.0                                  # keeps the bf16 gradients' range
    rate = {"norm": 4.0, "router": 4.0, "w1": 80.0, "w2": 80.0}
    losses = []
    for _ in range(steps):
        _, out, balance, saved = block.forward(x, r)
        err = out.float() - want
        losses.append(float(err.square().mean() + alpha * balance))
        dout = (2.0 * scale / want.numel() * err).to(torch.bfloat16)
        _, grads = block.backward(dout, None, alpha * scale, saved)
        for name, d in grads.items():
            p = getattr(block, name)
            p.copy_(p.float() - rate[name] / scale * d.float())
    assert F.fp8moe_get_device_status() == 0
    return losses


if __name__ == "__main__":
    for i, loss in enumerate(main()):
        print(f"step {i:3d}  loss {loss:.5f}")
