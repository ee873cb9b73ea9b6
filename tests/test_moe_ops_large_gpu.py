"""Tensors of more than 2^31 elements: the last rows of a large call have the
bits of a small call on those rows alone, and 2^31 bytes past the start
nothing wraps."""
import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda"


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _rand(*shape):
    """Random rows, made once and repeated with another sign and place."""
    base = torch.randn(4096, shape[1], device=DEV).to(torch.bfloat16)
    x = torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
    for i in range(0, shape[0], 4096):
        n = min(4096, shape[0] - i)
        x[i:i + n] = base.roll(i // 4096, 1)[:n]
    return x


def test_norm(F):
    T, H, n = 270000, 8192, 1024     # 2.2e9 elements
    x = _rand(T, H)
    w = 1 + 0.1 * torch.randn(H, device=DEV)
    h, y, rstd, q, s = F.fp8moe_add_rmsnorm_fwd(x, w, x, recipe=F.MXFP8)
    for cut in (slice(T - n, T), slice(131072, 131072 + n)):
        small = F.fp8moe_add_rmsnorm_fwd(x[cut], w, x[cut], recipe=F.MXFP8)
        for a, b in zip((h, y, rstd, q, s), small):
            assert torch.equal(a[cut], b)
    dx, dw = F.fp8moe_add_rmsnorm_bwd(x, h, rstd, w, y)
    cut = slice(T - n, T)
    small, _ = F.fp8moe_add_rmsnorm_bwd(x[cut], h[cut], rstd[cut], w, y[cut])
    assert torch.equal(dx[cut], small) and bool(torch.isfinite(dw).all())


def test_router(F):
    T, E, k, n = 2200000, 1000, 2, 4096   # 2.2e9 logits
    x = _rand(T, E)
    idx, w, counts, _, loss = F.fp8moe_router_fwd(x, k)
    assert int(counts[E]) == T and int(counts[:E].sum()) == T * k
    si, sw, *_ = F.fp8moe_router_fwd(x[T - n:], k)
    assert torch.equal(idx[T - n:], si) and torch.equal(w[T - n:], sw)
    dw = torch.ones(T, k, device=DEV)
    dw[:, 1] = -1
    d = F.fp8moe_router_bwd(x, idx, None, dw)
    assert torch.equal(d[T - n:], F.fp8moe_router_bwd(x[T - n:], si, None, dw[T - n:]))


def test_swiglu(F):
    M, Fd, n = 280000 // 128 * 128, 4096, 256   # 2.3e9 gate and up values
    h = _rand(M, 2 * Fd)
    dout = _rand(M, Fd)
    _, q0, s0, q1, s1 = F.fp8moe_swiglu_bwd(dout, h, None, F.SCALES_ROWMAJOR, F.SCALES_ROWMAJOR, need_dh=False, dim0=True,
                                            dim1=True)
    _, a0, b0, a1, b1 = F.fp8moe_swiglu_bwd(dout[M - n:], h[M - n:], None, F.SCALES_ROWMAJOR, F.SCALES_ROWMAJOR,
                                            need_dh=False, dim0=True, dim1=True)
    assert torch.equal(q0[M - n:], a0) and torch.equal(s0[M - n:], b0)
    assert torch.equal(q1[:, M - n:], a1) and torch.equal(s1[:, (M - n) // 32:], b1)
    assert F.fp8moe_get_device_status() == 0


def test_weight_grad(F):
    T, N, k = 140000, 8192, 2                  # y of 2.3e9 values
    y, dout = _rand(2 * T, N), _rand(T, N)
    row_of = torch.arange(2 * T, device=DEV, dtype=torch.int32).flip(0).reshape(T, k)
    dw = F.fp8moe_route_weight_grad(dout, y, row_of)
    n = 512
    assert torch.equal(dw[:n], F.fp8moe_route_weight_grad(dout[:n], y, row_of[:n]))
    ref = (dout[:n, None, :].double() * y[row_of[:n].long()].double()).sum(-1)
    size = (dout[:n, None, :].double() * y[row_of[:n].long()].double()).abs().sum(-1)
    assert bool(((dw[:n].double() - ref).abs() <= (N / 32 + 16) * 2.0 ** -24 * size).all())
