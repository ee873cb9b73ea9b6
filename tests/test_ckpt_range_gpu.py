"""The ends of fp32's range in the backward passes from MXFP8 checkpoints."""
import pytest
import torch

from test_canaries_gpu import DEV, Guarded

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _pack(F, h):
    """(codes, scales, the values as bf16) of h."""
    q, s = F.fp8moe_mxfp8_quantize_dim0(h)
    v = q.view(torch.float8_e4m3fn).float().view(h.shape[0], -1, 32) * torch.exp2(s.float() - 127)[..., None]
    return q, s, v.view(h.shape).to(BF16)


@pytest.mark.parametrize("T,N,k", [(1, 32, 1), (3, 64, 2), (50, 7168, 8), (700, 128, 3), (5000, 768, 5), (33, 4128, 7), (20, 480, 13)])
def test_weight_grad_of_large_gradients(F, T, N, k):
    """dout times a code is beyond fp32, their products with the scales are not.  Sums of
    N products: at most N / 16 + 16 additions a lane, each off by 2^-24."""
    g = torch.Generator(device=DEV).manual_seed(N + T)
    rows = T * k + 3
    yq, ys, y = _pack(F, torch.randn(rows, N, device=DEV, generator=g).mul_(2.0 ** -24).to(BF16))
    dout = torch.randn(T, N, device=DEV, generator=g).to(BF16)
    big = torch.rand(T, N, device=DEV, generator=g) < 0.3
    big[T // 2 + 1:] &= torch.rand(T - T // 2 - 1, 1, device=DEV, generator=g) < 0.5   # (and some tokens without)
    dout[big] *= 2.0 ** 124
    row_of = torch.randperm(rows, device=DEV, generator=g)[:T * k].reshape(T, k).to(I32)
    row_of[T // 2, k - 1] = rows
    if T > 2:
        row_of[0, 0] = -1
        yq[row_of[1, 0].long(), 5] = 0x7F
    got = F.fp8moe_route_weight_grad_ckpt(dout, yq, ys, row_of).double()
    there = (row_of >= 0) & (row_of < rows)
    d, size = dout.double(), torch.zeros(T, k, dtype=torch.float64, device=DEV)
    ref = torch.zeros_like(size)
    for j in range(k):
        p = d * y[row_of[:, j].long().clamp(0, rows - 1)].double()
        ref[:, j], size[:, j] = p.sum(1), p.abs().sum(1)
    if T > 2:
        assert bool(got[1, 0].isnan())
        got[1, 0], there[1, 0] = 0.0, False
    assert not got[~there].any() and bool(torch.isfinite(got).all())
    assert bool(((got - ref).abs() <= (N / 16 + 16) * 2.0 ** -24 * size)[there].all())
    # the bf16 call on the same values
    bf = F.fp8moe_route_weight_grad(dout, y, row_of).double()
    assert bool(((got - bf).abs() <= (N / 8 + 32) * 2.0 ** -24 * size)[there].all())


@pytest.mark.parametrize("M,Fd", [(7, 64), (33, 160), (20001, 160)])
def test_activation_far_in_the_last_rows(F, M, Fd):
    """Rows that are no whole block, with gates beyond the exponential, products beyond
    fp32, NaN codes and NaN scales among the last of them: the bf16 call's results, and
    nothing past the outputs."""
    g = torch.Generator(device=DEV).manual_seed(M)
    h = torch.randn(M, 2 * Fd, device=DEV, generator=g).mul_(2.0).to(BF16)
    h[M - 1, :32], h[M - 2, Fd:Fd + 32], h[M - 3, :64] = -300.0, 3e38, -2e38
    hq, hs, v = _pack(F, h)
    hq[M - 4, 5], hs[M - 5, 1], hs[M - 1, Fd // 32] = 0x7F, 255, 255
    v[M - 4, 5] = v[M - 5, 32:64] = v[M - 1, Fd:Fd + 32] = float("nan")
    dout = torch.randn(M, Fd, device=DEV, generator=g).to(BF16)
    dout[M - 2] *= 1e4
    for layout in (F.SCALES_ROWMAJOR, F.NO_GROUPS):
        n = M * Fd // 16 if layout == F.SCALES_ROWMAJOR else F.fp8moe_swizzled_scales_bytes(1, M, Fd // 16, 0, F.NO_GROUPS)
        guard = Guarded()
        s0 = guard((M, Fd // 16) if layout == F.SCALES_ROWMAJOR else (n,), U8)
        s0.zero_()
        got = F.fp8moe_swiglu_bwd_ckpt(dout, hq, hs, None, layout, dim0=True, out=guard((M, 2 * Fd), BF16),
                                       q0=guard((M, 2 * Fd), U8), s0=s0)[:3]
        want = F.fp8moe_swiglu_bwd(dout, v, None, layout, dim0=True)[:3]
        guard.check("far rows")
        assert torch.equal(got[0].isnan(), want[0].isnan())
        assert torch.equal(torch.nan_to_num(got[0], 7.0), torch.nan_to_num(want[0], 7.0))
        assert torch.equal(got[1] & 0x7F, want[1] & 0x7F) and torch.equal(got[2].view(-1), want[2].view(-1))   # (a NaN's sign is not told)
    assert F.fp8moe_get_device_status() == 0
