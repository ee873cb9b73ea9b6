"""The operators around the expert products write inside their outputs and
workspaces only (ragged shapes, so that tails and padding run), whatever stands
beside them."""
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


@pytest.mark.parametrize("T,H", [(1, 160), (77, 96), (130, 1056), (3, 2080), (5, 16416)])
def test_norm(F, T, H):
    g = Guarded()
    x, r, dy = _bf16((T, H), 1), _bf16((T, H), 2), _bf16((T, H), 3)
    w = torch.ones(H, device=DEV)
    F.fp8moe_add_rmsnorm_fwd(x, w, r, recipe=F.MXFP8, h=g((T, H), BF16), y=g((T, H), BF16), rstd=g((T,), F32),
                             q=g((T, H), U8), scale=g((T, H // 32), U8))
    F.fp8moe_add_rmsnorm_fwd(x, w, r, recipe=F.MXFP8, scale_layout=F.NO_GROUPS, h=g((T, H), BF16), y=g((T, H), BF16),
                             rstd=g((T,), F32), q=g((T, H), U8),
                             scale=g((F.fp8moe_swizzled_scales_bytes(1, T, H // 32),), U8))
    F.fp8moe_add_rmsnorm_fwd(x, w, recipe=F.ROWWISE, y=g((T, H), BF16), rstd=g((T,), F32), q=g((T, H), U8),
                             scale=g((T,), F32))
    g.check("forward")
    rstd = torch.ones(T, device=DEV)
    nws = F.fp8moe_add_rmsnorm_bwd_workspace_bytes(T, H)
    for dh in (None, r):
        F.fp8moe_add_rmsnorm_bwd(dy, x, rstd, w, dh, dx=g((T, H), BF16), dweight=g((H,), F32), workspace=g((nws,), U8))
    g.check("backward")


@pytest.mark.parametrize("T,E,k", [(1, 3, 2), (15, 33, 5), (17, 60, 4), (700, 250, 8), (9, 1000, 11)])
def test_router(F, T, E, k):
    g = Guarded()
    for x in (torch.randn(T, E, device=DEV), torch.randn(T, E, device=DEV).to(BF16)):
        nws = F.fp8moe_router_workspace_bytes(T, E)
        idx, w, counts, _, loss = F.fp8moe_router_fwd(
            x, k, topk_idx=g((T, k), I32), topk_w=g((T, k), F32), counts=g((E + 1,), I32), prob_sum=g((E,), F32),
            balance_loss=g((1,), F32), workspace=g((nws,), U8))
        F.fp8moe_router_bwd(x, idx, counts, w, loss, dlogits=g((T, E), x.dtype))
    g.check("router")
    y, dout = _bf16((T * k, 264), 1), _bf16((T, 264), 2)
    row_of = torch.arange(T * k, device=DEV, dtype=I32).reshape(T, k)
    F.fp8moe_route_weight_grad(dout, y, row_of, dw=g((T, k), F32))
    g.check("weight gradient")


@pytest.mark.parametrize("M,Fd", [(32, 32), (160, 96), (9824, 416)])
def test_swiglu(F, M, Fd):
    g = Guarded()
    h, dout = _bf16((M, 2 * Fd), 1), _bf16((M, Fd), 2)
    offs = torch.tensor([0, 32, 32, M], dtype=I32, device=DEV)
    size = F.fp8moe_swizzled_scales_bytes
    for W, call in ((Fd, lambda **kw: F.fp8moe_swiglu_fwd(h, offs, F.GROUP_ROWS, F.GROUP_COLS, **kw)),
                    (2 * Fd, lambda **kw: F.fp8moe_swiglu_bwd(dout, h, offs, F.GROUP_ROWS, F.GROUP_COLS, **kw))):
        call(dim0=True, dim1=True, out=g((M, W), BF16), q0=g((M, W), U8), q1=g((W, M), U8),
             s0=g((size(1, M, W // 32, 4, F.GROUP_ROWS),), U8), s1=g((size(1, W, M // 32, 4, F.GROUP_COLS),), U8))
    n = M - 5   # a ragged last row block, rows alone
    F.fp8moe_swiglu_fwd(h[:n], None, F.SCALES_ROWMAJOR, dim0=True, out=g((n, Fd), BF16), q0=g((n, Fd), U8),
                        s0=g((n, Fd // 32), U8))
    g.check("gated activation")
    assert F.fp8moe_get_device_status() == 0


@pytest.mark.parametrize("T", [1, 3, 40, 3000])
def test_new_results_are_apart(F, T):
    """Results that a call allocates are contiguous, aligned, do not overlap and
    outlive one another."""
    H, E, k = 512, 64, 6
    x, w = torch.randn(T, H, device=DEV).to(torch.bfloat16), torch.ones(H, device=DEV)
    h2 = torch.randn(32 * T, 2 * H, device=DEV).to(torch.bfloat16)
    logits = torch.randn(T, E, device=DEV)
    rstd = torch.ones(T, device=DEV)
    calls = [lambda: F.fp8moe_add_rmsnorm_fwd(x, w, x, recipe=F.MXFP8, need_y=True, need_rstd=True),
             lambda: F.fp8moe_add_rmsnorm_fwd(x, w, recipe=F.ROWWISE, need_y=True, need_rstd=True),
             lambda: F.fp8moe_add_rmsnorm_bwd(x, x, rstd, w),
             lambda: F.fp8moe_router_fwd(logits, k),
             lambda: F.fp8moe_swiglu_fwd(h2, dim0=True, dim1=True)]
    for call in calls:
        first = [t for t in call() if t is not None]
        want = [t.clone() for t in first]
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in first)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in first)
        for i, t in enumerate(first):
            t.zero_()
            assert all(torch.equal(a, b) for a, b in zip(first[i + 1:], want[i + 1:]))
        first = [t for t in call() if t is not None]
        last = first[-1]
        first = None
        call()
        torch.cuda.synchronize()
        assert torch.equal(last, want[-1])
