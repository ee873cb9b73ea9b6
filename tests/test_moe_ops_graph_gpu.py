"""The operators around the expert products in a CUDA graph, those among them
that launch a second kernel ahead of the first one's end, and the norm's tiled
output as an operand of a product."""
import numpy as np
import pytest
import torch

from oracle import grouped_mm as OG, moe_ops as OM, quant as OQ

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _replayed(call, inputs, others):
    """``call`` captured, then replayed on the inputs' first contents and on
    other ones: the bits of plain calls, whatever stands in the outputs."""
    flat = lambda r: [t for t in (r if isinstance(r, (tuple, list)) else [r]) if t is not None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flat(call())
    first = [t.clone() for t in inputs]
    for contents in (first, others, first):
        for t, c in zip(inputs, contents):
            t.copy_(c)
        want = [t.clone() for t in flat(call())]
        for _ in range(3):
            for t in out:
                t.view(torch.uint8).fill_(0xA5)
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("T,E,k", [(3, 64, 6), (16, 256, 8), (17, 256, 8), (300, 100, 4), (4096, 256, 8), (9000, 16, 2)])
def test_router(F, T, E, k):
    x, y = torch.randn(T, E, device=DEV), torch.randn(T, E, device=DEV)
    _replayed(lambda: F.fp8moe_router_fwd(x, k), [x], [y])
    idx, w, counts, _, loss = F.fp8moe_router_fwd(x, k)
    _replayed(lambda: F.fp8moe_router_bwd(x, idx, counts, w, loss), [x, w], [y, w + 1])


@pytest.mark.parametrize("T,H", [(1, 64), (5, 7168), (3000, 1024), (40, 16416)])
def test_norm(F, T, H):
    r = lambda: torch.randn(T, H, device=DEV).to(torch.bfloat16)
    x, res, w = r(), r(), torch.rand(H, device=DEV) + 0.5
    _replayed(lambda: F.fp8moe_add_rmsnorm_fwd(x, w, res, recipe=F.MXFP8), [x, res], [r(), r()])
    rstd = torch.rand(T, device=DEV) + 0.5
    _replayed(lambda: F.fp8moe_add_rmsnorm_bwd(x, res, rstd, w), [x, res], [r(), r()])


@pytest.mark.parametrize("M", [96, 20480])
def test_swiglu_and_weight_grad(F, M):
    Fd = 128
    r = lambda n: torch.randn(M, n, device=DEV).to(torch.bfloat16)
    h, d = r(2 * Fd), r(Fd)
    offs = torch.tensor([32, 32, M], dtype=torch.int32, device=DEV)
    lay = (F.GROUP_ROWS, F.GROUP_COLS)
    # (scale padding is written by nobody: kept buffers)
    kept = dict(zip(("q0", "s0", "q1", "s1"), F.fp8moe_swiglu_fwd(h, offs, *lay, dim0=True, dim1=True)[1:]))
    _replayed(lambda: (F.fp8moe_swiglu_fwd(h, offs, *lay, dim0=True, dim1=True, **kept)[0]), [h], [r(2 * Fd)])
    _replayed(lambda: F.fp8moe_swiglu_bwd(d, h), [h, d], [r(2 * Fd), r(Fd)])
    row_of = torch.randperm(M, device=DEV).to(torch.int32).view(-1, 2)
    do = torch.randn(M // 2, Fd, device=DEV).to(torch.bfloat16)
    _replayed(lambda: F.fp8moe_route_weight_grad(do, d, row_of), [d], [r(Fd)])


@pytest.mark.parametrize("T,H", [(32, 128), (96, 256), (288, 1056)])
def test_norm_feeds_a_product(F, T, H):
    """The tiled output is the A operand of a one-group product as it comes."""
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, H, generator=g).to(torch.bfloat16), torch.rand(H, generator=g) + 0.5
    b = (torch.randn(1, 64, H, generator=g) * 0.1).to(torch.bfloat16)
    n = lambda t: t.double().numpy()
    _, _, _, q, s = F.fp8moe_add_rmsnorm_fwd(x.to(DEV), w.to(DEV), eps=1e-5, recipe=F.MXFP8, scale_layout=F.NO_GROUPS,
                                             need_y=False)
    qb, sb, _, _ = F.fp8moe_mxfp8_quantize_dual(b.to(DEV), None, F.NO_GROUPS, F.NO_GROUPS, dim1=False)
    offs = torch.tensor([T], dtype=torch.int32, device=DEV)
    out = F.fp8moe_scaled_grouped_mm_fwd(F.MXFP8, q, s, qb, sb, offs)
    y = OM.add_rmsnorm(n(x), None, n(w), 1e-5)[2]
    deq = lambda v: OQ.dequant_mx(*OQ.mxfp8_quantize_dim0(v))
    ref, bound = OG.grouped_mm_fwd(deq(y), deq(n(b)), np.array([T]))
    # as for the activation's products: a code may round the other way
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= 8e-3 * np.abs(ref) + 2e-3 * bound)
    assert F.fp8moe_get_device_status() == 0
