"""Host-side checks of the operators around the expert products: refused
before any CUDA call (no GPU needed), and the workspace sizes."""
import ctypes

import pytest

OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
P = 1 << 20          # aligned, never dereferenced
MIS = P + 8
MX, ROW, BLOCKWISE = 1, 0, 3
ROWMAJOR, PLAIN, GROUP_ROWS, GROUP_COLS = -2, -1, 0, 1


@pytest.fixture(scope="module")
def lib():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as F
    return F.lib()


def _norm(lib, **kw):
    a = dict(x=P, ldx=64, residual=P, ldr=64, w=P, weight_type=0, T=4, H=64, eps=1e-5, h=P, y=P, rstd=P, recipe=MX, kind=0,
             q=P, scale=P, scale_layout=ROWMAJOR, stream=None)
    a.update(kw)
    return lib.fp8moe_add_rmsnorm_fwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0, ldx=0), INVALID), (dict(ldx=32), INVALID), (dict(ldr=32), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(weight_type=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(scale=None), INVALID),
    (dict(q=None), INVALID), (dict(residual=None), INVALID),            # h without a residual
    (dict(h=None, y=None, rstd=None, q=None, scale=None), INVALID),     # nothing asked for
    (dict(H=(1 << 20) + 32, ldx=1 << 21, ldr=1 << 21), INVALID), (dict(kind=5), INVALID),
    (dict(recipe=BLOCKWISE), UNSUP), (dict(recipe=MX, kind=1), UNSUP),
    (dict(scale_layout=GROUP_ROWS), INVALID),
    (dict(H=40, ldx=40, ldr=40), ALIGN), (dict(H=24, ldx=24, ldr=24, recipe=ROW), ALIGN),
    (dict(H=60, ldx=64), ALIGN), (dict(ldx=68), ALIGN), (dict(ldr=68), ALIGN), (dict(x=MIS), ALIGN),
    (dict(residual=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(h=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(q=MIS), ALIGN),
    (dict(rstd=P + 2), ALIGN), (dict(recipe=ROW, scale=P + 2), ALIGN),
    (dict(T=0), OK), (dict(T=0, h=None, y=None, rstd=None, q=None, scale=None, x=None), OK)])
def test_norm_forward(lib, kw, code):
    assert _norm(lib, **kw) == code


def _norm_bwd(lib, **kw):
    a = dict(dy=P, h=P, rstd=P, w=P, weight_type=0, dh=P, T=4, H=64, dx=P, dw=P, workspace=P, nbytes=1 << 20, stream=None)
    a.update(kw)
    return lib.fp8moe_add_rmsnorm_bwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(weight_type=-1), INVALID), (dict(dy=None), INVALID),
    (dict(h=None), INVALID), (dict(rstd=None), INVALID), (dict(w=None), INVALID), (dict(dx=None), INVALID),
    (dict(dw=None), INVALID), (dict(workspace=None), INVALID), (dict(nbytes=4 * 64 * 4 - 1), INVALID),
    (dict(H=60), ALIGN), (dict(dy=MIS), ALIGN), (dict(h=MIS), ALIGN), (dict(dh=MIS), ALIGN), (dict(dx=MIS), ALIGN),
    (dict(w=MIS), ALIGN), (dict(workspace=MIS), ALIGN), (dict(rstd=P + 1), ALIGN), (dict(dw=P + 2), ALIGN)])
def test_norm_backward(lib, kw, code):
    assert _norm_bwd(lib, **kw) == code


def _router(lib, **kw):
    a = dict(logits=P, logits_type=1, T=4, E=16, ldl=16, k=2, score=0, renormalize=1, scale=1.0, bias=None, mask=None,
             idx=P, w=P, counts=P, psum=P, loss=P, workspace=P, nbytes=1 << 20, stream=None)
    a.update(kw)
    return lib.fp8moe_router_fwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025, ldl=1025), INVALID), (dict(ldl=15), INVALID),
    (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(E=64, ldl=64, k=33), INVALID), (dict(logits_type=2), INVALID),
    (dict(score=2), INVALID), (dict(logits=None), INVALID), (dict(idx=None), INVALID), (dict(w=None), INVALID),
    (dict(counts=None), INVALID), (dict(psum=None, loss=None), INVALID), (dict(workspace=None), INVALID),
    (dict(nbytes=4 * 33 * 4 - 1), INVALID), (dict(T=1 << 30), INVALID),
    (dict(logits=P + 2), ALIGN), (dict(bias=P + 2), ALIGN), (dict(idx=P + 1), ALIGN), (dict(w=P + 2), ALIGN),
    (dict(counts=P + 2), ALIGN), (dict(psum=P + 2), ALIGN), (dict(loss=P + 2), ALIGN), (dict(workspace=P + 2), ALIGN),
    (dict(T=0, counts=None, psum=None, loss=None, logits=None, idx=None, w=None, workspace=None), OK)])
def test_router_forward(lib, kw, code):
    assert _router(lib, **kw) == code


def _router_bwd(lib, **kw):
    a = dict(logits=P, logits_type=1, T=4, E=16, ldl=16, k=2, score=0, renormalize=1, scale=1.0, mask=None, idx=P, counts=P,
             dw=P, dloss=P, dlogits=P, stream=None)
    a.update(kw)
    return lib.fp8moe_router_bwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), INVALID), (dict(ldl=8), INVALID), (dict(dw=None, dloss=None), INVALID), (dict(dlogits=None), INVALID),
    (dict(idx=None), INVALID), (dict(counts=None), INVALID), (dict(logits=None), INVALID),
    (dict(dlogits=P + 2), ALIGN), (dict(logits_type=0, logits=P + 2, dlogits=P + 1), ALIGN), (dict(dw=P + 2), ALIGN),
    (dict(T=0), OK)])
def test_router_backward(lib, kw, code):
    assert _router_bwd(lib, **kw) == code


@pytest.mark.parametrize("a,code", [
    ((P, P, P, -1, 64, 2, P), INVALID), ((P, P, P, 4, 64, 0, P), INVALID), ((None, P, P, 4, 64, 2, P), INVALID),
    ((P, P, None, 4, 64, 2, P), INVALID), ((P, P, P, 4, 64, 2, None), INVALID), ((P, P, P, 4, 60, 2, P), ALIGN),
    ((MIS, P, P, 4, 64, 2, P), ALIGN), ((P, MIS, P, 4, 64, 2, P), ALIGN), ((P, P, P + 2, 4, 64, 2, P), ALIGN),
    ((P, P, P, 0, 64, 2, P), OK)])
def test_weight_grad(lib, a, code):
    assert lib.fp8moe_route_weight_grad(*a, None) == code


def _swiglu(lib, bwd, **kw):
    a = dict(dout=P, h=P, ldh=128, M=64, F=64, offs=P, E=2, out=P, q0=P, s0=P, l0=GROUP_ROWS, q1=P, s1=P, l1=GROUP_COLS,
             stream=None)
    a.update(kw)
    if not bwd:
        del a["dout"]
    return (lib.fp8moe_swiglu_bwd if bwd else lib.fp8moe_swiglu_fwd)(*a.values())


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(F=0), INVALID), (dict(ldh=127), INVALID), (dict(h=None), INVALID),
    (dict(out=None, q0=None, s0=None, q1=None, s1=None), INVALID), (dict(s0=None), INVALID), (dict(q1=None), INVALID),
    (dict(l0=GROUP_COLS), INVALID), (dict(l1=GROUP_ROWS), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID),
    (dict(offs=None), INVALID), (dict(F=48, ldh=96), ALIGN), (dict(ldh=132), ALIGN), (dict(M=48), ALIGN),
    (dict(M=48, q1=None, s1=None), ALIGN), (dict(h=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(q0=MIS), ALIGN),
    (dict(q1=MIS), ALIGN), (dict(offs=P + 2), ALIGN), (dict(M=0), OK)])
def test_swiglu(lib, bwd, kw, code):
    assert _swiglu(lib, bwd, **kw) == code
    if bwd:
        assert _swiglu(lib, True, dout=None) == INVALID and _swiglu(lib, True, dout=MIS) == ALIGN


def test_workspaces(lib):
    assert lib.fp8moe_add_rmsnorm_bwd_workspace_bytes(3, 64) == 3 * 64 * 4
    assert lib.fp8moe_add_rmsnorm_bwd_workspace_bytes(1 << 20, 64) == 512 * 64 * 4
    assert lib.fp8moe_add_rmsnorm_bwd_workspace_bytes(-1, 64) == -1
    assert lib.fp8moe_router_workspace_bytes(3, 16) == 3 * 33 * 4
    assert lib.fp8moe_router_workspace_bytes(1 << 20, 16) == 512 * 33 * 4
    assert lib.fp8moe_router_workspace_bytes(4, 0) == -1


def test_binding_refuses_foreign_arguments():
    """The binding checks types and shapes before it asks for a pointer."""
    import torch

    import mxfp8_moe_quantization_gb300 as F
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    for call in (lambda: F.fp8moe_add_rmsnorm_fwd(cpu, w), lambda: F.fp8moe_add_rmsnorm_bwd(cpu, cpu, w[:4], w),
                 lambda: F.fp8moe_router_fwd(cpu, 2), lambda: F.fp8moe_swiglu_fwd(cpu),
                 lambda: F.fp8moe_swiglu_bwd(None, cpu),
                 lambda: F.fp8moe_router_bwd(cpu, torch.zeros(4, 2, dtype=torch.int32), dtopk_w=w),
                 lambda: F.fp8moe_route_weight_grad(cpu, cpu, torch.zeros(4, 2, dtype=torch.int32))):
        with pytest.raises(F.Fp8MoeError):
            call()
