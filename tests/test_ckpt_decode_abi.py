"""Host-side checks of the calls on MXFP8 checkpoints and of the few tokens'
expert layer: refused before any CUDA call (no GPU needed), and the workspace
sizes."""
import pytest

OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
P = 1 << 20          # aligned, never dereferenced
MIS = P + 8
ROWMAJOR, PLAIN, GROUP_ROWS, GROUP_COLS = -2, -1, 0, 1


@pytest.fixture(scope="module")
def lib():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as F
    return F.lib()


def _decode(lib, **kw):
    a = dict(x=P, ldx=64, idx=P, w=P, T=4, k=2, w1=P, s1=P, w2=P, s2=P, E=8, H=64, F=96, out=P, workspace=P, nbytes=1 << 40,
             stream=None)
    a.update(kw)
    return lib.fp8moe_mxfp8_moe_decode(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(T=513, k=2), INVALID), (dict(T=1, k=1025), INVALID), (dict(E=0), INVALID),
    (dict(E=1025), INVALID), (dict(H=0, ldx=0), INVALID), (dict(F=0), INVALID), (dict(H=(1 << 20) + 32, ldx=1 << 21), INVALID),
    (dict(F=(1 << 20) + 32), INVALID), (dict(E=1024, T=512, H=1 << 20, ldx=1 << 20, F=1 << 20), INVALID), (dict(ldx=56), INVALID),
    (dict(H=48, ldx=48), ALIGN), (dict(F=80), ALIGN), (dict(ldx=68), ALIGN),
    (dict(x=None), INVALID), (dict(idx=None), INVALID), (dict(w=None), INVALID), (dict(w1=None), INVALID), (dict(s1=None), INVALID),
    (dict(w2=None), INVALID), (dict(s2=None), INVALID), (dict(out=None), INVALID), (dict(workspace=None), INVALID),
    (dict(nbytes=0), INVALID), (dict(x=MIS), ALIGN), (dict(w1=MIS), ALIGN), (dict(s1=MIS), ALIGN), (dict(w2=MIS), ALIGN),
    (dict(s2=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(workspace=MIS), ALIGN), (dict(idx=P + 2), ALIGN), (dict(w=P + 2), ALIGN),
    (dict(T=0, x=None, idx=None, w=None, workspace=None, nbytes=0), OK)])
def test_decode(lib, kw, code):
    assert _decode(lib, **kw) == code


def test_decode_workspace(lib):
    """Exactly what is asked for is enough, one byte less is not."""
    size = lib.fp8moe_mxfp8_moe_decode_workspace_bytes
    for bad in ((-1, 2, 8, 64, 96), (4, 0, 8, 64, 96), (4, 2, 0, 64, 96), (4, 2, 8, 48, 96), (4, 2, 8, 64, 80), (1024, 2, 8, 64, 96)):
        assert size(*bad) == -1
    assert size(0, 2, 8, 64, 96) == 0
    for T, k, E, H, F in ((4, 2, 8, 64, 96), (1, 8, 256, 7168, 2048), (64, 16, 16, 5120, 8192)):
        n = size(T, k, E, H, F)
        assert n > 0
        assert _decode(lib, T=T, k=k, E=E, H=H, ldx=H, F=F, nbytes=n - 1) == INVALID
        # at least the two products' sums of every pair
        assert n >= T * k * (2 * F + H) * 4


def test_decode_partial_sums_fit(lib):
    """The partial sums of any routing stay inside the workspace: a tile's parts,
    counted from the runs of the streams as they are cut, times the live pairs."""
    size = lib.fp8moe_mxfp8_moe_decode_workspace_bytes
    up = lambda a, b: (a + b - 1) // b
    pieces = lambda K: up(up(K, 128), 2)

    def parts(ents, R, K, grid):
        rt, kp = up(R, 128), pieces(K)
        C = ents * rt * kp
        want = (C + 1) // 2
        runs = min(want, grid)
        base = (2 if C == 2 * runs else 1) if want < grid else C // grid
        rest = C - base * runs
        owner = lambda c: c // (base + 1) if c < rest * (base + 1) else rest + (c - rest * (base + 1)) // base
        return max(owner(t * kp + kp - 1) - owner(t * kp) + 1 for t in range(ents * rt))

    for T, k, E, H, F in ((1, 6, 64, 2048, 1408), (2, 2, 4, 4128, 64), (23, 8, 256, 512, 256), (64, 16, 16, 1056, 352), (5, 3, 7, 96, 160)):
        each = T * k // E
        nb = 2 if T < 2 else T if T <= 24 else 24 if each <= 14 else 32 if each <= 24 else 64
        total = size(T, k, E, H, F)
        for n in {1, 2, T, T * k // 2 + 1, T * k}:
            for ents in {up(n, nb), min(n, E), min(n, E) + n // nb}:
                if up(n, nb) <= ents:
                    for grid in (148, 152, 160):
                        need = n * 4 * (parts(ents, 2 * F, H, grid) * 2 * F + parts(ents, H, F, grid) * H)
                        assert need <= total, (T, k, E, H, F, n, ents, grid)


def _fwd(lib, **kw):
    a = dict(h=P, ldh=128, M=64, F=64, offs=P, E=2, out=P, q0=P, s0=P, l0=GROUP_ROWS, q1=P, s1=P, l1=GROUP_COLS, hq=P, hs=P,
             stream=None)
    a.update(kw)
    return lib.fp8moe_swiglu_fwd_ckpt(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(F=0, ldh=0), INVALID), (dict(ldh=120), INVALID), (dict(h=None), INVALID), (dict(hq=None), INVALID),
    (dict(hs=None), INVALID), (dict(s0=None), INVALID), (dict(q1=None), INVALID), (dict(l0=GROUP_COLS), INVALID),
    (dict(offs=None), INVALID), (dict(E=0), INVALID), (dict(F=48, ldh=96), ALIGN), (dict(M=40), ALIGN), (dict(h=MIS), ALIGN),
    (dict(hq=MIS), ALIGN), (dict(q0=MIS), ALIGN), (dict(M=0, h=None, hq=None, hs=None), OK)])
def test_swiglu_forward(lib, kw, code):
    assert _fwd(lib, **kw) == code


def _bwd(lib, **kw):
    a = dict(dout=P, hq=P, hs=P, M=64, F=64, offs=P, E=2, dh=P, q0=P, s0=P, l0=GROUP_ROWS, q1=P, s1=P, l1=GROUP_COLS, aq1=P, as1=P,
             stream=None)
    a.update(kw)
    return lib.fp8moe_swiglu_bwd_ckpt(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(F=0), INVALID), (dict(F=(1 << 28) + 32), INVALID), (dict(dout=None), INVALID), (dict(hq=None), INVALID),
    (dict(hs=None), INVALID), (dict(aq1=None), INVALID), (dict(as1=None), INVALID), (dict(s0=None), INVALID), (dict(s1=None), INVALID),
    (dict(l1=GROUP_ROWS), INVALID), (dict(q1=None, s1=None, l1=GROUP_ROWS), INVALID), (dict(offs=None), INVALID),
    (dict(dh=None, q0=None, s0=None, q1=None, s1=None, aq1=None, as1=None), INVALID),
    (dict(F=48), ALIGN), (dict(M=40), ALIGN), (dict(M=40, q0=None, s0=None, q1=None, s1=None), ALIGN), (dict(dout=MIS), ALIGN),
    (dict(hq=MIS), ALIGN), (dict(aq1=MIS), ALIGN), (dict(dh=MIS), ALIGN), (dict(offs=P + 2), ALIGN), (dict(M=0, dout=None, hq=None), OK)])
def test_swiglu_backward(lib, kw, code):
    assert _bwd(lib, **kw) == code


def _norm(lib, **kw):
    a = dict(dy=P, hq=P, hs=P, rstd=P, w=P, weight_type=0, dh=P, T=4, H=64, dx=P, dw=P, workspace=P, nbytes=1 << 20, stream=None)
    a.update(kw)
    return lib.fp8moe_add_rmsnorm_bwd_ckpt(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(weight_type=-1), INVALID), (dict(dy=None), INVALID), (dict(hq=None), INVALID),
    (dict(hs=None), INVALID), (dict(rstd=None), INVALID), (dict(w=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID),
    (dict(workspace=None), INVALID), (dict(nbytes=4 * 64 * 4 - 1), INVALID), (dict(H=40), ALIGN), (dict(dy=MIS), ALIGN),
    (dict(hq=MIS), ALIGN), (dict(dh=MIS), ALIGN), (dict(dx=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(rstd=P + 1), ALIGN)])
def test_norm_backward(lib, kw, code):
    assert _norm(lib, **kw) == code


def _grad(lib, **kw):
    a = dict(dout=P, yq=P, ys=P, rows=8, row_of=P, T=4, N=64, k=2, dw=P, stream=None)
    a.update(kw)
    return lib.fp8moe_route_weight_grad_ckpt(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(N=-32), INVALID), (dict(k=0), INVALID), (dict(rows=-1), INVALID), (dict(rows=(1 << 31) + 1), INVALID),
    (dict(T=1 << 30), INVALID), (dict(N=1 << 31), INVALID), (dict(dout=None), INVALID), (dict(yq=None), INVALID), (dict(ys=None), INVALID),
    (dict(row_of=None), INVALID), (dict(dw=None), INVALID), (dict(N=48), ALIGN), (dict(dout=MIS), ALIGN), (dict(yq=MIS), ALIGN),
    (dict(row_of=P + 2), ALIGN), (dict(dw=P + 2), ALIGN), (dict(T=0, dout=None, yq=None), OK)])
def test_weight_grad(lib, kw, code):
    assert _grad(lib, **kw) == code
