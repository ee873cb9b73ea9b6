"""Host-side checks of the weight gradient that knows y's rows (no GPU needed)."""
import pytest

OK, INVALID, ALIGN = 0, 1, 2
P = 1 << 20          # aligned, never dereferenced


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(rows=(1 << 31) + 1), INVALID), (dict(y=None), INVALID), (dict(dout=None), INVALID),
    (dict(row_of=None), INVALID), (dict(dw=None), INVALID), (dict(k=0), INVALID), (dict(N=60), ALIGN), (dict(y=P + 8), ALIGN),
    (dict(dw=P + 2), ALIGN), (dict(T=0), OK), (dict(T=0, y=None, rows=0), OK)])
def test_refusals(kw, code):
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as F
    a = dict(dout=P, y=P, rows=4, row_of=P, T=4, N=64, k=2, dw=P, stream=None)
    a.update(kw)
    assert F.lib().fp8moe_route_weight_grad_bounded(*a.values()) == code
