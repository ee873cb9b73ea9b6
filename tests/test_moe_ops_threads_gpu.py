"""Calls of two host threads at once, through the C ABI (which runs without the
interpreter's lock): neither refuses the other's."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _together(calls, seconds=4.0):
    """Every call again and again on a stream of its own; the set of statuses each gave."""
    import time
    end, seen, streams = time.time() + seconds, [set() for _ in calls], [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(i):
        n = 0
        while time.time() < end and seen[i] <= {0}:
            seen[i].add(calls[i](streams[i].cuda_stream))
            n += 1
            if n % 64 == 0:
                streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return seen


def test_norm_backward_of_two_row_lengths(F):
    """The same kernel with a deep ring and with a shallow one."""
    def call(T, H):
        dy, h = (torch.randn(T, H, device=DEV).to(torch.bfloat16) for _ in range(2))
        rstd, w = torch.ones(T, device=DEV), torch.ones(H, dtype=torch.bfloat16, device=DEV)
        dx, dw = torch.empty_like(dy), torch.empty(H, device=DEV)
        ws = torch.empty(F.fp8moe_add_rmsnorm_bwd_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
        keep = (dy, h, rstd, w, dx, dw, ws)
        p = [t.data_ptr() for t in keep]

        def run(stream):
            assert keep
            return F.lib().fp8moe_add_rmsnorm_bwd(p[0], p[1], p[2], p[3], 0, None, T, H, p[4], p[5], p[6], ws.numel(), stream)
        return run, keep

    (a, ka), (b, kb) = call(160, 8192), call(160, 2080)
    assert _together([a, b]) == [{0}, {0}]
    # and their results are those of calls alone
    for run, keep in ((a, ka), (b, kb)):
        dx, dw = keep[4].clone(), keep[5].clone()
        assert run(None) == 0
        torch.cuda.synchronize()
        assert torch.equal(dx, keep[4]) and torch.equal(dw, keep[5])


def test_scale_swizzle_of_two_widths(F):
    """Rows of 16-byte multiples, one kernel for every width."""
    def call(R, Cs):
        s = torch.randint(0, 255, (R, Cs), dtype=torch.uint8, device=DEV)
        out = torch.empty(F.fp8moe_swizzled_scales_bytes(1, R, Cs), dtype=torch.uint8, device=DEV)
        return lambda stream: F.lib().fp8moe_swizzle_scales_128x4(s.data_ptr(), 1, R, Cs, None, 0, F.NO_GROUPS, out.data_ptr(),
                                                                  stream)

    assert _together([call(256, 384), call(256, 16)]) == [{0}, {0}]
