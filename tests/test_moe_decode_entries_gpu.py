"""The few tokens' layer to both sides of its rules: how many choices a reading of an
expert serves, where terms are made on the way, one accumulator or two."""
import pytest
import torch

from test_ckpt_decode_edges_gpu import DEV, I32, _decode_ok, _layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _spread(args, hot):
    """Distinct choices of a token; the first of `hot` tokens the same."""
    T, E = args[0].shape[0], args[5].shape[0]
    k = args[1].shape[1]
    g = torch.Generator(device=DEV).manual_seed(hot)
    args[1] = torch.rand(T, E, device=DEV, generator=g)[:, 1:].topk(k, 1)[1].to(I32) + 1
    args[1][:hot, 0] = 0
    return args


@pytest.mark.parametrize("T,H,Fd,E,k,hot", [(60, 64, 512, 1000, 2, 7), (60, 64, 512, 1000, 2, 8), (60, 64, 512, 1000, 2, 9),
                                            (12, 96, 160, 256, 2, 0), (9, 544, 96, 64, 1, 3), (30, 96, 4128, 512, 1, 8),
                                            (20, 1056, 96, 200, 2, 8)])
def test_terms_on_the_way_of_many_tokens(F, T, H, Fd, E, k, hot):
    """Few pairs an entry on average, one entry of up to eight and one more."""
    _decode_ok(F, _spread(_layer(F, T, H, Fd, E, k, seed=T), hot))


@pytest.mark.parametrize("T,E,k", [(20, 5, 4), (21, 5, 4), (20, 2, 1), (21, 2, 1), (24, 2, 1), (25, 2, 1), (26, 2, 1), (48, 2, 1), (50, 2, 1),
                                   (40, 64, 4), (32, 1, 1), (63, 1, 1), (64, 1, 1), (65, 1, 1), (129, 1, 1)])
@pytest.mark.parametrize("H,Fd", [(64, 96), (288, 32)])
def test_entries_of_every_kind(F, T, E, k, H, Fd):
    args = _layer(F, T, H, Fd, E, k, seed=T + E)
    _decode_ok(F, args)
    args[1].zero_()          # all the same expert, as many entries as that takes
    _decode_ok(F, args)


@pytest.mark.parametrize("T", [20, 21, 32, 33, 60, 64, 70])
@pytest.mark.parametrize("E", [1, 3])
def test_many_row_tiles_of_a_cta(F, T, E):
    """Its accumulators are used again, with as many columns as an entry has."""
    args = _layer(F, T, 65536, 64, E, 1, seed=T)
    args[1].fill_(E - 1)
    _decode_ok(F, args)
    args = _layer(F, T, 64, 32768, E, 1, seed=T)
    args[1].fill_(E - 1)
    _decode_ok(F, args)


def test_streams_of_two_priorities(F):
    """Calls in flight at once, some of which go first, beside other kernels: the bits
    of calls alone."""
    one, few = _layer(F, 1, 2048, 1408, 8, 6), _layer(F, 20, 256, 512, 6, 2)
    want = [F.fp8moe_mxfp8_moe_decode(*one), F.fp8moe_mxfp8_moe_decode(*few)]
    x = torch.randn(4096, 2048, device=DEV).to(torch.bfloat16)
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1, 0)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        got.append((F.fp8moe_mxfp8_moe_decode(*one, stream=streams[0]), want[0]))
        got.append((F.fp8moe_mxfp8_moe_decode(*few, stream=streams[1]), want[1]))
        if i % 4 == 0:
            F.fp8moe_quantize_tensorwise(x, stream=streams[2])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got) and F.fp8moe_get_device_status() == 0
