"""What the few tokens' expert layer keeps of its values between the products, on
layers whose exact results are known.

The activation goes to the second product in four e4m3 terms of five bits, each off
by at most half a step: 2^-19 of itself; its sigmoid, a product and an fp32 sum of
two products add less than 2^-20."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def F():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as m
    return m


def _codes(v):
    """e4m3 codes of values that are e4m3 numbers."""
    q = v.float().to(torch.float8_e4m3fn)
    assert torch.equal(q.float(), v.float())
    return q.view(torch.uint8).to(DEV)


def _ones(F, E, R, K):
    return torch.full((F.fp8moe_swizzled_scales_bytes(E, R, K // 32, 0, F.NO_GROUPS),), 127, dtype=torch.uint8, device=DEV)


def _layer(F, x, idx, w1, w2):
    """The call on E times the same expert, all scales and weights 1."""
    E = int(idx.max()) + 1
    many = lambda m: _codes(m).expand(E, *m.shape).contiguous()
    out = F.fp8moe_mxfp8_moe_decode(x.to(DEV), idx.to(DEV), torch.ones(idx.shape, device=DEV), many(w1), _ones(F, E, *w1.shape),
                                    many(w2), _ones(F, E, *w2.shape))
    assert F.fp8moe_get_device_status() == 0
    return out.double().cpu().numpy()


def _choices(T, E):
    idx = torch.arange(T, dtype=torch.int32)[:, None] % E
    idx[-1] = E - 1
    return idx


@pytest.mark.parametrize("T,E", [(1, 1), (1, 3), (6, 4), (8, 1), (23, 4), (40, 4), (100, 4), (200, 4)])
def test_digits_of_the_activation(F, T, E):
    """Outputs are differences of two neighbouring activations that agree in their
    first digits.  Gates are 64, whose sigmoid is 1 to 2^-92; up is a sum of integers
    below 2^24, exact in any order."""
    g = torch.Generator().manual_seed(T + E)
    H, Fd = 64, 64
    x = torch.zeros(T, H)
    x[:, 0] = 64.0
    x[:, 32:63] = torch.randint(-255, 256, (T, 31), generator=g).float()
    x[:, 63] = torch.randint(-127, 128, (T,), generator=g).float()
    w1 = torch.zeros(2 * Fd, H)
    w1[:Fd, 0] = 1.0
    up = torch.randint(8, 16, (Fd // 2, 31), generator=g) * 2 ** torch.randint(0, 5, (Fd // 2, 31), generator=g)
    up = up * (1 - 2 * torch.randint(0, 2, up.shape, generator=g))
    w1[Fd::2, 32:63] = w1[Fd + 1::2, 32:63] = up.float()
    w1[Fd + 1::2, 63] = 1.0
    w2 = torch.zeros(H, Fd)
    pair = torch.arange(H) % (Fd // 2)
    w2[torch.arange(H), 2 * pair], w2[torch.arange(H), 2 * pair + 1] = -1.0, 1.0
    out = _layer(F, x.to(BF16), _choices(T, E), w1, w2)
    a = 64.0 * (x.double() @ w1[Fd:].double().t()).numpy()
    ref = np.broadcast_to(64.0 * x[:, 63:].double().numpy(), out.shape)
    first, second = np.abs(a)[:, 2 * pair], np.abs(a)[:, 2 * pair + 1]
    # the terms of both, and the bf16 output's rounding
    tol = 2.0 ** -18 * (first + second)
    assert np.all(np.abs(out - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))


GATES = [0.0, 1.0, -1.0, 30.0, -30.0, 90.0, -79.5, -80.0, -80.5, -87.0, -88.0, -88.5, -89.0, -92.0, -100.0, -120.0, -150.0, -180.0,
         -194.0, -200.0, -260.0, -300.0, -1e4, -1e20, -3e38]


@pytest.mark.parametrize("up", [1.0, -3.5, 1e19, 2.0 ** 100, 3e38])
@pytest.mark.parametrize("T", [1, 8, 0])
def test_far_gates(F, up, T):
    """silu(g) u for gates to both sides of where the sigmoid leaves fp32: 2^-15 of
    itself below -80, where the exponent's argument is rounded; what each of the four
    terms has below fp32's normal numbers may be lost."""
    gates = torch.tensor(GATES).to(BF16)
    gates = gates[gates * up < 1e38] if up > 0 else gates   # (a product beyond fp32 is not a number)
    H, Fd = 64, 32
    w1, w2 = torch.zeros(2 * Fd, H), torch.zeros(H, Fd)
    w1[:Fd, 0], w1[Fd:, 32] = 1.0, 1.0
    w2[torch.arange(H), torch.arange(H) % Fd] = 1.0
    for part in gates.split(T or len(gates)):
        x = torch.zeros(len(part), H)
        x[:, 0], x[:, 32] = part.float(), up
        x = x.to(BF16)
        out = _layer(F, x, _choices(len(part), 4), w1, w2)
        g, u = x[:, 0].double().numpy(), x[:, 32].double().numpy()
        with np.errstate(over="ignore"):
            ref = (g / (1.0 + np.exp(-g)) * u)[:, None]
        tol = 2.0 ** -15 * np.abs(ref) + 2.0 ** -124
        assert np.all(np.abs(out - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)), (part, out[:, 0], ref)


def test_long_sums_are_not_cut_off_far(F):
    """The tensor core cuts its sums off after every 32 products, by less than 2^-23 of
    the sum so far; a chain of eight pieces has 64 such steps and here a quarter of the
    first half's sum S at its end, half of that on average.  Eight chains: 2^-17 S, and a tenth
    more as they are not alike.  The second half is the first with the other sign, so that
    the output is what was cut off.  (One chain of 512 steps: up to 2^-15 S.)"""
    H, Fd = 152 * 128, 16384
    half = Fd // 2
    g = torch.Generator(device=DEV).manual_seed(1)
    codes = lambda *s: torch.randint(0, 0x7F, s, dtype=torch.uint8, device=DEV, generator=g)
    w1, w2 = torch.zeros(1, 2 * Fd, H, dtype=torch.uint8, device=DEV), torch.empty(1, H, Fd, dtype=torch.uint8, device=DEV)
    w2[0, :, :half] = codes(H, half)
    w2[0, :, half:] = w2[0, :, :half] | 0x80
    up = codes(half, 31)
    w1[0, :Fd, 0] = 0x38                                        # gates of 64
    w1[0, Fd:Fd + half, 32:63] = w1[0, Fd + half:, 32:63] = up
    x = torch.zeros(1, H, device=DEV)
    x[0, 0], x[0, 32:63] = 64.0, torch.rand(31, device=DEV, generator=g) + 0.5
    x = x.to(BF16)
    out = F.fp8moe_mxfp8_moe_decode(x, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, 1, device=DEV), w1,
                                    _ones(F, 1, 2 * Fd, H), w2, _ones(F, 1, H, Fd))
    assert F.fp8moe_get_device_status() == 0
    a = 64.0 * (up.view(torch.float8_e4m3fn).double() @ x[0, 32:63].double())
    S = torch.cat([w2[0, r:r + 2432, :half].view(torch.float8_e4m3fn).double() @ a for r in range(0, H, 2432)])
    assert bool((out[0].double().abs() <= 1.1 * 2.0 ** -17 * S).all())
