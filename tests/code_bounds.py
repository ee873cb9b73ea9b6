"""Bounds on rounded outputs whose input is known to a tolerance: rounding is
monotone, so the code (or bf16) of a value within [v - tol, v + tol] lies
between those of the two ends."""
import numpy as np
import torch

from oracle import formats as OF


def _between(q, lo, hi, kind, what):
    got = OF.decode(q, kind)
    low, high = OF.decode(OF.encode(lo, kind), kind), OF.decode(OF.encode(hi, kind), kind)
    bad = ~((low <= got) & (got <= high))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes outside, first at {np.argwhere(bad)[0]}"


def check_bf16(got, v, tol, what):
    """bf16 tensor ``got`` of values v known to tol."""
    v = np.asarray(v, np.float64)
    low, high = (torch.from_numpy(np.asarray(e, np.float32)).to(torch.bfloat16).float().numpy()
                 for e in (v - tol, v + tol))
    g = got.float().cpu().numpy()
    bad = ~((low <= g) & (g <= high))
    assert got.dtype == torch.bfloat16 and not bad.any(), f"{what}: {int(bad.sum())} outside, first at {np.argwhere(bad)[0]}"


def check_mx(q, byte, v, tol, what):
    """Codes q [.., C] and e8m0 bytes [.., C / 32] of values v known to tol."""
    v = np.asarray(v, np.float64)
    tol = np.broadcast_to(tol, v.shape)
    blocks = lambda a: a.reshape(a.shape[:-1] + (a.shape[-1] // 32, 32))
    a = np.abs(blocks(v))
    low = OF.e8m0_from_amax(np.maximum(a - blocks(tol), 0.0).max(-1))
    high = OF.e8m0_from_amax((a + blocks(tol)).max(-1))
    assert np.all((low <= byte) & (byte <= high)), f"{what}: scale bytes"
    e = np.repeat(byte.astype(np.int64) - 127, 32, axis=-1)
    scale = np.ldexp(1.0, (-e).astype(np.int32))
    _between(q, (v - tol) * scale, (v + tol) * scale, OF.FN, what)


def check_rows(q, inv, v, rel, kind, what):
    """Rowwise codes q [R, C] and scales inv [R] of values v known to a relative error."""
    v = np.asarray(v, np.float64)
    ref = np.maximum(np.abs(v).max(axis=1), 1e-12) / OF.FP8_MAX[kind]
    assert np.all(np.abs(inv - ref) <= (rel + 2.0 ** -22) * ref), f"{what}: scales"
    x = v / ref[:, None]
    tol = (2 * rel + 2.0 ** -21) * np.abs(x)
    _between(q, x - tol, x + tol, kind, what)
