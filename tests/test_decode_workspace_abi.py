"""The few tokens' layer's workspace, region by region (no GPU needed): partial sums of
the first product, of the second, terms.

A product whose K is one piece (256) has one partial sum a tile, so that its region is
pairs x rows x 4 bytes; with the terms' bytes taken off as well, what is left is the other
product's region alone."""
import pytest

X_TERMS, ACT_TERMS = 2, 4


@pytest.fixture(scope="module")
def lib():
    from mxfp8_moe_quantization_gb300 import build as B
    B.build()
    import mxfp8_moe_quantization_gb300 as F
    return F.lib()


def _up(a, b):
    return (a + b - 1) // b


def _pieces(K):
    return _up(_up(K, 128), 2)


def _entry(T, k, E):
    each = T * k // E
    return 2 if T < 2 else T if T <= 20 else 20 if each <= 12 else 32 if each <= 24 else 64


def _terms(T, k, E, H, F):
    """Per tile of 128 of K: a row of 128 bytes a term, rounded up to 8 rows an entry, and
    up to 1024 bytes of scales an entry."""
    P = T * k
    ents = min(P, E) + P // _entry(T, k, E)
    per = lambda K, n: _pieces(K) * 2 * ((n * P + 7 * ents) * 128 + 1024 * ents)
    return max(per(H, X_TERMS), per(F, ACT_TERMS))


def _most_parts(ents, R, K, grid):
    """Runs that meet a tile, the most over a stream's tiles, as the streams are cut."""
    kp = _pieces(K)
    C = ents * _up(R, 128) * kp
    want = (C + 1) // 2
    runs = min(want, grid)
    base = (2 if C == 2 * runs else 1) if want < grid else C // grid
    rest = C - base * runs
    owner = lambda c: c // (base + 1) if c < rest * (base + 1) else rest + (c - rest * (base + 1)) // base
    return max(owner(t + kp - 1) - owner(t) + 1 for t in range(0, C, kp))


# T, k, E and K, R of the product under test
CASES = [(1, 6, 64, 2048, 2816), (2, 2, 4, 4128, 64), (8, 4, 9, 1056, 320), (20, 2, 3, 5120, 128), (23, 8, 256, 512, 512),
         (64, 1, 16, 5120, 512), (64, 8, 8, 2048, 256), (64, 16, 60, 1056, 704), (5, 3, 7, 8224, 128), (1, 1, 1, 65536, 64)]


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("T,k,E,K,R", CASES)
def test_partial_sums_have_room(lib, T, k, E, K, R, first):
    """For every number of live pairs and of entries that a routing can give."""
    other = min(R // 2 if first else R, 256)       # the other product's K: one piece
    H, F = (K, other) if first else (other, K)
    rows = (2 * F, H) if first else (H, 2 * F)      # of this product and of the other
    P, nb = T * k, _entry(T, k, E)
    region = lib.fp8moe_mxfp8_moe_decode_workspace_bytes(T, k, E, H, F) - _terms(T, k, E, H, F) - P * rows[1] * 4
    counts = sorted({1, 2, nb, nb + 1, P // 2, P - 1, P} & set(range(1, P + 1)))
    most = 0
    for n in counts:
        # at least a full entry each; at most an entry an expert, and one more for every full one
        for ents in range(_up(n, nb), min(n, min(n, E) + n // nb) + 1):
            for grid in (148, 152, 160):
                need = _most_parts(ents, rows[0], K, grid) * n * rows[0] * 4
                assert need <= region, (n, ents, grid)
                most = max(most, need)
    assert 2 * most >= region      # (a bound, not more than twice what some routing needs)


def test_terms_are_counted_as_they_lie(lib):
    """Entries in a row, each behind those before it: the last byte of the last entry."""
    for T, k, E, H, F in ((1, 6, 64, 2048, 1408), (23, 8, 256, 512, 256), (64, 8, 8, 2048, 4096), (64, 16, 60, 96, 1056)):
        nb = _entry(T, k, E)
        for K, n in ((H, X_TERMS), (F, ACT_TERMS)):
            tiles = _pieces(K) * 2
            for sizes in ([nb] * (T * k // nb), [1] * min(T * k, E), [min(nb, T * k)]):
                first = 0
                for e, pairs in enumerate(sizes):
                    rows = _up(n * pairs, 8) * 8
                    scales = rows * 16 if rows <= 32 else 512 if rows <= 128 else 1024
                    at = tiles * ((n * first + 7 * e) * 128 + 1024 * e)
                    first += pairs
                    end = at + tiles * (rows * 128 + scales)
                    assert end <= tiles * ((n * first + 7 * (e + 1)) * 128 + 1024 * (e + 1)) <= _terms(T, k, E, H, F)
