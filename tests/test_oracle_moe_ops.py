"""The oracles of the operators around the expert products: gradients against
central differences of their forwards, closed forms and small cases by hand."""
import numpy as np
import pytest

from oracle import moe_ops as OM


def _differences(f, x, g, step=1e-6):
    """d <f(x), g> / dx by central differences, element by element."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        for sign in (1.0, -1.0):
            y = x.copy()
            y[i] += sign * step
            out[i] += sign * float(np.sum(f(y) * g)) / (2 * step)
    return out


def test_norm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    x, r, w = rng.normal(size=(3, 8)), rng.normal(size=(3, 8)), rng.normal(size=8)
    dy, dh = rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    a, rstd, _ = OM.add_rmsnorm(x, r, w, 1e-3)
    dx, dw = OM.add_rmsnorm_grad(dy, a, rstd, w, dh)
    both = lambda v: OM.add_rmsnorm(v, r, w, 1e-3)
    num = _differences(lambda v: both(v)[2], x, dy) + _differences(lambda v: both(v)[0], x, dh)
    assert np.allclose(dx, num, atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: OM.add_rmsnorm(x, r, v, 1e-3)[2], w, dy), atol=1e-7)
    # the norm ignores the row's length: dx without dh is orthogonal to a up to eps
    one, _ = OM.add_rmsnorm_grad(dy, a, 1 / np.sqrt(np.mean(a * a, axis=1)), w)
    assert np.allclose(np.sum(one * a, axis=1), 0.0, atol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_is_the_difference_quotient(score, renorm):
    rng = np.random.default_rng(2)
    T, E, k = 4, 6, 3
    x = rng.normal(size=(T, E))
    x[1, 2] = -np.inf
    mask = np.array([1, 1, 0, 1])
    f = OM.router(x, k, score, renorm, 2.5, rng.normal(size=E) * 0.1, mask)
    dw, dloss = rng.normal(size=(T, k)), 1.7
    d = OM.router_grad(x, f["idx"], f["counts"], f["tokens"], dw, dloss, score, renorm, 2.5, mask)

    def value(v):
        o = OM.router(v, k, score, renorm, 2.5, token_mask=mask, idx=f["idx"])
        # the counts are constants of the gradient
        loss = E / (k * o["tokens"] ** 2) * np.dot(f["counts"], o["prob_sum"])
        return np.array(np.sum(o["w"] * dw) + dloss * loss)

    num = np.zeros_like(x)
    for t in range(T):
        for e in range(E):
            if np.isfinite(x[t, e]):
                for sign in (1.0, -1.0):
                    y = x.copy()
                    y[t, e] += sign * 1e-6
                    num[t, e] += sign * float(value(y)) / 2e-6
    assert np.allclose(d, num, atol=1e-7)
    assert np.all(d[2] == 0.0) and d[1, 2] == 0.0


def test_router_small_cases():
    # ties to the lowest id, a masked expert last with weight 0 and no count
    f = OM.router(np.array([[1.0, 2.0, 2.0, -np.inf]]), 4, "softmax", False, 1.0)
    assert f["idx"].tolist() == [[1, 2, 0, 3]]
    assert f["w"][0, 3] == 0.0 and f["counts"].tolist() == [1, 1, 1, 0]
    # uniform routing has loss 1 whatever k
    f = OM.router(np.zeros((4, 4)), 4, "sigmoid", True, 1.0)
    assert f["loss"] == pytest.approx(1.0) and np.allclose(f["w"], 0.25)
    # nothing left: the lowest ids, zero weights, no tokens counted
    f = OM.router(np.full((2, 3), -np.inf), 2, "softmax", True, 1.0)
    assert f["idx"].tolist() == [[0, 1], [0, 1]] and not f["w"].any() and f["loss"] == 0.0


def test_swiglu_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(3)
    h, d = rng.normal(size=(3, 8)) * 2, rng.normal(size=(3, 4))
    assert np.allclose(OM.swiglu_grad(d, h), _differences(OM.swiglu, h, d), atol=1e-7)
    assert OM.swiglu(np.array([[-1e4, 3.0]]))[0, 0] == 0.0


def test_weight_grad_by_hand():
    y = np.array([[1.0, 2.0], [3.0, 4.0]])
    assert OM.weight_grad(np.array([[1.0, 10.0]]), y, np.array([[1, -1, 0]])).tolist() == [[43.0, 0.0, 21.0]]
