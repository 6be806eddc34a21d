"""The oracle of the router, the norms around a block and clipping (CPU): values worked
out by hand, and every gradient against central differences of the forward formulas."""
import numpy as np
import pytest

from oracle import block as O

INF = np.inf


def differences(f, x, h=1e-5):
    """Central differences of the scalar f over the array x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        if not np.isfinite(x[i]):
            continue
        at = x[i]
        x[i] = at + h
        hi = f()
        x[i] = at - h
        lo = f()
        x[i] = at
        g[i] = (hi - lo) / (2 * h)
    return g


def test_choices_by_hand():
    x = np.array([[1.0, 3.0, 3.0, -INF], [-INF, -INF, 2.0, -INF], [-INF] * 4, [0.0, -0.0, -5.0, 7.0]])
    assert O.choose(x, 3, False).tolist() == [[1, 2, 0], [2, -1, -1], [-1, -1, -1], [3, 0, 1]]
    assert O.choose(x, 1, True, bias=np.array([0.9, 0.0, 0.1, 0.0])).tolist() == [[0], [2], [-1], [0]]
    assert O.choose(x, 2, False, mask=np.array([0, 1, 1, 0])).tolist() == [[-1, -1], [2, -1], [-1, -1], [-1, -1]]


def test_balance_loss_is_one_when_even_and_grows():
    E, k = 4, 1
    even = np.eye(E) * 1e-9                                   # a choice each, probabilities alike
    ids, w, counts, sums, n, loss = O.route(even, k, False, True, 1.0)
    assert counts.tolist() == [1] * E and n == E and abs(loss - 1) < 1e-6
    one = np.tile(np.array([50.0, 0, 0, 0]), (8, 1))
    assert abs(O.route(one, k, False, True, 1.0)[5] - E) < 1e-6


def test_weights_of_underflowing_scores():
    x = np.array([[-2000.0, -2001.0, -2001.0]])
    w, p = O.route_weights(x, np.array([[1, 2]]), True, True, 1.0)
    assert np.allclose(w, 0.5) and abs(p.sum() - 1) < 1e-12


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("loss", [False, True])
def test_router_gradient(sigmoid, renorm, loss):
    rng = np.random.default_rng(0)
    T, E, k = 6, 7, 3
    x = rng.normal(size=(T, E))
    x[1, 2:] = -INF                                           # two open experts: a choice is missing
    x[2] = -INF
    x[3, 4] = -INF
    ids = O.choose(x, k, sigmoid, mask=np.array([1, 1, 1, 1, 0, 1]))
    dw, dloss = rng.normal(size=(T, k)), 0.7
    counts = np.bincount(ids[ids >= 0], minlength=E)
    n = int((ids >= 0).any(1).sum())

    def f():
        w, p = O.route_weights(x, ids, sigmoid, renorm, 1.5)
        return (w * dw).sum() + (dloss * E / (k * n * n) * (counts * p.sum(0)).sum() if loss else 0)

    dx, mass = O.route_bwd(dw, x, ids, sigmoid, renorm, 1.5, *((dloss, counts, n) if loss else ()))
    assert np.abs(dx - differences(f, x)).max() < 1e-8
    assert (np.abs(dx) <= mass * (1 + 1e-12) + 1e-300).all()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("pre", [False, True])
def test_norm_gradients(post, gate, pre):
    rng = np.random.default_rng(1)
    T, H = 3, 10
    R, Y = rng.normal(size=(T, H)), rng.normal(size=(T, H))
    w_post = rng.normal(size=H) if post else None
    w_pre = rng.normal(size=H) if pre else None
    g = None if gate is None else rng.normal(size=H if gate == "channel" else (T, 1))
    dR, dN = rng.normal(size=(T, H)), rng.normal(size=(T, H))

    def f():
        out, N, _ = O.residual_norm(R, Y, w_post, g, 0.7, w_pre, 1e-3)
        return (out * dR).sum() + ((N * dN).sum() if pre else 0)

    stream = O.residual_norm(R, Y, w_post, g, 0.7, w_pre, 1e-3)[0]
    got = O.residual_norm_bwd(dR, dN if pre else None, stream, Y, w_post, g, 0.7, w_pre, 1e-3)
    for name, x in (("dR", R), ("dY", Y), ("dw_post", w_post), ("dgate", g), ("dw_pre", w_pre)):
        if x is None:
            assert name not in got
            continue
        d, mass = got[name]
        assert d.shape == x.shape and np.abs(d - differences(f, x)).max() < 1e-8
        assert (np.abs(d) <= mass * (1 + 1e-12)).all()


def test_norm_without_a_block():
    R = np.array([[3.0, 4.0]])
    out, N, _ = O.residual_norm(R, w_pre=np.array([1.0, 2.0]), eps=1e-12)
    assert (out == R).all() and np.allclose(N, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])


def test_clip_by_hand():
    assert O.clip([np.array([3.0]), np.array([[4.0]])], 1.0) == (5.0, 0.2)
    assert O.clip([np.array([3.0, 4.0])], 10.0) == (5.0, 1.0)
