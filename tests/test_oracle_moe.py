"""The mixture-of-experts oracle against hand values and differences (CPU)."""
import numpy as np
import pytest

from oracle import moe as O


def test_sort_by_hand():
    ids = np.array([[2, 0], [2, -1], [0, 2], [7, 2]])           # 3 experts; -1 and 7 are dropped
    offs, counts, row_slot, slot_row = O.sort(ids, 3, 4, 12)
    assert offs.tolist() == [0, 4, 4, 12] and counts.tolist() == [2, 0, 4]
    assert row_slot.tolist() == [1, 4, -1, -1, 0, 2, 5, 7, -1, -1, -1, -1]
    assert slot_row.tolist() == [[4, 0], [5, -1], [1, 6], [-1, 7]]


def test_rows_needed_is_enough_and_reached():
    rng = np.random.default_rng(0)
    for T, k, G, align in [(1, 1, 5, 128), (3, 2, 4, 128), (200, 2, 3, 128), (7, 3, 64, 1)]:
        need = O.rows_needed(T, k, G, align)
        worst = 0
        for _ in range(200):
            c = np.bincount(rng.integers(0, G, T * k), minlength=G)
            worst = max(worst, int((-(-c // align) * align).sum()))
        assert worst <= need
    assert O.rows_needed(3, 1, 3, 128) == 384 and O.rows_needed(0, 2, 8, 128) == 0


def test_pow2_scale_by_hand():
    x = np.zeros((1, 300))
    x[0, 0], x[0, 130], x[0, 256] = 448.0, 448.0 * (1 + 2.0 ** -30), 1e-60
    codes, s = O.quantise(x, True)
    assert s.tolist() == [[1.0, 2.0, 2.0 ** -126]]
    assert codes[0, 0] == 0x7E and codes[0, 130] == 0x76 and codes[0, 256] == 0


@pytest.mark.parametrize("g0", [-30.0, -1.2784645, -0.5, 0.0, 3.0, 25.0])
def test_swiglu_gradient_is_the_difference_quotient(g0):
    rng = np.random.default_rng(1)
    g, u, da = g0 + rng.standard_normal(20), rng.standard_normal(20), rng.standard_normal(20)
    dg, du, _ = O.swiglu_bwd(da, g, u)
    h = 1e-5
    ng = da * (O.swiglu(g + h, u) - O.swiglu(g - h, u)) / (2 * h)
    nu = da * (O.swiglu(g, u + h) - O.swiglu(g, u - h)) / (2 * h)
    # central differences: h^2 / 6 times the third derivative (below 1 here) plus cancellation 1e-16 |a| / h
    scale = np.abs(da) * (1 + np.abs(u)) * (1 + np.abs(g))
    assert np.all(np.abs(dg - ng) <= 1e-9 * scale) and np.all(np.abs(du - nu) <= 1e-9 * scale)


def test_combine_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(2)
    ids = np.array([[0, 1], [1, -1], [0, 0]])
    _, _, _, slot_row = O.sort(ids, 2, 1, 6)
    y, w, d = rng.standard_normal((6, 5)), rng.standard_normal((3, 2)), rng.standard_normal((3, 5))
    dy, dw, _ = O.combine_bwd(d, y, slot_row, w)
    f = lambda y, w: float((O.combine(y, slot_row, w)[0] * d).sum())
    h = 1e-4                                                     # f is linear in each argument: only cancellation
    for i in np.ndindex(y.shape):
        yp, ym = y.copy(), y.copy()
        yp[i] += h
        ym[i] -= h
        assert abs((f(yp, w) - f(ym, w)) / (2 * h) - dy[i]) < 1e-9
    for i in np.ndindex(w.shape):
        wp, wm = w.copy(), w.copy()
        wp[i] += h
        wm[i] -= h
        assert abs((f(y, wp) - f(y, wm)) / (2 * h) - dw[i]) < 1e-9


def test_wgrad_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(3)
    offs, counts = np.array([0, 4, 4, 8]), np.array([3, 0, 2])
    x, dy, w = rng.standard_normal((8, 3)), rng.standard_normal((8, 2)), rng.standard_normal((3, 2, 3))
    dw, _ = O.wgrad(dy, x, offs, counts)
    expert = np.array([0, 0, 0, -1, 2, 2, -1, -1])

    def f(w):
        return sum(float((x[r] @ w[e].T) @ dy[r]) for r, e in enumerate(expert) if e >= 0)

    for i in np.ndindex(w.shape):
        wp, wm = w.copy(), w.copy()
        wp[i] += 1e-4
        wm[i] -= 1e-4
        assert abs((f(wp) - f(wm)) / 2e-4 - dw[i]) < 1e-9
