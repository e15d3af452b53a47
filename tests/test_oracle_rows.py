"""The oracle's row plan, router, expert products and adapters against closed
forms and brute force (parity unpinned: the pages describe none of them)."""
import numpy as np

from oracle import rows as R


def test_group_rows_worked_example():
    offsets, order, pos = R.group_rows([2, 0, -1, 2, 5, 0], 4)
    assert offsets.tolist() == [0, 2, 2, 4, 4]
    assert order.tolist() == [1, 5, 0, 3, -1, -1]
    assert pos.tolist() == [2, 0, -1, 3, -1, 1]


def test_route_ties_masks_and_weights():
    inf = np.inf
    ids, w = R.moe_route([[1.0, 3.0, 3.0, -inf], [-inf, np.nan, -inf, 2.0], [-inf] * 4, [inf, 0.0, 0.0, inf]], 2, True)
    assert ids.tolist() == [[1, 2], [3, -1], [-1, -1], [0, 3]]
    assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]])
    ids, w = R.moe_route([[0.0, np.log(3.0)]], 1, False)
    assert ids.tolist() == [[1]] and np.allclose(w, [[0.75]])


def test_expert_products_brute_force():
    g = np.random.default_rng(1)
    codes, s = g.integers(-127, 128, (3, 5, 8)), g.random((3, 5)) + 1
    x, ids = g.standard_normal((4, 8)), np.array([[2, 0], [0, -1], [2, 1], [0, 2]])
    offsets, order, pos = R.group_rows(ids, 3)
    y = R.y_experts(codes, s, x, offsets, order, 2)
    w = g.random((4, 2))
    out = R.y_combine(y, pos, w)
    for t in range(4):
        want = np.zeros(5)
        for j in range(2):
            e = ids[t, j]
            if e >= 0:
                row = np.array([sum(codes[e, n, k] * x[t, k] for k in range(8)) / s[e, n] for n in range(5)])
                assert np.allclose(y[pos[t * 2 + j]], row)
                want += w[t, j] * row
        assert np.allclose(out[t], want)
    assert np.all(np.isnan(y[offsets[-1]:]))
    s_x = g.random(4) + 1
    assert np.allclose(R.y_experts(codes, s, x, offsets, order, 2, s_x)[0], y[0] / s_x[order[0] // 2])
    ordered = x[order[:offsets[-1]] // 2]
    assert np.allclose(R.y_experts(codes, s, ordered, offsets, None, 1), y[:offsets[-1]])


def test_swiglu_limits():
    assert np.allclose(R.y_swiglu(np.array([0.0, 1e4, -1e4]), np.array([3.0, 2.0, 2.0])), [0, 2e4, 0])


def test_lora_brute_force():
    g = np.random.default_rng(2)
    x, a, b = g.standard_normal((3, 4)), g.standard_normal((2, 2, 4)), g.standard_normal((2, 5, 2))
    d = R.lora_delta(x, [1, -1, 2], a, b, [2.0, 3.0])
    want = [3.0 * sum(b[1, n, r] * a[1, r, k] * x[0, k] for r in range(2) for k in range(4)) for n in range(5)]
    assert np.allclose(d[0], want) and not d[1:].any()
