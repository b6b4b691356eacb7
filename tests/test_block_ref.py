"""The plain references of block_ref.py against values written by hand and against
independent forms (CPU)."""
import numpy as np

from tests import block_ref as R


def test_int8_rows_by_hand():
    v = np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5], [0, 0, 0, 0, -0.0, 0],
                  [1, np.inf, 0, 0, 0, 0], [1, np.nan, 0, 0, 0, 0], [-254, 3, 1, 5, 0, 2]], np.float32)
    q, s = R.int8_rows(v)
    assert q[0].tolist() == [127, -127, 0, 2, 2, 0] and s[0] == 1
    assert q[1].tolist() == [0] * 6 and s[1] == 0
    assert (q[2:4] == 0).all() and np.isnan(s[2:4]).all()
    assert q[4].tolist() == [-127, 2, 0, 2, 0, 1] and s[4] == 2  # 1.5 -> 2, 0.5 -> 0, 2.5 -> 2


def test_int8_rows_are_the_nearest_and_hold_at_the_ends_of_the_range():
    g = np.random.default_rng(1)
    for e in (-149, -140, -126, -101, -100, -20, 0, 60, 126):
        v = np.float32(g.standard_normal((4, 64))) * np.float32(2.0) ** np.float32(min(e, 120))
        v = np.ldexp(v, max(e, 120) - 120 if e > 120 else 0).astype(np.float32)
        q, s = R.int8_rows(v)
        top = np.abs(v).max(-1)
        live = top > 0
        assert (np.abs(q[live]).max(-1) == 127).all() and np.abs(q.astype(int)).max() <= 127
        exact = v[live].astype(np.float64) * 127 / top[live, None]
        assert (np.abs(q[live] - exact) <= 0.5 + 127 * 3 * 2.0 ** -24).all()


def test_product_by_hand():
    xq, wq = np.array([[1, -2], [-128, 127]], np.int8), np.array([[3, 4], [-128, -128]], np.int8)
    y, _ = R.product(xq, np.array([0.5, 2], np.float32), wq, np.array([1, 0.25], np.float32),
                     np.array([10, 0], np.float32))
    assert y.tolist() == [[-2.5 + 10, 16.0], [2 * 124 + 10, 0.5 * 128]]
    f = R.product_f32(xq, np.array([0.5, 2], np.float32), wq, np.array([1, 0.25], np.float32))
    assert f.dtype == np.float32 and f.tolist() == [[-2.5, 16.0], [248, 64]]


def test_norm_by_hand():
    y, r = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    rms = np.sqrt(12.5)
    h, _, n, _ = R.norm(y, r, np.array([1.0, 2.0]), np.array([2.0, 1.0]), np.array([[1.0, 0.5]]), 3.0, 0.0)
    want = np.array([1 + 3 * 6 / rms, -1 + 1.5 * 4 / rms])
    assert np.allclose(h, want, rtol=1e-15)
    assert np.allclose(n, want / np.sqrt((want ** 2).mean()) * [1, 2], rtol=1e-15)
    h, _, n, _ = R.norm(None, r, np.array([1.0, 1.0]), None, None, 1.0, 3.0)
    assert (h == r).all() and np.allclose(n, r / 2)


def test_route_by_hand():
    l = np.array([[0.0, 1.0, 2.0, -1.0, 3.0, -np.inf], [np.nan] * 6, [0, 0, 0, 0, 0, 0]], np.float32)
    ids, w = R.route(l, 2, None, True, 3, 1, 2, False, 2.0)
    # groups (0,1) (2,3) (4,5): sums 1.23, 1.15, 0.95
    assert ids.tolist() == [[1, 0], [-1, -1], [0, 1]]
    assert np.allclose(w[0], [2 / (1 + np.exp(-1)), 1.0]) and (w[1] == 0).all()
    ids, w = R.route(l, 2, None, False, 3, 2, 1, True, 1.0)  # a group's best: 1, 2, 3
    assert ids[0].tolist() == [4, 2] and np.allclose(w[0], np.exp([3, 2]) / np.exp([3, 2]).sum())
    b = np.array([0, 0, -np.inf, 9, 0, np.nan], np.float32)
    ids, w = R.route(l, 3, b, True, 1, 1, 1, False, 1.0)
    assert ids[0].tolist() == [3, 4, 1] and np.allclose(w[0, 0], 1 / (1 + np.e))
    l = np.array([[np.inf, np.inf, 5.0]], np.float32)
    ids, w = R.route(l, 3, None, False, 1, 1, 1, True, 1.0)
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0.5, 0.5, 0.0]]


def test_route_bias_moves_the_choice_and_not_the_weights():
    g = np.random.default_rng(2)
    l = g.standard_normal((50, 24)).astype(np.float32)
    b = (g.standard_normal(24) * 0.3).astype(np.float32)
    ids, w = R.route(l, 4, b, True, 4, 2, 2, True, 1.0)
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    picked = np.take_along_axis(s, ids, -1)
    assert np.allclose(w, picked / picked.sum(-1, keepdims=True), rtol=1e-6)
    assert all(len(set(row // 6)) <= 2 for row in ids)
    plain, _ = R.route(l, 4, None, True, 4, 2, 2, True, 1.0)
    assert (plain != ids).any()
