"""Pins of the oracle of the dispatch operators and integer products: worked
values, gradients against differences, exact rational sums."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import dispatch, serve


def test_sort_by_hand():
    ids = np.array([[2, 0], [-1, 2], [0, 7], [2, -5]])
    splits, rows = dispatch.sort(ids, 3)
    assert rows.tolist() == [[2, 0], [-6, 3], [1, -7], [4, -8]]
    assert splits.tolist() == [2, 0, 6]  # three slots of expert 2 and the three empty ones
    s, r = dispatch.sort(np.zeros((0, 4), int), 2)
    assert s.tolist() == [0, 0] and r.shape == (0, 4)


@pytest.mark.parametrize("seed", range(4))
def test_rows_are_a_permutation_in_expert_order(seed):
    rng = np.random.default_rng(seed)
    ids = rng.integers(-1, 5, (17, 3))
    splits, rows = dispatch.sort(ids, 5)
    at = np.array([dispatch.place(e) for e in rows.flat])
    assert sorted(at) == list(range(51)) and splits.sum() == 51
    by_row = ids.reshape(-1)[np.argsort(at)]
    filled = by_row[by_row >= 0]
    assert (np.diff(filled) >= 0).all() and (by_row[len(filled):] < 0).all()
    for e in range(5):  # stable
        assert (np.diff(at[ids.reshape(-1) == e]) > 0).all()


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    ids = np.array([[1, 0, 2], [0, -1, 1], [-1, -1, -1], [2, 1, 0]])
    _, rows = dispatch.sort(ids, 3)
    y, w, c = rng.standard_normal((12, 5)), rng.random((4, 3)), rng.standard_normal((4, 5))
    f = lambda y, w: float((dispatch.combine(y, rows, w)[0] * c).sum())  # noqa: E731
    dy, dw, _ = dispatch.combine_backward(c, y, rows, w)
    h = 1e-6
    for i in np.ndindex(y.shape):
        d = np.zeros_like(y)
        d[i] = h
        assert abs((f(y + d, w) - f(y - d, w)) / (2 * h) - dy[i]) < 1e-8
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((f(y, w + d) - f(y, w - d)) / (2 * h) - dw[i]) < 1e-8
    x = rng.standard_normal((4, 5))  # gather and the unweighted combine are adjoint
    g = rng.standard_normal((12, 5))
    assert abs((dispatch.gather(x, rows) * g).sum() - (x * dispatch.combine(g, rows, None)[0]).sum()) < 1e-12


@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(renorm):
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((6, 7))
    logits[1, 2:5] = -np.inf
    logits[2] = -np.inf
    logits[3, 1:] = -np.inf  # fewer experts than slots
    ids, w = serve.route(logits, 3, renorm)
    d = rng.standard_normal((6, 3))
    got, _ = dispatch.route_backward(d, ids, w, None if renorm else logits, 7, renorm)
    h = 1e-6

    def loss(l):
        i, w = serve.route(l, 3, renorm)
        assert (i == ids).all()
        return float((w * d * (i >= 0)).sum())

    for i in np.ndindex(logits.shape):
        if logits[i] > -np.inf:
            e = np.zeros_like(logits)
            e[i] = h
            assert abs((loss(logits + e) - loss(logits - e)) / (2 * h) - got[i]) < 1e-8
        else:
            assert got[i] == 0


def test_int8_by_hand():
    x = np.array([[127, -127, 63.5, 0.5, 1.5, 2.5, -0.5, 0], [0] * 8, [np.inf] + [0] * 7, [1, np.nan] + [0] * 6,
                  [2.0 ** -110] + [0] * 7], np.float32)
    q, s = dispatch.int8_quantize(x)
    assert q[0].tolist() == [127, -127, 64, 0, 2, 2, 0, 0] and s[0] == 1
    assert q[1].tolist() == [0] * 8 and s[1] == np.float32(2.0 ** -100) / np.float32(127)
    assert np.isnan(s[2]) and np.isnan(s[3]) and not q[2:4].any()
    assert s[4] == s[1] and not q[4].any()


def test_int8_codes_are_nearest():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 64)) * 10.0 ** rng.integers(-20, 20, (50, 1))).astype(np.float32)
    x = (x.view(np.uint32) & 0xFFFF0000).view(np.float32)
    q, s = dispatch.int8_quantize(x)
    assert np.abs(q.astype(int)).max(1).tolist() == [127] * 50
    # within half a step of the value, up to the rounding of the scale and its inverse
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= s[:, None] * (0.5 + 127 * 2.0 ** -22)).all()


def test_int8_gemm_against_rationals():
    rng = np.random.default_rng(1)
    qa, qw = rng.integers(-128, 128, (5, 16)), rng.integers(-128, 128, (6, 16))
    sa, sw = rng.random(5).astype(np.float32), rng.random(6).astype(np.float32)
    y, _ = dispatch.int8_gemm(qa, sa, qw, sw, [2, 3])
    for i in range(5):
        g = 0 if i < 2 else 1
        for n in range(3):
            want = Fraction(float(sa[i])) * Fraction(float(sw[g * 3 + n])) * sum(int(a) * int(b) for a, b in zip(qa[i], qw[g * 3 + n]))
            assert abs(float(want) - y[i, n]) <= 2.0 ** -50 * abs(float(want))
