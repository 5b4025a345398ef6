"""Pins of the oracle of sorted rows and 4-bit products: closed forms, the framework's own grouping, differences."""
import numpy as np
import pytest

from oracle import rows as R
from oracle.permute import group_pairs


def test_places_agree_with_the_grouping_of_pairs():
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 7, size=(23, 3))
    offsets, pos = R.places(ids, 7)
    off, perm = group_pairs(ids, 7)
    assert (offsets == off).all()
    assert (pos.reshape(-1)[perm] == np.arange(len(perm))).all() and (pos < 0).sum() == (ids < 0).sum()


def test_sorted_rows_of_two_tokens():
    rows, offsets, pos = R.sort_rows([[1.0, 2.0], [3.0, 4.0]], [[2, 0], [0, -1]], 3)
    assert offsets.tolist() == [0, 2, 2, 3] and pos.tolist() == [[2, 0], [1, -1]]
    assert rows.tolist() == [[1, 2], [3, 4], [1, 2]]


def test_combine_of_sorted_rows_is_a_multiple_of_the_tokens():
    rng = np.random.default_rng(1)
    x, ids = rng.standard_normal((5, 4)), rng.integers(-1, 3, size=(5, 2))
    w = rng.random((5, 2))
    rows, _, pos = R.sort_rows(x, ids, 3)
    y, size = R.combine_rows(rows, pos, w, 2 * x)
    by = 2 + (w * (ids >= 0)).sum(1, keepdims=True)
    assert np.allclose(y, by * x, rtol=1e-14) and np.allclose(size, by * np.abs(x), rtol=1e-14)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(2)
    rows, pos, w, dy = rng.standard_normal((4, 3)), np.array([[2, 0], [-1, 3]]), rng.random((2, 2)), rng.standard_normal((2, 3))
    d_rows, d_w, _ = R.combine_rows_backward(dy, rows, pos, w)
    f = lambda r, v: (R.combine_rows(r, pos, v)[0] * dy).sum()
    h = 1e-6
    for i in np.ndindex(rows.shape):
        e = np.zeros_like(rows)
        e[i] = h
        want = d_rows[i[0]][i[1]] if i[0] in d_rows else 0.0
        assert abs((f(rows + e, w) - f(rows - e, w)) / (2 * h) - want) < 1e-8
    for i in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((f(rows, w + e) - f(rows, w - e)) / (2 * h) - d_w[i]) < 1e-8


def test_weights_of_one_byte_and_of_groups():
    W = R.w4_weights(np.array([[0x81, 0xf0]]), np.array([[2.0, 0.5]]), np.array([[1, 4]]))
    assert W.tolist() == [[0.0, 14.0, -2.0, 5.5]]
    assert R.w4_weights(np.array([[0x81]]), np.array([[2.0]])).tolist() == [[-14.0, 0.0]]


@pytest.mark.parametrize("swiglu", [False, True])
def test_products_by_expert(swiglu):
    rng = np.random.default_rng(3)
    codes, scales = rng.integers(0, 256, size=(3, 4, 8)), rng.random((3, 4, 2))
    x = rng.standard_normal((5, 16))
    out, _ = R.w4_linear(x, codes, scales, None, [0, 2, 2, 4], swiglu)
    assert sorted(out) == [0, 1, 2, 3]
    for r, e in ((0, 0), (1, 0), (2, 2), (3, 2)):
        v = x[r] @ R.w4_weights(codes[e], scales[e]).T
        want = v[:2] / (1 + np.exp(-v[:2])) * v[2:] if swiglu else v
        assert np.allclose(out[r], want, rtol=1e-13)
