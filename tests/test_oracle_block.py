"""The block oracle against closed forms, brute force and differences (CPU)."""
import itertools

import numpy as np
import pytest

from oracle import block as O
from oracle.router import router_topk


def test_route_without_bias_and_groups_is_the_router():
    lg = np.random.default_rng(0).standard_normal((50, 37)).astype(np.float32)
    for renorm in (True, False):
        ids, w, _ = O.route(lg, 5, renorm=renorm)
        rid, rw = router_topk(lg, 5, renorm)
        assert np.array_equal(ids, rid) and np.allclose(w, rw, rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group", ["max", "top2"])
def test_route_groups_by_enumeration(score, group):
    # every pair of the four groups, then every pair of their experts: the best of each is what route picks
    rng = np.random.default_rng(1)
    lg, b = rng.standard_normal((20, 12)), rng.standard_normal(12) * 0.2
    ids, w, _ = O.route(lg, 2, score, b, 4, 2, group, renorm=True, scale=2.0)
    s = 1 / (1 + np.exp(-lg)) if score == "sigmoid" else np.exp(lg) / np.exp(lg).sum(1, keepdims=True)
    for t in range(20):
        key = (s[t] + b).reshape(4, 3)
        worth = [max(r) if group == "max" else sum(sorted(r)[1:]) for r in key]
        gs = max(itertools.combinations(range(4), 2), key=lambda c: sum(worth[g] for g in c))
        can = [3 * g + i for g in gs for i in range(3)]
        pick = sorted(can, key=lambda e: -key.reshape(-1)[e])[:2]
        assert list(ids[t]) == pick
        assert np.allclose(w[t], 2.0 * s[t, pick] / s[t, pick].sum())


def test_route_rows_with_too_few_experts():
    lg = np.full((4, 6), -np.inf)
    lg[1, 3] = 0.5
    lg[2] = np.nan
    lg[3] = [1, 2, np.nan, -np.inf, 2, 0]
    ids, w, _ = O.route(lg, 3, "sigmoid", mask=np.array([1, 1, 1, 1], np.uint8))
    assert ids.tolist() == [[-1] * 3, [3, -1, -1], [-1] * 3, [1, 4, 0]]
    assert w[0].sum() == 0 and w[1, 0] == 1 and w[1, 1:].sum() == 0
    assert O.route(lg, 3, mask=np.zeros(4, np.uint8))[0].max() == -1


def _difference(f, x, d=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += d
        b[i] -= d
        g[i] = (f(a) - f(b)) / (2 * d)
    return g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    lg, dw = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    lg[1, 2] = -np.inf
    ids, _, _ = O.route(lg, 4, score, rng.standard_normal(9) * 0.1)
    ids[2, 3] = -1

    def weights(z):
        _, s = O.route_scores(z, score)
        tot = 0.0
        for t in range(3):
            on = ids[t] >= 0
            p = s[t, ids[t][on]]
            tot += 1.7 * ((p / p.sum() if renorm else p) * dw[t][on]).sum()
        return tot
    want = _difference(weights, np.where(np.isinf(lg), -60.0, lg))
    assert np.allclose(O.route_backward(lg, ids, dw, score, renorm, 1.7), want, atol=1e-8)


@pytest.mark.parametrize("post,gate,nxt,alpha", [(True, "channel", True, 1.0), (True, "token", True, 0.5),
                                                 (False, None, True, 1.0), (True, None, False, 0.3),
                                                 (False, "channel", True, 0.7), (False, "token", False, 1.0)])
def test_block_norm_gradient_against_differences(post, gate, nxt, alpha):
    rng = np.random.default_rng(3)
    T, H = 3, 7
    p = {"x": rng.standard_normal((T, H)), "y": rng.standard_normal((T, H)),
         "post": 1 + 0.1 * rng.standard_normal(H) if post else None,
         "gate": {None: None, "channel": rng.standard_normal(H), "token": rng.standard_normal((T, 1))}[gate],
         "nxt": 1 + 0.1 * rng.standard_normal(H) if nxt else None}
    du, dh = rng.standard_normal((T, H)), rng.standard_normal((T, H)) if nxt else None
    g, mag = O.block_norm_backward(p["x"], p["y"], du, dh, p["post"], p["gate"], alpha, p["nxt"], 1e-3)
    for name, key in (("x", "x"), ("y", "y"), ("post", "post"), ("gate", "gate"), ("nxt", "next")):
        if p[name] is None:
            continue

        def loss(v):
            q = dict(p, **{name: v})
            u, h = O.block_norm(q["x"], q["y"], q["post"], q["gate"], alpha, q["nxt"], 1e-3)
            return (u * du).sum() + (0 if h is None else (h * dh).sum())
        assert np.allclose(g[key], _difference(loss, p[name]), atol=1e-7), name
        assert np.all(mag[key] >= np.abs(g[key]) - 1e-12)


def test_block_norm_of_one_value():
    # a row of equal values v: n(y) = v / sqrt(v^2 + eps)
    y = np.full((2, 5), 3.0)
    u, h = O.block_norm(np.zeros((2, 5)), y, np.ones(5), None, 1.0, 2 * np.ones(5), 7.0)
    assert np.allclose(u, 0.75) and np.allclose(h, 2 * 0.75 / np.sqrt(0.5625 + 7))


def test_adapter_linear_is_the_merged_weight():
    rng = np.random.default_rng(4)
    x, W = rng.standard_normal((5, 8)), rng.standard_normal((6, 8))
    A, B, c = rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 6, 2)), np.array([0.5, 2.0, 1.0])
    ids = np.array([2, -1, 0, 1, 7])
    out, size, low = O.adapter_linear(x, W, A, B, ids, c)
    for t, a in enumerate(ids):
        M = W + c[a] * B[a] @ A[a] if 0 <= a < 3 else W
        assert np.allclose(out[t], M @ x[t])
    assert np.all(size + low >= np.abs(out) - 1e-12) and low[1].sum() == 0
