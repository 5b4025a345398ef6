"""What stands around the routed experts in a block, in fp64: routing with a
balance bias and expert groups, the norms before and after the block with gate
and residual scale, the projection with low-rank adapters; and the gradients of
the first two, written out by hand from the formulas."""
from __future__ import annotations

import numpy as np


def route_scores(logits, score, mask=None):
    """(logits with -inf where an expert is not eligible, scores)."""
    z = np.array(logits, dtype=np.float64)
    z[np.isnan(z)] = -np.inf
    if mask is not None:
        z[np.asarray(mask) == 0] = -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-z))
            s[z < -np.log(np.finfo(np.float32).max)] = 0.0   # e^-l is past fp32's range: the score is 0
        else:
            top = z.max(axis=1, keepdims=True)
            e = np.where(z == -np.inf, 0.0, np.where(z == top, 1.0, np.exp(z - top)))
            den = e.sum(axis=1, keepdims=True)
            s = np.divide(e, den, out=np.zeros_like(e), where=den > 0)
    return z, s


def _order(v):
    """Indices by descending value, ties to the lower index."""
    return np.lexsort((np.arange(len(v)), -v))


def route(logits, k, score="softmax", bias=None, n_group=1, topk_group=1, group="top2", renorm=True, scale=1.0,
          mask=None):
    """(ids [T, k], w [T, k], margin [T]): margin is the smallest gap between unequal values that
    the choice or its order hangs on."""
    z, s = route_scores(logits, score, mask)
    T, E = z.shape
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    margin = np.full(T, np.inf)
    for t in range(T):
        can = z[t] > -np.inf
        key = z[t].copy() if bias is None else np.where(can, s[t] + bias, -np.inf)
        if topk_group < n_group:
            val = key if bias is not None or group == "max" else np.where(can, s[t], -np.inf)
            worth = np.empty(n_group)
            for g, part in enumerate(val.reshape(n_group, -1)):
                top = np.sort(part)[::-1]
                worth[g] = top[0]
                if group == "top2" and len(top) > 1 and top[1] > -np.inf:
                    worth[g] += top[1]
            o = _order(worth)
            a, b = worth[o[topk_group - 1]], worth[o[topk_group]]
            if a != b:
                margin[t] = min(margin[t], a - b)
            keep = np.zeros(n_group, dtype=bool)
            keep[o[:topk_group]] = True
            key[~np.repeat(keep, E // n_group)] = -np.inf
        o = _order(key)
        for a, b in zip(o[:k], o[1:k + 1]):
            if key[a] != key[b]:
                margin[t] = min(margin[t], key[a] - key[b])
        sel = [e for e in o[:k] if key[e] > -np.inf]
        ids[t, :len(sel)] = sel
        kept = s[t, sel]
        if renorm and score == "softmax" and sel:
            kept = route_scores(z[t:t + 1, sel], "softmax")[1][0]
        elif renorm and sel:
            kept = kept / kept.sum() if kept.sum() > 0 else 0 * kept
        w[t, :len(sel)] = scale * kept
    return ids, w, margin


def route_backward(logits, ids, dw, score="softmax", renorm=True, scale=1.0, mask=None):
    """d logits with the choice held fixed."""
    z, s = route_scores(logits, score, mask)
    d = np.zeros_like(z)
    for t in range(z.shape[0]):
        at = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < z.shape[1] and z[t, e] > -np.inf]
        if not at:
            continue
        j, e = map(list, zip(*at))
        g = scale * np.asarray(dw[t], dtype=np.float64)[j]
        if renorm:
            if score == "softmax":
                q, c = route_scores(z[t:t + 1, e], "softmax")[1][0], 1.0
            else:
                c = 1.0 / (1.0 + np.exp(z[t, e]))
                q = s[t, e] / s[t, e].sum() if s[t, e].sum() > 0 else 0 * g
            d[t, e] = q * c * (g - (q * g).sum())
        elif score == "sigmoid":
            d[t, e] = g * s[t, e] / (1.0 + np.exp(z[t, e]))
        else:
            d[t] = -s[t] * (g * s[t, e]).sum()
            d[t, e] += g * s[t, e]
    return d


def _f64(*a):
    return [None if v is None else np.asarray(v, dtype=np.float64) for v in a]


def block_norm(x, y=None, post=None, gate=None, alpha=1.0, nxt=None, eps=1e-6):
    """(u, h): gate [H] or [T, 1]."""
    x, y, post, gate, nxt = _f64(x, y, post, gate, nxt)
    u = alpha * x
    if y is not None:
        v = y if post is None else y / np.sqrt((y * y).mean(1, keepdims=True) + eps) * post
        u = u + (v if gate is None else gate * v)
    return u, None if nxt is None else u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * nxt


def block_norm_backward(x, y, du, dh, post=None, gate=None, alpha=1.0, nxt=None, eps=1e-6):
    """({name: gradient}, {name: the magnitudes of the terms it is the sum of}): what rounding errors
    are measured by, since the terms of a norm's gradient can cancel."""
    x, y, du, dh, post, gate, nxt = _f64(x, y, du, dh, post, gate, nxt)
    u, _ = block_norm(x, y, post, gate, alpha, None, eps)
    D = np.zeros_like(u) if du is None else du
    m = np.abs(D)
    g, mag = {}, {}
    if nxt is not None:
        ru = 1.0 / np.sqrt((u * u).mean(1, keepdims=True) + eps)
        A = dh * nxt
        D = D + ru * (A - u * ru ** 2 * (A * u).mean(1, keepdims=True))
        m = m + ru * (np.abs(A) + np.abs(u) * ru ** 2 * np.abs(A * u).mean(1, keepdims=True))
        g["next"] = (dh * u * ru).sum(0)
        mag["next"] = (np.abs(dh) * ru * (np.abs(alpha * x) + np.abs(u - alpha * x))).sum(0)   # u can cancel too
    g["x"], mag["x"] = alpha * D, abs(alpha) * m
    if y is not None:
        ry = 1.0 if post is None else 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        n = y * ry
        v = n if post is None else n * post
        if gate is not None:
            axis, keep = (0, False) if gate.ndim == 1 else (1, True)
            g["gate"] = (D * v).sum(axis, keepdims=keep)
            mag["gate"] = (m * np.abs(v)).sum(axis, keepdims=keep)
        B = D if gate is None else gate * D
        m = m if gate is None else np.abs(gate) * m
        if post is not None:
            g["post"], mag["post"] = (B * n).sum(0), (m * np.abs(n)).sum(0)
            B, m = B * post, m * np.abs(post)
            B = ry * (B - n * (B * n).mean(1, keepdims=True))
            m = ry * (m + np.abs(n) * (m * np.abs(n)).mean(1, keepdims=True))
        g["y"], mag["y"] = B, m
    return g, mag


def adapter_linear(x, W, A=None, B=None, ids=None, scale=None):
    """(out, size, low): the sums of the magnitudes of the products behind each output, of the
    projection and of the adapter."""
    x, W = _f64(x, W)
    out, size = x @ W.T, np.abs(x) @ np.abs(W).T
    low = np.zeros_like(out)
    for t in range(x.shape[0]):
        a = -1 if A is None else int(ids[t])
        if A is None or not 0 <= a < len(A):
            continue
        Aa, Ba = _f64(A[a], B[a])
        c = 1.0 if scale is None else float(scale[a])
        out[t] += c * (Ba @ (Aa @ x[t]))
        low[t] = abs(c) * (np.abs(Ba) @ (np.abs(Aa) @ np.abs(x[t])))
    return out, size, low
