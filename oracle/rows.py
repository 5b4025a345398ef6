"""Rows sorted by expert and back, and products with 4-bit weights that share a scale in groups, in fp64: the
definitions written out pair by pair and group by group, with the gradients by hand."""
from __future__ import annotations

import numpy as np

from .mlp import silu


def places(ids, E):
    """(offsets [E + 1], pos [T, k]): a pair's place among those with 0 <= id < E, stably sorted by id, or -1."""
    ids = np.asarray(ids, dtype=np.int64)
    flat = ids.reshape(-1)
    pos = np.full(flat.shape, -1, dtype=np.int64)
    offsets = np.zeros(E + 1, dtype=np.int64)
    at = 0
    for e in range(E):
        offsets[e] = at
        for p in np.nonzero(flat == e)[0]:
            pos[p] = at
            at += 1
    offsets[E] = at
    return offsets, pos.reshape(ids.shape)


def sort_rows(x, ids, E):
    """(rows [offsets[E], H], offsets, pos)."""
    offsets, pos = places(ids, E)
    x = np.asarray(x, dtype=np.float64)
    rows = np.zeros((offsets[E], x.shape[1]))
    for t, j in np.argwhere(pos >= 0):
        rows[pos[t, j]] = x[t]
    return rows, offsets, pos


def combine_rows(rows, pos, w=None, base=None):
    """(y [T, H], the sum of the terms' magnitudes): sum_j w rows[pos] + base."""
    rows, pos = np.asarray(rows, dtype=np.float64), np.asarray(pos)
    T, k = pos.shape
    y = np.zeros((T, rows.shape[1]))
    size = np.zeros_like(y)
    if base is not None:
        y += base
        size += np.abs(base)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < len(rows):
                term = rows[pos[t, j]] * (1.0 if w is None else float(w[t, j]))
                y[t] += term
                size[t] += np.abs(term)
    return y, size


def combine_rows_backward(dy, rows, pos, w=None):
    """({row: its gradient}, d_w [T, k], the magnitudes that d_w sums)."""
    dy, pos = np.asarray(dy, dtype=np.float64), np.asarray(pos)
    rows = np.asarray(rows, dtype=np.float64)
    d_rows, d_w, size = {}, np.zeros(pos.shape), np.zeros(pos.shape)
    for t, j in np.argwhere((pos >= 0) & (pos < len(rows))):
        p = int(pos[t, j])
        d_rows[p] = dy[t] * (1.0 if w is None else float(w[t, j]))
        d_w[t, j] = (dy[t] * rows[p]).sum()
        size[t, j] = np.abs(dy[t] * rows[p]).sum()
    return d_rows, d_w, size


def w4_weights(codes, scales, zeros=None):
    """[..., N, K] of codes [..., N, K / 2] (even elements in the low nibble): (q - z) s, z = 8 without zeros."""
    codes = np.asarray(codes, dtype=np.int64)
    q = np.stack([codes % 16, codes // 16], axis=-1).reshape(*codes.shape[:-1], -1).astype(np.float64)
    s = np.asarray(scales, dtype=np.float64)
    g = q.shape[-1] // s.shape[-1]
    z = np.full(s.shape, 8.0) if zeros is None else np.asarray(zeros, dtype=np.float64)
    return (q - np.repeat(z, g, axis=-1)) * np.repeat(s, g, axis=-1)


def w4_linear(x, codes, scales, zeros=None, offsets=None, swiglu=False):
    """({row: its result}, {row: the magnitudes it is the sum of}); with swiglu the magnitudes of what a relative
    error of the gate's and the up's sums moves."""
    x = np.asarray(x, dtype=np.float64)
    W = w4_weights(codes, scales, zeros)
    if W.ndim == 2:
        W = W[None]
    offsets = np.array([0, len(x)]) if offsets is None else np.asarray(offsets)
    out, size = {}, {}
    for e in range(len(W)):
        for r in range(int(offsets[e]), int(offsets[e + 1])):
            v, m = W[e] @ x[r], np.abs(W[e]) @ np.abs(x[r])
            if swiglu:
                n = len(v) // 2
                g, u = v[:n], v[n:]
                slope = 1.1 * m[:n]   # |silu'| < 1.1
                v, m = silu(g) * u, slope * np.abs(u) + (np.abs(silu(g)) + 1.1e-6 * m[:n]) * m[n:] + np.abs(silu(g) * u)
            out[r], size[r] = v, m
    return out, size
