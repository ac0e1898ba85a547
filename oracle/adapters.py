"""Float64 CPU oracle of the local experts with low-rank adapters of many requests beside their
projections.  Test infrastructure only."""

from __future__ import annotations

import numpy as np


def project(x, w, a, b, scale, ids):
    """x [n, K] through w [N, K], and row i through scale[id] (x A^T) B^T of its adapter ids[i] (a [count, R, K],
    b [count, N, R]; an id outside [0, count) has none)."""
    y = x @ w.T
    if a is not None:
        for q, i in enumerate(ids):
            if 0 <= i < len(a):
                y[q] += scale[i] * (b[i] @ (a[i] @ x[q]))
    return y


def grouped_ffn(x_sorted, offsets, ids, w, ad, scale):
    """y_sorted of rows sorted by expert.  w: "gate", "up" [L, I, H], "down" [L, H, I]; ad: "gate_a" [count, L, R, H],
    "gate_b" [count, L, I, R] and so on, absent for a projection without adapters; ids: the adapter of every row."""
    y = np.zeros((len(x_sorted), w["down"].shape[1]))
    for e in range(len(offsets) - 1):
        rows = slice(offsets[e], offsets[e + 1])
        if offsets[e + 1] == offsets[e]:
            continue

        def through(v, name):
            a, b = ad.get(name + "_a"), ad.get(name + "_b")
            return project(v, w[name][e], None if a is None else a[:, e], None if b is None else b[:, e], scale, ids[rows])
        g = through(x_sorted[rows], "gate")
        y[rows] = through(g / (1.0 + np.exp(-g)) * through(x_sorted[rows], "up"), "down")
    return y
