"""Float64 CPU oracle of the join of a block with the residual stream: the norm of the block's
output, its gate and scale, the residual sum and the next block's norm, and their gradients.

Test infrastructure only.  Beside every result stands the sum of the magnitudes that went into
it, which is what a float32 evaluation's error is measured against.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import numpy as np


class Join(NamedTuple):
    post_norm: bool = False
    gate: str = "none"        # "none", "channel" [H], "token" [rows], "element" [rows, H]
    sigmoid: bool = False
    eps: float = 1e-6
    offset: float = 0.0
    scale: float = 1.0


def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _factor(w, offset, H):
    return np.ones(H) if w is None else offset + w


def _gate(j: Join, gate):
    """The gate's value and its derivative, laid out against [rows, H]."""
    if j.gate == "none":
        return np.ones((1, 1)), np.zeros((1, 1))
    g = gate[:, None] if j.gate == "token" else gate[None, :] if j.gate == "channel" else gate
    if not j.sigmoid:
        return g, np.ones_like(g)
    s = 1.0 / (1.0 + np.exp(-g))
    return s, s / (1.0 + np.exp(g))  # s (1 - s), without the difference


def forward(j: Join, x, y=None, gate=None, w_post=None, w_pre=None, next_norm: bool = True) -> dict:
    """{"z", "h"} and, under "mag_z" and "mag_h", the magnitudes that went into them."""
    H = x.shape[1]
    z, mag, out = x, np.abs(x), {}
    if y is not None:
        b = y * _rstd(y, j.eps) * _factor(w_post, j.offset, H) if j.post_norm else y
        g, _ = _gate(j, gate)
        add = j.scale * g * b
        z, mag = x + add, np.abs(x) + np.abs(add)
        out.update(z=z, mag_z=mag)
    if next_norm:
        r, f = _rstd(z, j.eps), _factor(w_pre, j.offset, H)
        out.update(h=z * r * f, mag_h=mag * r * np.abs(f))
    return out


def backward(j: Join, z, y=None, gate=None, w_post=None, w_pre=None, dz: Optional[np.ndarray] = None,
             dh: Optional[np.ndarray] = None) -> dict:
    """The gradients, and under "mag_..." the magnitudes that went into each."""
    H = z.shape[1]
    D = np.zeros_like(z) if dz is None else dz
    mD = np.abs(D)
    out = {}
    if dh is not None:
        r = _rstd(z, j.eps)
        zh, a = z * r, dh * _factor(w_pre, j.offset, H)
        D = D + r * (a - zh * (a * zh).mean(axis=1, keepdims=True))
        mD = mD + r * (np.abs(a) + np.abs(zh) * np.abs(a * zh).mean(axis=1, keepdims=True))
        if w_pre is not None:
            out.update(dw_pre=(dh * zh).sum(0), mag_dw_pre=np.abs(dh * zh).sum(0))
    out.update(dx=D, mag_dx=mD)
    if y is None:
        return out
    g, dg = _gate(j, gate)
    r = _rstd(y, j.eps) if j.post_norm else np.ones((len(y), 1))
    yh, f = y * r, _factor(w_post, j.offset, H)
    db, mdb = j.scale * g * D, abs(j.scale) * np.abs(g) * mD
    if j.post_norm:
        c, mc = db * f, mdb * np.abs(f)
        out["dy"] = r * (c - yh * (c * yh).mean(axis=1, keepdims=True))
        out["mag_dy"] = r * (mc + np.abs(yh) * (mc * np.abs(yh)).mean(axis=1, keepdims=True))
        if w_post is not None:
            out.update(dw_post=(db * yh).sum(0), mag_dw_post=(mdb * np.abs(yh)).sum(0))
    else:
        out.update(dy=db, mag_dy=mdb)
    if j.gate != "none":
        v, mv = j.scale * D * yh * f * dg, abs(j.scale) * mD * np.abs(yh * f) * np.abs(dg)
        axis = {"channel": 0, "token": 1, "element": None}[j.gate]
        out["dgate"], out["mag_dgate"] = (v, mv) if axis is None else (v.sum(axis), mv.sum(axis))
    return out
