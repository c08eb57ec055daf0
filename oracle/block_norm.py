"""Float64 block norm: the norms after and before a transformer block with
its gate and the scaled residual sum, and their gradients.

    z = x * rstd(x) * gain(post)                  (z = x without a post norm)
    r = a * residual + b * gate * z
    y = r * rstd(r) * gain(next)                  (no y without a next norm)

rstd(v) = 1 / sqrt(mean(v^2) + eps) over a row, gain(w) = w + offset.  The
gate is None or [gate rows, hidden], each row for rows / gate rows
consecutive rows of x.  The backward is written gradient by gradient, with a
reduction for each mean, unlike the kernels.  Every function takes and
returns float64 arrays; nothing is rounded.
"""
from __future__ import annotations

import numpy as np

from .rms_norm import gain


def rstd(v: np.ndarray, eps: float) -> np.ndarray:
    return 1.0 / np.sqrt(np.mean(v * v, axis=-1) + eps)


def gate_rows(gate, rows: int, hidden: int) -> np.ndarray:
    """The gate of every row: [rows, hidden]."""
    if gate is None:
        return np.ones((rows, hidden))
    return np.repeat(np.reshape(gate, (-1, hidden)), rows // (gate.size // hidden), axis=0)


def forward(x, residual, post, gate, nxt, eps, offset=0, a=1.0, b=1.0):
    """(r, y, rstd_post, rstd_next); None for what a missing norm gives."""
    rows, hidden = x.shape
    r1 = y = r2 = None
    z = x
    if post is not None:
        r1 = rstd(x, eps)
        z = x * r1[:, None] * gain(post, offset)
    r = a * residual + b * gate_rows(gate, rows, hidden) * z
    if nxt is not None:
        r2 = rstd(r, eps)
        y = r * r2[:, None] * gain(nxt, offset)
    return r, y, r1, r2


def _norm_backward(dy, v, w, rs, offset):
    """(dv, dw) of y = v * rs * gain(w), rs the row statistic of v."""
    vh = v * rs[:, None]
    g = dy * gain(w, offset)
    return rs[:, None] * (g - vh * np.mean(g * vh, axis=-1, keepdims=True)), np.sum(dy * vh, axis=0)


def backward(dy, dr, x, r, post, gate, nxt, r1, r2, offset=0, a=1.0, b=1.0):
    """(dx, dresidual, dpost, dgate, dnext) for the given rows of statistics
    r1, r2; dgate [gate rows, hidden]."""
    rows, hidden = x.shape
    total = np.zeros_like(x) if dr is None else dr
    dpost = dgate = dnext = None
    if nxt is not None:
        dv, dnext = _norm_backward(dy, r, nxt, r2, offset)
        total = total + dv
    dbranch = b * total
    z = x if post is None else x * r1[:, None] * gain(post, offset)
    if gate is not None:
        n = gate.size // hidden
        dgate = np.sum(np.reshape(dbranch * z, (n, rows // n, hidden)), axis=1)
    dz = dbranch * gate_rows(gate, rows, hidden)
    dx = dz
    if post is not None:
        dx, dpost = _norm_backward(dz, x, post, r1, offset)
    return dx, a * total, dpost, dgate, dnext
