"""Float64 head norm and rotation, and their gradients.

    u = v * rstd(v) * gain(gamma)   over each head's row v
    y = R(position) u               R a matrix of plane rotations

rstd(v) = 1 / sqrt(mean(v^2) + eps), gain(w) = w + offset.  The rotation is
written as a [dim, dim] matrix for each position, its transpose the
backward's, unlike the kernels.  Arrays of heads are [batch, tokens, heads,
dim], positions [batch, tokens]; every function takes and returns float64
arrays; nothing is rounded.
"""
from __future__ import annotations

import numpy as np

from .rms_norm import gain


def matrices(positions, inv_freq, dim: int, interleaved: bool) -> np.ndarray:
    """R for every position: [*positions.shape, dim, dim]."""
    pairs = len(inv_freq)
    m = np.zeros((*positions.shape, dim, dim))
    m[..., np.arange(dim), np.arange(dim)] = 1.0
    for p in range(pairs):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
        # the angle modulo a turn, in the widest floats there are
        a = np.mod(positions.astype(np.longdouble) * np.longdouble(inv_freq[p]),
                   2 * np.longdouble("3.14159265358979323846264338327950288"))
        c, s = np.cos(a).astype(np.float64), np.sin(a).astype(np.float64)
        m[..., i, i], m[..., i, j] = c, -s
        m[..., j, i], m[..., j, j] = s, c
    return m


def rstd(v: np.ndarray, eps: float) -> np.ndarray:
    return 1.0 / np.sqrt(np.mean(v * v, axis=-1) + eps)


def forward(v, gamma, turn, eps, offset=0):
    """(y, rstd, u) of one tensor of heads."""
    r = rstd(v, eps)
    u = v * r[..., None] * gain(gamma, offset)
    return np.einsum("btij,bthj->bthi", turn, u), r, u


def backward(dy, v, gamma, turn, r, offset=0):
    """(dv, dgamma) for the given statistics r."""
    du = np.einsum("btji,bthj->bthi", turn, dy)
    vh = v * r[..., None]
    g = du * gain(gamma, offset)
    dv = r[..., None] * (g - vh * np.mean(g * vh, axis=-1, keepdims=True))
    return dv, np.sum(du * vh, axis=(0, 1, 2))
