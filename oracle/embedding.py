"""Float64 embedding: rows of a table for a batch of ids, scaled, and the
table's gradient, token by token.  An id outside the table gives a row of
zeros and takes no part in the gradient; nor does ``padding_idx``.
"""
from __future__ import annotations

import numpy as np


def forward(ids, weight, scale: float = 1.0) -> np.ndarray:
    y = np.zeros((len(ids), weight.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < len(weight):
            y[t] = scale * weight[i]
    return y


def backward(dy, ids, vocab: int, scale: float = 1.0, padding_idx=None, start=None):
    """(dweight, the sum of the terms' sizes, the number of terms of each id)."""
    total = np.zeros((vocab, dy.shape[1])) if start is None else np.array(start)
    size, count = np.abs(total), np.zeros(vocab, dtype=np.int64)
    for t, i in enumerate(ids):
        if 0 <= i < vocab and i != padding_idx:
            total[i] += scale * dy[t]
            size[i] += np.abs(scale * dy[t])
            count[i] += 1
    return total, size, count
