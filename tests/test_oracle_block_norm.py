"""The float64 block norm against independent definitions: torch's float64
rms_norm composed with the gate and the sum, its autograd, and differences."""
import itertools

import numpy as np
import pytest
import torch

from oracle import block_norm as obn

EPS = 1e-5
FLAGS = [f for f in itertools.product((True, False), (0, 1, 3), (True, False)) if f[0] or f[2]]


def inputs(post, gates, nxt, rows=6, hidden=10, seed=0):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    return dict(x=n(rows, hidden), residual=n(rows, hidden),
                post=n(hidden) if post else None, gate=n(gates, hidden) if gates else None,
                nxt=n(hidden) if nxt else None)


def by_torch(t, offset, a, b):
    hidden = t["x"].shape[1]
    z = t["x"]
    if t["post"] is not None:
        z = torch.nn.functional.rms_norm(z, (hidden,), t["post"] + offset, EPS)
    if t["gate"] is not None:
        n = t["gate"].shape[0]
        z = (z.view(n, -1, hidden) * t["gate"][:, None]).view(z.shape)
    r = a * t["residual"] + b * z
    y = None
    if t["nxt"] is not None:
        y = torch.nn.functional.rms_norm(r, (hidden,), t["nxt"] + offset, EPS)
    return r, y


@pytest.mark.parametrize("post,gates,nxt", FLAGS)
@pytest.mark.parametrize("offset,a,b", [(0, 1.0, 1.0), (1, 0.5, -0.25)])
def test_matches_torch_and_its_autograd(post, gates, nxt, offset, a, b):
    v = inputs(post, gates, nxt)
    t = {k: None if u is None else torch.from_numpy(u).requires_grad_() for k, u in v.items()}
    r_t, y_t = by_torch(t, offset, a, b)
    r, y, r1, r2 = obn.forward(v["x"], v["residual"], v["post"], v["gate"], v["nxt"], EPS, offset,
                               a, b)
    assert np.allclose(r, r_t.detach().numpy(), rtol=1e-13, atol=1e-13)
    assert (y is None) == (y_t is None)
    rng = np.random.default_rng(1)
    dr = rng.standard_normal(r.shape)
    dy = rng.standard_normal(r.shape) if nxt else None
    loss = (r_t * torch.from_numpy(dr)).sum()
    if nxt:
        assert np.allclose(y, y_t.detach().numpy(), rtol=1e-13, atol=1e-13)
        loss = loss + (y_t * torch.from_numpy(dy)).sum()
    loss.backward()
    got = obn.backward(dy, dr, v["x"], r, v["post"], v["gate"], v["nxt"], r1, r2, offset, a, b)
    for g, k in zip(got, ("x", "residual", "post", "gate", "nxt")):
        assert (g is None) == (t[k] is None), k
        if g is not None:
            assert np.allclose(g, t[k].grad.numpy(), rtol=1e-11, atol=1e-12), k


@pytest.mark.parametrize("post,gates,nxt", [(True, 2, True), (False, 1, True), (True, 0, False)])
def test_matches_differences(post, gates, nxt):
    v = inputs(post, gates, nxt, rows=4, hidden=5, seed=3)
    rng = np.random.default_rng(2)
    dr, dy = rng.standard_normal((4, 5)), rng.standard_normal((4, 5))

    def loss(u):
        r, y, _, _ = obn.forward(u["x"], u["residual"], u["post"], u["gate"], u["nxt"], EPS, 1,
                                 0.75, 1.5)
        return np.sum(r * dr) + (np.sum(y * dy) if nxt else 0.0)

    r, _, r1, r2 = obn.forward(v["x"], v["residual"], v["post"], v["gate"], v["nxt"], EPS, 1, 0.75,
                               1.5)
    got = obn.backward(dy if nxt else None, dr, v["x"], r, v["post"], v["gate"], v["nxt"], r1, r2,
                       1, 0.75, 1.5)
    h = 1e-6
    for g, k in zip(got, ("x", "residual", "post", "gate", "nxt")):
        if g is None:
            continue
        for at in np.ndindex(*v[k].shape):
            up, down = dict(v), dict(v)
            up[k], down[k] = v[k].copy(), v[k].copy()
            up[k][at] += h
            down[k][at] -= h
            d = (loss(up) - loss(down)) / (2 * h)
            assert abs(d - g[at]) <= 1e-7 * (1 + abs(d)), (k, at)
