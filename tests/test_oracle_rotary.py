"""What pins the float64 oracles of the head norm with rotation and of the
embedding: finite differences, closed forms, torch on the CPU."""
import numpy as np
import pytest
import torch

from oracle import embedding as oem
from oracle import rms_norm as orm
from oracle import rotary as oro


def case(interleaved, dim=8, pairs=3, seed=0):
    g = np.random.default_rng(seed)
    v, dy = g.standard_normal((2, 2, 3, 2, dim))
    gamma = 1 + 0.1 * g.standard_normal(dim)
    pos = g.integers(0, 1000, (2, 3))
    freq = 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    return v, dy, gamma, pos, oro.matrices(pos, freq, dim, interleaved), freq


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("offset", [0, 1])
def test_backward_against_differences(interleaved, offset):
    v, dy, gamma, _, turn, _ = case(interleaved)
    f = lambda v, w: np.sum(dy * oro.forward(v, w, turn, 1e-5, offset)[0])  # noqa: E731
    dv, dw = oro.backward(dy, v, gamma, turn, oro.rstd(v, 1e-5), offset)
    e = 1e-6
    for at in [(0, 0, 0, 0), (1, 2, 1, 7), (0, 1, 1, 4)]:
        d = np.zeros_like(v)
        d[at] = e
        assert abs((f(v + d, gamma) - f(v - d, gamma)) / (2 * e) - dv[at]) < 1e-7
    for j in range(8):
        d = np.eye(8)[j] * e
        assert abs((f(v, gamma + d) - f(v, gamma - d)) / (2 * e) - dw[j]) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    v, _, gamma, pos, turn, freq = case(interleaved)
    y, r, u = oro.forward(v, gamma, turn, 1e-5)
    flat = v.reshape(-1, 8)
    want, rs = orm.forward_exact(flat, gamma, 1e-5, 0)[:2]
    assert np.allclose(u.reshape(-1, 8), want, rtol=1e-12) and np.allclose(r.ravel(), rs)
    assert np.allclose(np.sum(y * y, -1), np.sum(u * u, -1))            # a rotation
    assert np.array_equal(y[..., 6:], u[..., 6:])                       # three pairs of four
    i, j = (0, 1) if interleaved else (0, 3)
    z = (u[..., i] + 1j * u[..., j]) * np.exp(1j * pos[..., None] * freq[0])
    assert np.allclose(y[..., i] + 1j * y[..., j], z)
    assert np.allclose(oro.matrices(np.zeros((1, 1), int), freq, 8, interleaved)[0, 0], np.eye(8))


def test_scores_depend_on_the_distance_alone():
    g = np.random.default_rng(1)
    a, b = g.standard_normal((2, 16))
    freq = 100.0 ** (-np.arange(8) / 8)
    m = oro.matrices(np.array([[5, 9, 1005, 1009]]), freq, 16, False)[0]
    assert np.isclose(m[0] @ a @ (m[1] @ b), m[2] @ a @ (m[3] @ b))


def test_embedding_against_torch():
    gen = torch.Generator().manual_seed(0)
    ids = torch.randint(0, 7, (40,), generator=gen)
    w = torch.randn(7, 5, generator=gen, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(40, 5, generator=gen, dtype=torch.float64)
    y = torch.nn.functional.embedding(ids, w, padding_idx=3) * 2.5
    y.backward(dy)
    assert np.allclose(oem.forward(ids.numpy(), w.detach().numpy(), 2.5), y.detach().numpy())
    got, size, count = oem.backward(dy.numpy(), ids.numpy(), 7, 2.5, 3)
    assert np.allclose(got, w.grad.numpy()) and count.sum() == int((ids != 3).sum())
    assert np.all(size >= np.abs(got) - 1e-12)


def test_embedding_outside_the_table():
    ids = np.array([-1, 0, 2, 7])
    w = np.ones((2, 3))
    assert np.array_equal(oem.forward(ids, w), [[0] * 3, [1] * 3, [0] * 3, [0] * 3])
    got, _, count = oem.backward(np.ones((4, 3)), ids, 2, start=w)
    assert np.array_equal(got, [[2] * 3, [1] * 3]) and list(count) == [1, 0]
