"""The direct binding of the usual calls: it declines what needs a second
look, and where it takes a call the results are those of the other way."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import bwd_rms_norm_gb300 as lib
    from bwd_rms_norm_gb300 import build
    if not (os.path.exists(lib.LIB_PATH) and os.path.exists(lib.BINDING_PATH)):
        build.build()
    lib.load_library()
    return lib


def test_declines_on_the_host(L):
    b, z = L._binding, torch.zeros(4, 8)
    w = torch.ones(8)
    assert b.block_fwd(z, z, w, None, w, 1e-5, 0, 1.0, 1.0) is None       # not CUDA
    assert b.block_fwd(z, z) is None                                      # too few arguments
    assert b.block_fwd(None, z, w, None, w, 1e-5, 0, 1.0, 1.0) is None
    assert b.block_fwd("x", 3, w, None, w, 1e-5, 0, 1.0, 1.0) is None
    assert b.block_bwd(*[z] * 4, *[None] * 5, 0, 1.0, 1.0, True) is None
    assert b.grad_norm([z]) is None and b.grad_norm([]) is None
    assert b.grad_norm(z) is None and b.grad_norm(None) is None and b.grad_norm(iter([z])) is None
    assert b.grad_clip([z], 1.0, 1e-6, None, None) is None
    with pytest.raises((ValueError, TypeError)):
        b.init(1, 2)


@pytest.fixture
def other_way(L, monkeypatch):
    def call(f, *args, **kw):
        with monkeypatch.context() as m:
            m.setattr(L, "_binding", None)
            return f(*args, **kw)
    return call


def same(a, b):
    a, b = (v if isinstance(v, tuple) else (v,) for v in (a, b))
    assert len(a) == len(b)
    for u, v in zip(a, b):
        assert (u is None) == (v is None)
        if u is not None:
            assert u.shape == v.shape and u.dtype == v.dtype and u.device == v.device
            assert torch.equal(u, v)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,res", [("float32", "float32"), ("bfloat16", "bfloat16"),
                                       ("float16", "float32")])
@pytest.mark.parametrize("post,gates,nxt", [(1, (), 1), (1, (96,), 0), (0, (4, 1, 96), 1),
                                            (1, (4, 96), 1)])
def test_block_norm(L, other_way, dtype, res, post, gates, nxt):
    t, ts = getattr(torch, dtype), getattr(torch, res)
    x = torch.randn(4, 6, 96, device="cuda").to(t)
    r = torch.randn(4, 6, 96, device="cuda").to(ts)
    w = torch.rand(96, device="cuda").to(t) + 1
    p = torch.nn.Parameter(w) if post else None
    g = torch.rand(gates, device="cuda").to(t) if gates else None
    n = w if nxt else None
    args = (x, r, p, g, n, 1e-5, 1, 0.5, 2.0)
    assert L._binding.block_fwd(*args) is not None
    out = L.rms_norm_block_fwd(*args)
    same(out, other_way(L.rms_norm_block_fwd, *args))
    back = (x if nxt else None, r, x, out[0], out[2], out[3], p, g, n, 1, 0.5, 2.0)
    for with_dgate in (True, False):
        assert L._binding.block_bwd(*back, with_dgate) is not None
        got = L.rms_norm_block_bwd(*back, with_dgate=with_dgate)
        same(got, other_way(L.rms_norm_block_bwd, *back, with_dgate=with_dgate))


@pytest.mark.gpu
def test_gradients(L, other_way):
    grads = [torch.randn(n, device="cuda").to(d) for n, d in
             ((1000, torch.float32), (7, torch.bfloat16), (0, torch.float16), (300, torch.float16))]
    out = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    norm = L.rms_norm_grad_norm(grads)
    assert L._binding.grad_norm(tuple(grads)) is not None
    same(norm, other_way(L.rms_norm_grad_norm, grads))
    for kw in (dict(), dict(total_norm=norm * 2)):
        assert L._binding.grad_clip(grads, 1.0, 1e-6, out, kw.get("total_norm")) is not None
        a = L.rms_norm_grad_clip(grads, 1.0, out=out, **kw)
        first = [o.clone() for o in out]
        same(a, other_way(L.rms_norm_grad_clip, grads, 1.0, out=out, **kw))
        same(tuple(first), tuple(out))
    copies = [g.clone() for g in grads]
    same(L.rms_norm_grad_clip(grads, 1.0), other_way(L.rms_norm_grad_clip, copies, 1.0))
    same(tuple(grads), tuple(copies))


@pytest.mark.gpu
def test_declines_on_the_gpu(L):
    """What the Python functions refuse, with their messages."""
    b = L._binding
    x = torch.randn(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    ok = (x, x.clone(), w, None, w, 1e-5, 0, 1.0, 1.0)
    assert b.block_fwd(*ok) is not None
    for i, bad in ((0, x.double()), (0, x.cpu()), (0, x.t()), (1, x[:2]), (1, x.half()),
                   (2, w[:4]), (2, w.half()), (3, torch.ones(3, 8, device="cuda")),
                   (3, torch.ones(2, 4, device="cuda")), (4, w.view(2, 4)), (5, -1.0),
                   (5, float("nan")), (6, 2), (6, 0.5), (7, float("inf")), (7, "1")):
        args = list(ok)
        args[i] = bad
        assert b.block_fwd(*args) is None, i
        with pytest.raises((RuntimeError, ValueError, TypeError)):
            L.rms_norm_block_fwd(*args) if not (i == 6 and bad == 0.5) else int("x")
    assert b.grad_norm([x, x.cpu()]) is None and b.grad_norm([x.double()]) is None
    assert b.grad_clip([x], -1.0, 1e-6, None, None) is None
    assert b.grad_clip([x], 1.0, 1e-6, [x[:2]], None) is None
    assert b.grad_clip([x, x], 1.0, 1e-6, None, None) is None
    with pytest.raises(L.RMSNormError):
        L.rms_norm_grad_clip([x, x], 1.0)


def test_built_for_this_pytorch(L):
    assert L._binding.built_for == torch.__version__


@pytest.mark.gpu
@pytest.mark.parametrize("direct", [True, False])
def test_scaling_is_seen_by_autograd(L, other_way, direct):
    """A tensor that a graph has saved and that is scaled in place is noticed."""
    clip = L.rms_norm_grad_clip if direct else (
        lambda *a, **k: other_way(L.rms_norm_grad_clip, *a, **k))
    w = torch.ones(8, device="cuda", requires_grad=True)
    t = torch.full((8,), 3.0, device="cuda")
    loss = (w * t).sum()
    clip([t], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    out = torch.empty_like(t)
    v = out._version
    clip([t], 1.0, out=[out])
    assert out._version > v
    with torch.inference_mode():
        u = torch.full((8,), 3.0, device="cuda")
    clip([u], 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("x,gate", [((4, 6, 96), (4, 1, 96)), ((4, 6, 96), (4, 96)),
                                    ((2, 3, 4, 96), (2, 3, 1, 96)), ((3, 4, 96), (3, 4, 96))])
def test_gates_of_leading_dimensions(L, x, gate):
    a, r, g = (torch.randn(s, device="cuda") for s in (x, x, gate))
    w = torch.ones(96, device="cuda")
    got = L.rms_norm_block_fwd(a, r, None, g, w)[0]
    full = g.reshape(gate[:-1] + (1,) * (len(x) - len(gate)) + (96,))
    assert torch.allclose(got, r + full * a, rtol=1e-6, atol=1e-6)


@pytest.mark.gpu
def test_no_rows_and_no_gate_rows(L):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    w = torch.ones(96, device="cuda")
    for gate in (e(0, 1, 96), e(4, 96), e(96)):
        x = e(0, 5, 96)
        r, y, r1, r2 = L.rms_norm_block_fwd(x, x, w, gate, w)
        assert r.shape == y.shape == x.shape
        got = L.rms_norm_block_bwd(x, x, x, r, r1, r2, w, gate, w)
        assert got[3].shape == gate.shape
        assert all(torch.count_nonzero(v).item() == 0 for v in got)


@pytest.mark.gpu
def test_outputs_that_are_given(L):
    x, r = (torch.randn(4, 6, 96, device="cuda") for _ in range(2))
    w = torch.rand(96, device="cuda") + 1
    args = (x, r, w, None, w, 1e-5, 0, 1.0, 1.0)
    want = L.rms_norm_block_fwd(*args)
    outs = [torch.empty_like(v) for v in want]
    got = L._binding.block_fwd(*args, *outs)
    assert all(g.data_ptr() == o.data_ptr() for g, o in zip(got, outs))
    same(got, want)
    same(L.rms_norm_block_fwd(*args, *outs), want)
    for k, bad in ((0, torch.empty(24, 96, device="cuda")), (1, outs[1].half()),
                   (2, torch.empty(24, device="cuda")), (3, torch.empty(4, 6))):
        assert L._binding.block_fwd(*args, *outs[:k], bad, *outs[k + 1:]) is None
    back = (x, r, x, want[0], want[2], want[3], w, None, w, 0, 1.0, 1.0, True)
    ref = L.rms_norm_block_bwd(*back)
    ws = torch.empty(L.rms_norm_block_bwd_workspace_size(24, 96, 0), dtype=torch.uint8,
                     device="cuda")
    dx, dr = torch.empty_like(x), torch.empty_like(r)
    got = L._binding.block_bwd(*back, dx, dr, ws)
    assert got[0].data_ptr() == dx.data_ptr() and got[1].data_ptr() == dr.data_ptr()
    same(got, ref)
    same(L.rms_norm_block_bwd(*back, dx, dr, ws), ref)
    with pytest.raises(L.RMSNormError):                # too small: said by the other way
        L.rms_norm_block_bwd(*back, dx, dr, ws[:-16])
    with pytest.raises(L.RMSNormError):                # an output in an input
        L.rms_norm_block_fwd(*args, r, *outs[1:])
