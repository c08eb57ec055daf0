"""The direct binding of the head norm with rotation and of the embedding: it
declines what needs a second look, and where it takes a call the results are
those of the other way."""
import ctypes
import os
import subprocess

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
    b, q, w, s = L._binding, torch.zeros(4, 2, 8), torch.ones(8), torch.ones(4, 2)
    f, ids = torch.ones(4), torch.zeros(4, dtype=torch.int64)
    assert b.rotary_fwd(q, None, w, None, f, None, 1e-5, 0, False, True) is None    # not CUDA
    assert b.rotary_fwd(q, None) is None
    assert b.rotary_fwd(None, None, w, None, f, None, 1e-5, 0, False, True) is None
    assert b.rotary_fwd("q", 3, w, None, f, None, 1e-5, 0, False, True) is None
    assert b.rotary_bwd(q, None, q, None, w, None, s, None, f, None, 0, False) is None
    assert b.embedding_fwd(ids, q[0], 1.0, None) is None
    assert b.embedding_fwd(ids, None, 1.0, None) is None and b.embedding_fwd(ids) is None
    assert b.embedding_bwd(q, ids, 5, 1.0, None, None, None, False) is None
    assert b.embedding_bwd(q, ids, "5", 1.0, None, None, None, False) is None
    for bad in ((1, 2), (0,) * 6, tuple("abcdef")):
        with pytest.raises((ValueError, TypeError)):
            b.init_more(*bad)


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
            assert u.shape == v.shape and u.dtype == v.dtype and u.stride() == v.stride()
            assert torch.equal(u, v)


def rotary(dtype, layout, keys, dims=4):
    t = getattr(torch, dtype)
    r = lambda *s: torch.randn(*s, device="cuda").to(t)  # noqa: E731
    packed = r(2, 6, 8, 32)
    q, k = packed[:, :, :4], packed[:, :, 4:6]
    if layout == "heads":
        q, k = r(2, 4, 6, 32).transpose(1, 2), r(2, 2, 6, 32).transpose(1, 2)
    elif layout == "both":       # heads outside, and inside wider rows
        q, k = r(2, 4, 6, 40).transpose(1, 2)[..., :32], r(2, 2, 6, 40).transpose(1, 2)[..., :32]
    elif layout == "one":
        q, k = q[:1, :, :1], k[:1, :, :1]
    if dims == 3:
        q, k = q[0], k[0]
    return (q, k, r(32), r(32)) if keys else (q, None, r(32), None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("layout", ["packed", "heads", "both", "one"])
@pytest.mark.parametrize("keys,dims", [(True, 4), (False, 4), (True, 3)])
def test_rotary(L, other_way, dtype, layout, keys, dims):
    x = rotary(dtype, layout, keys, dims)
    lead = x[0].shape[:-2]
    f32 = torch.rand(16, device="cuda")
    for freq, pos in ((f32, None), (f32.double(), torch.randint(0, 99, lead, device="cuda")),
                      (f32[:3].contiguous(), torch.arange(6, device="cuda").int()), (None, None),
                      (f32[:0], None)):
        args = *x, freq, pos
        kw = dict(eps=1e-3, offset=1, interleaved=True)
        got = L._binding.rotary_fwd(*args, 1e-3, 1, True, True)
        assert got is not None
        same(L.rms_norm_rotary_fwd(*args, **kw), got)
        same(other_way(L.rms_norm_rotary_fwd, *args, **kw), got)
        same(other_way(L.rms_norm_rotary_fwd, *args, with_rstd=False, **kw),
             L._binding.rotary_fwd(*args, 1e-3, 1, True, False))
        up = [None if t is None else torch.randn_like(t) for t in x[:2]]
        back = *up, *x, *got[2:], freq, pos
        grads = L._binding.rotary_bwd(*back, 1, True)
        assert grads is not None
        same(other_way(L.rms_norm_rotary_bwd, *back, offset=1, interleaved=True), grads)


@pytest.mark.gpu
def test_rotary_given_outputs(L, other_way):
    x = rotary("bfloat16", "packed", True)
    freq = torch.rand(16, device="cuda")
    want = L.rms_norm_rotary_fwd(*x, freq)
    outs = [torch.zeros_like(t) for t in want]
    before = [t._version for t in outs]
    got = L._binding.rotary_fwd(*x, freq, None, 1e-6, 0, False, True, *outs)
    assert all(a is b for a, b in zip(got, outs)) and all(
        t._version > v for t, v in zip(outs, before))
    same(got, want)
    for k in range(4):
        for bad in (outs[k].double(), outs[k][:, :3], outs[k].cpu(), 3):
            given = *outs[:k], bad, *outs[k + 1:]
            assert L._binding.rotary_fwd(*x, freq, None, 1e-6, 0, False, True, *given) is None
    assert L._binding.rotary_fwd(*x, freq, None, 1e-6, 0, False, False, *outs) is None
    with pytest.raises(RuntimeError, match="not wanted"):
        L.rms_norm_rotary_fwd(*x, freq, rstd_q=outs[2], with_rstd=False)
    up = [torch.randn_like(t) for t in x[:2]]
    back = *up, *x, *want[2:], freq, None
    grads = other_way(L.rms_norm_rotary_bwd, *back)
    dq, dk = (torch.zeros_like(t) for t in grads[:2])
    assert L.rms_norm_rotary_bwd_workspace_size(2, 6, 4, 2, 32) == 0
    got = L._binding.rotary_bwd(*back, 0, False, dq, dk, None)
    assert got[0] is dq and got[1] is dk
    same(got, grads)


@pytest.mark.gpu
def test_rotary_given_workspace(L, other_way):
    q = torch.randn(600, 8, 32, device="cuda").bfloat16()
    w, freq = torch.ones(32, device="cuda").bfloat16(), torch.rand(16, device="cuda")
    rstd = L.rms_norm_rotary_fwd(q, None, w, None, freq)[2]
    back = torch.randn_like(q), None, q, None, w, None, rstd, None, freq, None
    grads = other_way(L.rms_norm_rotary_bwd, *back)
    need = L.rms_norm_rotary_bwd_workspace_size(1, 600, 8, 0, 32)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    same(L._binding.rotary_bwd(*back, 0, False, None, None, ws), grads)
    same(L._binding.rotary_bwd(*back, 0, False), grads)
    assert L._binding.rotary_bwd(*back, 0, False, None, None, ws[:-16]) is None
    with pytest.raises(L.RMSNormError):
        L.rms_norm_rotary_bwd(*back, workspace=ws[:-16])


@pytest.mark.gpu
def test_rotary_declines(L):
    q, k, qg, kg = rotary("bfloat16", "packed", True)
    f = torch.rand(16, device="cuda")
    pos = torch.zeros(2, 6, dtype=torch.int64, device="cuda")
    call = lambda *a: L._binding.rotary_fwd(*a, 1e-6, 0, False, True)  # noqa: E731
    assert call(q, k, qg, kg, f, pos) is not None
    for bad in ((q, k, qg, None, f, pos), (q, None, qg, kg, f, pos), (q.half(), k, qg, kg, f, pos),
                (q, k[:, :5], qg, kg, f, pos), (q, k[0], qg, kg, f, pos),
                (q, k, qg[:31], kg, f, pos), (q, k, qg, kg.float(), f, pos),
                (q, k, qg, kg, f.half(), pos), (q, k, qg, kg, torch.rand(17, device="cuda"), pos),
                (q, k, qg, kg, torch.rand(16, 2, device="cuda")[:, 0], pos),
                (q, k, qg, kg, f, pos[:, :5]), (q, k, qg, kg, f, pos.float()),
                (q, k, qg, kg, f, pos[:1]), (q, k, qg, kg, f, pos.cpu()), (q[0, 0], k, qg, kg, f, pos),
                (q[..., ::2], k[..., ::2], qg[:16], kg[:16], f[:8], pos)):
        assert call(*bad) is None, bad
        with pytest.raises(RuntimeError):
            L.rms_norm_rotary_fwd(*bad)
    for kind in ((0.5, False, True), (2, False, True), (0, 2, True), (0, 0.5, True)):
        assert L._binding.rotary_fwd(q, k, qg, kg, f, pos, 1e-6, *kind) is None
    with pytest.raises(L.RMSNormError):
        L.rms_norm_rotary_fwd(q, k, qg, kg, f, pos, eps=-1.0)


PAIRS = [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float32"),
         ("float32", "bfloat16")]


@pytest.mark.gpu
@pytest.mark.parametrize("types", PAIRS, ids="-".join)
@pytest.mark.parametrize("shape", [(7,), (2, 3), (1,), ()])
def test_embedding(L, other_way, types, shape):
    t, u = (getattr(torch, n) for n in types)
    ids = torch.randint(-1, 9, shape, device="cuda")
    w, dy = torch.randn(9, 20, device="cuda").to(t), torch.randn(*shape, 20, device="cuda").to(t)
    for i in (ids, ids.int()):
        got = L._binding.embedding_fwd(i, w, 1.5, u)
        assert got is not None
        same(other_way(L.rms_norm_embedding_fwd, i, w, 1.5, u), got)
        y = torch.zeros_like(got)
        assert L._binding.embedding_fwd(i, w, 1.5, None, y) is y and torch.equal(y, got)
        back = L._binding.embedding_bwd(dy, i, 9, 1.5, 2, u, None, False)
        assert back is not None
        same(other_way(L.rms_norm_embedding_bwd, dy, i, 9, 1.5, 2, u), back)
        start = [torch.ones_like(back) for _ in range(2)]
        version = start[0]._version
        got = L._binding.embedding_bwd(dy, i, 9, 1.5, None, None, start[0], True)
        assert got is start[0] and got._version > version
        same(other_way(L.rms_norm_embedding_bwd, dy, i, 9, 1.5, dweight=start[1],
                       accumulate=True), got)


@pytest.mark.gpu
def test_embedding_declines(L):
    ids, w = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(5, 8, device="cuda")
    dy = torch.ones(4, 8, device="cuda")
    for bad in ((ids.float(), w, 1.0, None), (ids, w.double(), 1.0, None), (ids, w[0], 1.0, None),
                (ids, w[:, ::2], 1.0, None), (ids, w, 1.0, torch.float64), (ids.cpu(), w, 1.0, None),
                (ids, w.half(), 1.0, torch.bfloat16), (ids.view(2, 2).T[:1], w.cpu(), 1.0, None),
                (ids, w, float("inf"), None)):
        assert L._binding.embedding_fwd(*bad) is None, bad
        with pytest.raises(RuntimeError):
            L.rms_norm_embedding_fwd(*bad)
    plain = (dy, ids, 5, 1.0, None, None, None, False)
    assert L._binding.embedding_bwd(*plain) is not None
    for at, bad in ((0, dy[:3]), (0, dy.cpu()), (0, dy.double()), (1, ids.float()), (2, 0),
                    (2, -5), (3, float("nan")), (4, 5), (4, -1), (5, torch.float64),
                    (6, torch.ones(4, 8, device="cuda")), (7, True)):
        args = *plain[:at], bad, *plain[at + 1:]
        assert L._binding.embedding_bwd(*args) is None, (at, bad)
        with pytest.raises(RuntimeError):
            L.rms_norm_embedding_bwd(*args)


@pytest.mark.gpu
def test_a_failed_launch_is_not_made_again(L, tmp_path):
    (tmp_path / "stub.c").write_text(
        "#include <stddef.h>\nint calls;\nint entry() { ++calls; return 7; }\n"
        "size_t workspace() { return 64; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", str(tmp_path / "stub.c"), "-o",
                    str(tmp_path / "stub.so")], check=True)
    stub = ctypes.CDLL(str(tmp_path / "stub.so"))
    at = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    entry, workspace = at(stub.entry), at(stub.workspace)
    q, w, s = torch.ones(4, 2, 8, device="cuda"), torch.ones(8, device="cuda"), torch.ones(
        4, 2, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    L._binding.init_more(entry, entry, workspace, entry, entry, workspace)
    try:
        for k, call in enumerate((
                lambda: L.rms_norm_rotary_fwd(q, None, w, None, None),
                lambda: L.rms_norm_rotary_bwd(q, None, q, None, w, None, s, None, None),
                lambda: L.rms_norm_embedding_fwd(ids, q[0]),
                lambda: L.rms_norm_embedding_bwd(q[:, 0].contiguous(), ids, 5))):
            with pytest.raises(L.RMSNormError, match="status 7") as e:
                call()
            assert e.value.status == 7 and ctypes.c_int.in_dll(stub, "calls").value == k + 1
    finally:
        L._load_binding(L.load_library())
