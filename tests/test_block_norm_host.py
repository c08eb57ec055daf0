"""Host-side checks of the block norm: the C entries refuse bad arguments
before any CUDA call, the Python layer bad tensors before the library."""
import ctypes
import os

import pytest
import torch

FAKE, NULL = ctypes.c_void_p(0x1000), None   # never dereferenced


@pytest.fixture(scope="module")
def L():
    import bwd_rms_norm_gb300 as lib
    from bwd_rms_norm_gb300 import build
    if not os.path.exists(lib.LIB_PATH):
        build.build()
    lib.load_library()
    return lib


def fwd(L, **k):
    g = lambda n, d=FAKE: k.get(n, d)  # noqa: E731
    return L.load_library().rms_norm_block_fwd(
        g("x"), g("res"), g("post"), g("gate"), k.get("gates", 2), g("next"), g("r"), g("y"),
        g("r1"), g("r2"), k.get("rows", 4), k.get("hidden", 64), k.get("a", 1.0), k.get("b", 1.0),
        k.get("eps", 1e-5), k.get("offset", 0), k.get("dtype", 1), k.get("res_dtype", 1), None)


def bwd(L, **k):
    lib = L.load_library()
    g = lambda n, d=FAKE: k.get(n, d)  # noqa: E731
    need = lib.rms_norm_block_bwd_workspace_size(4, 64, 2)
    return lib.rms_norm_block_bwd(
        g("dy"), g("dr"), g("x"), g("r"), g("post"), g("gate"), k.get("gates", 2), g("next"),
        g("r1"), g("r2"), g("dx"), g("dres"), g("dpost"), g("dgate"), g("dnext"),
        k.get("rows", 4), k.get("hidden", 64), k.get("a", 1.0), k.get("b", 1.0),
        k.get("offset", 0), k.get("dtype", 1), k.get("res_dtype", 1), g("ws"),
        k.get("ws_bytes", need), None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_shared_refusals(L, call):
    for bad in (dict(dtype=3), dict(dtype=-1), dict(res_dtype=2), dict(dtype=0, res_dtype=1),
                dict(res_dtype=7)):
        assert call(L, **bad) == 4, bad
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(hidden=0), dict(hidden=65537),
                dict(gates=3), dict(gates=0), dict(gates=8), dict(gates=-2)):
        assert call(L, **bad) == 2, bad
    for bad in (dict(offset=2), dict(a=float("nan")), dict(b=float("inf"))):
        assert call(L, **bad) == 8, bad
    assert call(L, post=NULL, next=NULL) == 1
    assert call(L, x=NULL) == 1


def test_forward_refusals(L):
    for k in ("res", "r", "y", "r1", "r2"):
        assert fwd(L, **{k: NULL}) == 1, k
    for e in (-1e-6, float("nan"), float("inf")):
        assert fwd(L, eps=e) == 3
    assert fwd(L, rows=0, gates=1, x=NULL, res=NULL, r=NULL, y=NULL, r1=NULL, r2=NULL) == 0
    assert L.last_launch_count() == 0


def test_backward_refusals(L):
    for k in ("dy", "r", "r1", "r2", "dx", "dres", "dpost", "dnext", "ws"):
        assert bwd(L, **{k: NULL}) == 1, k
    # without the next norm the stream's gradient is the only one
    assert bwd(L, next=NULL, dnext=NULL, dr=NULL) == 1
    assert bwd(L, ws=ctypes.c_void_p(0x1004)) == 5
    need = L.rms_norm_block_bwd_workspace_size(4, 64, 2)
    assert bwd(L, ws_bytes=need - 4) == 6


def test_workspace_size(L):
    size = L.rms_norm_block_bwd_workspace_size
    assert size(4, 64, 2) == (3 * 4 + 2) * 64 * 4
    assert size(10000, 64, 0) == (3 * 608 + 1) * 64 * 4
    assert size(0, 64, 0) == 0 and size(4, 0, 0) == 0 and size(4, 64, 5) == 0
    assert size(4, 64, -1) == 0
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "rms_norm.h")).read()
    assert f"#define RMSN_BLOCK_MAX_PARTIALS {L.RMSN_BLOCK_MAX_PARTIALS}\n" in text


def good(**k):
    t = dict(x=torch.zeros(4, 8), residual=torch.zeros(4, 8), post_gamma=torch.ones(8),
             gate=torch.ones(2, 8), next_gamma=torch.ones(8))
    t.update(k)
    return t


@pytest.mark.parametrize("change,match", [
    (dict(), "CUDA"),
    (dict(x=torch.zeros(4, 8, dtype=torch.int32)), "float32, bfloat16"),
    (dict(post_gamma=None, next_gamma=None), "nothing to normalise"),
    (dict(residual=torch.zeros(4, 9)), "shape"),
    (dict(residual=torch.zeros(4, 8, dtype=torch.float16)), "float32"),
    (dict(x=torch.zeros(4, 8, dtype=torch.float16), post_gamma=None, gate=None,
          next_gamma=torch.ones(8, dtype=torch.float16),
          residual=torch.zeros(4, 8, dtype=torch.bfloat16)), "float16"),
    (dict(post_gamma=torch.ones(8, dtype=torch.float16)), "float32"),
    (dict(next_gamma=torch.ones(2, 4)), "shape"),
    (dict(gate=torch.ones(3, 8)), "divide"),
    (dict(gate=torch.ones(8, 8)), "divide"),
    (dict(gate=torch.ones(2, 4)), "columns"),
    (dict(gate=torch.tensor(1.0)), "columns"),
    (dict(gate=torch.ones(0, 8)), "divide"),
    (dict(gate=torch.ones(2, 8, dtype=torch.float16)), "float32"),
    (dict(y=torch.zeros(4, 9)), "shape"),
    (dict(rstd_next=torch.zeros(3)), "elements"),
    (dict(residual_out=torch.zeros(4, 8, dtype=torch.float16)), "float32"),
])
def test_python_forward_refusals(L, change, match):
    with pytest.raises(RuntimeError, match=match):
        L.rms_norm_block_fwd(**good(**change))


@pytest.mark.parametrize("change,match", [
    (dict(), "CUDA"),
    (dict(dy=None), "needed"),
    (dict(rstd_next=None), "needed"),
    (dict(rstd_post=None), "needed"),
    (dict(next_gamma=None, dresidual_out=None), "needed"),
    (dict(dy=torch.zeros(4, 9)), "shape"),
    (dict(dresidual_out=torch.zeros(4, 8, dtype=torch.float16)), "float32"),
    (dict(rstd_post=torch.zeros(5)), "elements"),
    (dict(dx=torch.zeros(8, 4)), "shape"),
])
def test_python_backward_refusals(L, change, match):
    t = good(dy=torch.zeros(4, 8), dresidual_out=torch.zeros(4, 8), rstd_post=torch.ones(4),
             rstd_next=torch.ones(4))
    t["residual_out"] = t.pop("residual")
    t.update(change)
    with pytest.raises(RuntimeError, match=match):
        L.rms_norm_block_bwd(**t)


def test_module_host_side(L):
    m = L.RMSNormBlock(16, gate_init=0.1)
    assert sorted(n for n, _ in m.named_parameters()) == ["gate", "next_weight", "post_weight"]
    assert torch.equal(m.post_weight.detach(), torch.ones(16))
    assert torch.equal(m.gate.detach(), torch.full((16,), 0.1))
    m = L.RMSNormBlock(16, offset=1, post=False, dtype=torch.bfloat16)
    assert [n for n, _ in m.named_parameters()] == ["next_weight"]
    assert torch.count_nonzero(m.next_weight).item() == 0
    with pytest.raises(ValueError):
        L.RMSNormBlock(16, offset=2)
    with pytest.raises(ValueError):
        L.RMSNormBlock(16, post=False, next=False)
    with pytest.raises(ValueError):
        L.RMSNormBlock(16, gate_init=1.0)(torch.zeros(2, 16), torch.zeros(2, 16), torch.ones(16))
    with pytest.raises(RuntimeError, match="CUDA"):
        m(torch.zeros(3, 16, dtype=torch.bfloat16), torch.zeros(3, 16, dtype=torch.bfloat16))


def apart(n):
    return {k: ctypes.c_void_p(0x100000 * (i + 1)) for i, k in enumerate(n)}


FWD = ("x", "res", "post", "gate", "next", "r", "y", "r1", "r2")
BWD = ("dy", "dr", "x", "r", "post", "gate", "next", "r1", "r2", "dx", "dres", "dpost", "dgate",
       "dnext", "ws")


@pytest.mark.parametrize("call,names,outs", [
    (fwd, FWD, ("r", "y", "r1", "r2")),
    (bwd, BWD, ("dx", "dres", "dpost", "dgate", "dnext", "ws"))])
def test_outputs_that_share_memory(L, call, names, outs):
    """Every pair of an output with another argument: at the same address, and
    where the argument's last byte is the output's first."""
    size = dict(x=512, res=512, post=128, gate=256, next=128, r=512, y=512, r1=16, r2=16, dy=512,
                dr=512, dx=512, dres=512, dpost=256, dgate=512, dnext=256, ws=0)
    for o in outs:
        for k in names:
            if k == o:
                continue
            at = apart(names)
            at[k] = at[o]
            assert call(L, **at) == 8, (o, k)
            if k != "ws" and o != "ws":
                at[o] = ctypes.c_void_p(at[k].value + size[k] - 4)
                assert call(L, **at) == 8, (o, k)


@pytest.mark.parametrize("x,gate,runs", [
    ((4, 6, 8), (4, 8), True), ((4, 6, 8), (4, 1, 8), True), ((4, 6, 8), (4, 6, 8), True),
    ((4, 6, 8), (8,), True), ((4, 6, 8), (1, 1, 8), True), ((4, 6, 8), (24, 8), True),
    ((1, 6, 8), (1, 6, 8), True), ((4, 1, 8), (4, 8), True), ((12, 8), (4, 8), True),
    ((4, 6, 8), (1, 6, 8), False), ((4, 6, 8), (6, 8), False), ((4, 4, 8), (4, 8), False),
    ((2, 3, 4, 8), (2, 1, 4, 8), False), ((2, 3, 4, 8), (2, 3, 1, 8), True),
    ((2, 3, 4, 8), (2, 3, 8), True), ((2, 3, 3, 8), (3, 1, 8), False)])
def test_gates_that_broadcast_otherwise(L, x, gate, runs):
    t = good(x=torch.zeros(x), residual=torch.zeros(x), gate=torch.ones(gate))
    with pytest.raises(RuntimeError, match="CUDA" if runs else "repeat|divide"):
        L.rms_norm_block_fwd(**t)
