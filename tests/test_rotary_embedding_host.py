"""Host-side checks of the head norm with rotation and of the embedding: the C
entries refuse bad arguments before any CUDA call, the Python layer bad
tensors before the library."""
import ctypes
import os

import pytest
import torch

FAKE, NULL = ctypes.c_void_p(0x10000), None   # never dereferenced
OK, ERR_NULL, SHAPE, EPS, DTYPE, ALIGN, WORKSPACE, ARG = 0, 1, 2, 3, 4, 5, 6, 8


@pytest.fixture(scope="module")
def L():
    import bwd_rms_norm_gb300 as lib
    from bwd_rms_norm_gb300 import build
    if not os.path.exists(lib.LIB_PATH):
        build.build()
    lib.load_library()
    return lib


def heads(L, at, b=0, t=0, h=0):
    return None if at is None else L._Heads(at, b, t, h)


def plain(L, at, n, tokens=4, dim=64):
    """A contiguous tensor of n heads at an address."""
    return heads(L, at, tokens * n * dim, n * dim, dim)


# addresses of the arguments, apart from one another; batch 2, 4 tokens, 4 + 2 heads of 64
def fwd(L, **k):
    g = lambda n, d: k[n] if n in k else d  # noqa: E731
    return L.load_library().rms_norm_rotary_fwd(
        g("q", plain(L, 0x100000, 4)), g("k", plain(L, 0x200000, 2)), g("qg", 0x300000),
        g("kg", 0x310000), g("freq", 0x320000), g("f64", 0), g("pos", 0x330000), g("p64", 0),
        g("ps", 4), g("qo", plain(L, 0x400000, 4)), g("ko", plain(L, 0x500000, 2)),
        g("rq", 0x600000), g("rk", 0x610000), g("batch", 2), g("tokens", 4), g("hq", 4),
        g("hk", 2), g("dim", 64), g("rot", 64), g("ilv", 0), g("eps", 1e-5), g("offset", 0),
        g("dtype", 1), None)


def bwd(L, **k):
    g = lambda n, d: k[n] if n in k else d  # noqa: E731
    lib = L.load_library()
    need = lib.rms_norm_rotary_bwd_workspace_size(2, g("tokens", 4), 4, 2, 64)
    return lib.rms_norm_rotary_bwd(
        g("dqo", plain(L, 0x700000, 4)), g("dko", plain(L, 0x710000, 2)),
        g("q", plain(L, 0x100000, 4)), g("k", plain(L, 0x200000, 2)), g("qg", 0x300000),
        g("kg", 0x310000), g("rq", 0x600000), g("rk", 0x610000), g("freq", 0x320000), g("f64", 0),
        g("pos", 0x330000), g("p64", 0), g("ps", 4), g("qo", plain(L, 0x400000, 4)),
        g("ko", plain(L, 0x500000, 2)), g("dqg", 0x800000), g("dkg", 0x810000), g("batch", 2),
        g("tokens", 4), g("hq", 4), g("hk", 2), g("dim", 64), g("rot", 64), g("ilv", 0),
        g("offset", 0), g("dtype", 1), g("ws", 0x900000), g("ws_bytes", need), None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_rotary_refusals(L, call):
    for bad in (dict(dtype=3), dict(dtype=-1)):
        assert call(L, **bad) == DTYPE, bad
    for bad in (dict(dim=0), dict(dim=1025), dict(rot=63), dict(rot=66), dict(rot=-2),
                dict(batch=-1), dict(tokens=-1), dict(hq=0), dict(hk=-1), dict(tokens=1 << 31),
                dict(batch=1 << 16, tokens=1 << 15), dict(hq=1 << 29), dict(ps=-1),
                dict(q=heads(L, 0x100000, 1024, -256, 64)),
                dict(ko=heads(L, 0x500000, 1 << 60, 128, 64))):
        assert call(L, **bad) == SHAPE, bad
    for bad in (dict(offset=2), dict(offset=-1), dict(ilv=2), dict(f64=2), dict(p64=-1)):
        assert call(L, **bad) == ARG, bad
    for bad in (dict(q=NULL), dict(k=NULL), dict(qo=NULL), dict(ko=NULL), dict(qg=NULL),
                dict(kg=NULL), dict(freq=NULL), dict(q=heads(L, None, 0, 0, 0)),
                dict(q=L._Heads(0, 1, 1, 1))):
        assert call(L, **bad) == ERR_NULL, bad
    for bad in (dict(q=plain(L, 0x100001, 4)), dict(ko=plain(L, 0x500001, 2)), dict(qg=0x300001),
                dict(freq=0x320002), dict(freq=0x320004, f64=1), dict(pos=0x330002),
                dict(pos=0x330004, p64=1), dict(rq=0x600002)):
        assert call(L, **bad) == ALIGN, bad


@pytest.mark.parametrize("call", [fwd, bwd])
def test_rotary_overlaps(L, call):
    q, k = 0x100000, 0x200000
    nb = 2 * 4 * 4 * 64 * 2   # bytes of q
    for bad in (dict(qo=plain(L, q + 2, 4)), dict(qo=plain(L, q + nb - 2, 4)),
                dict(qo=plain(L, k, 4)), dict(ko=plain(L, q, 2)), dict(qo=plain(L, 0x500000, 4)),
                dict(qo=heads(L, q, 1024, 64, 256)),       # its own bytes in another order
                dict(qo=heads(L, 0x400000, 1024, 256, 0)),  # heads on one another
                dict(qo=heads(L, 0x400000, 1024, 255, 64)),
                dict(qo=plain(L, 0x300000 - 64, 4)), dict(ko=plain(L, 0x320000 + 126, 2)),
                dict(qo=plain(L, 0x330000 - nb + 2, 4)), dict(qo=plain(L, 0x600000, 4))):
        assert call(L, **bad) == ARG, bad
    # views of one packed buffer that share an element: a head too far, a token too near
    t = 8 * 64
    for qo, ko in ((heads(L, 0x400000, 4 * t, t, 64), heads(L, 0x400000 + 3 * 128, 4 * t, t, 64)),
                   (heads(L, 0x400000, 4 * t, t, 64), heads(L, 0x400000 + 7 * 128, 4 * t, t, 64)),
                   (heads(L, 0x400000, 4 * t, t, 64),
                    heads(L, 0x400000 + 4 * 128, 4 * t + 256, t, 64))):
        assert call(L, qo=qo, ko=ko) == ARG


def places(at, strides, sizes, dim):
    """The elements of a tensor of heads, as numbers of 2-byte places."""
    import numpy as np
    n = np.full((1,), at // 2)
    for s, k in zip((*strides, 1), (*sizes, dim)):
        n = (n[:, None] + s * np.arange(k)).ravel()
    return n


@pytest.mark.parametrize("call", [fwd, bwd])
def test_rotary_overlaps_of_any_strides(L, call):
    import numpy as np
    rng = np.random.default_rng(0)
    met = 0
    for _ in range(2000):
        at, st = [0x400000, 0x400000 + 2 * int(rng.integers(0, 4000))], []
        for _ in range(2):
            h = 64 * int(rng.integers(1, 4)) + int(rng.integers(0, 3))
            t = int(rng.integers(1, 1200))
            st.append((int(rng.integers(1, 5000)), t, h))
        elements = [places(a, s, (2, 4, n), 64) for a, s, n in zip(at, st, (4, 2))]
        if all(len(set(e)) == len(e) for e in elements) and not set(elements[0]) & set(elements[1]):
            continue
        met += 1
        assert call(L, qo=heads(L, at[0], *st[0]), ko=heads(L, at[1], *st[1])) == ARG, (at, st)
    assert met > 500


def test_rotary_backward_refusals(L):
    for bad in (dict(dqo=NULL), dict(dko=NULL), dict(rq=NULL), dict(rk=NULL), dict(dqg=NULL),
                dict(dkg=NULL)):
        assert bwd(L, **bad) == ERR_NULL, bad
    for bad in (dict(dqg=0x300000), dict(dqg=0x810000), dict(qo=plain(L, 0x710000, 4)),
                dict(dqg=0x600000)):
        assert bwd(L, **bad) == ARG, bad
    assert bwd(L, dqg=0x800002) == ALIGN
    # few rows need none; more do
    assert L.rms_norm_rotary_bwd_workspace_size(2, 4, 4, 2, 64) == 0
    need = L.rms_norm_rotary_bwd_workspace_size(2, 1024, 4, 2, 64)
    assert need == 1216 * 64 * 4
    at = lambda a, n: plain(L, a, n, tokens=1024)  # noqa: E731
    long = dict(tokens=1024, dqo=at(0x700000, 4), dko=at(0xa00000, 2), q=at(0x100000, 4),
                k=at(0x200000, 2), qo=at(0x400000, 4), ko=at(0x500000, 2), ps=1024)
    assert bwd(L, ws=NULL, **long) == ERR_NULL
    assert bwd(L, ws_bytes=need - 1, **long) == WORKSPACE
    assert bwd(L, ws=0x900008, **long) == ALIGN
    for bad in (dict(ws=0x100000), dict(dkg=0x900000), dict(ws=0x610000 - 16)):
        assert bwd(L, **bad, **long) == ARG, bad
    for bad in ((-1, 4, 4, 2, 64), (2, 4, 0, 2, 64), (2, 4, 4, 2, 0), (0, 4, 4, 2, 64)):
        assert L.rms_norm_rotary_bwd_workspace_size(*bad) == 0
    assert L.rms_norm_rotary_bwd_workspace_size(8, 4096, 32, 8, 128) == 1216 * 128 * 4


def test_rotary_forward_refusals(L):
    for e in (-1e-6, float("nan"), float("inf")):
        assert fwd(L, eps=e) == EPS
    assert fwd(L, tokens=0, q=NULL, k=NULL) == OK and fwd(L, batch=0) == OK


def test_rotary_python_refusals(L):
    z = lambda *s, **k: torch.zeros(*s, **k)  # noqa: E731
    q, w, f = z(4, 2, 8), z(8), z(4)
    call = lambda **k: L.rms_norm_rotary_fwd(  # noqa: E731
        k.pop("q", q), k.pop("k", None), k.pop("qg", w), k.pop("kg", None), k.pop("f", f), **k)
    with pytest.raises(RuntimeError, match="CUDA"):
        call()
    with pytest.raises(RuntimeError, match="float32, bfloat16"):
        call(q=q.double())
    with pytest.raises(RuntimeError, match="head_dim"):
        call(q=z(4, 8))
    for off in (2, 0.5, -1):
        with pytest.raises(L.RMSNormError):
            call(offset=off)
    with pytest.raises(L.RMSNormError):
        call(interleaved=2)
    with pytest.raises(L.RMSNormError):
        L.rms_norm_rotary_bwd(q, None, q, None, w, None, z(4, 2), None, f, offset=3)


def emb(L, **k):
    g = lambda n, d: k[n] if n in k else d  # noqa: E731
    return L.load_library().rms_norm_embedding_fwd(
        g("ids", 0x1000), g("i64", 1), g("w", 0x100000), g("y", 0x200000), g("tokens", 8),
        g("vocab", 16), g("hidden", 64), g("scale", 1.0), g("wt", 1), g("yt", 1), None)


def emb_bwd(L, **k):
    g = lambda n, d: k[n] if n in k else d  # noqa: E731
    lib = L.load_library()
    need = lib.rms_norm_embedding_bwd_workspace_size(g("tokens", 8), 16, 64)
    return lib.rms_norm_embedding_bwd(
        g("y", 0x200000), g("ids", 0x1000), g("i64", 1), g("w", 0x100000), g("tokens", 8),
        g("vocab", 16), g("hidden", 64), g("scale", 1.0), g("pad", -1), g("acc", 0), g("yt", 1),
        g("wt", 1), g("ws", 0x300000), g("ws_bytes", need), None)


@pytest.mark.parametrize("call", [emb, emb_bwd])
def test_embedding_refusals(L, call):
    for bad in (dict(wt=3), dict(yt=-1), dict(wt=1, yt=2), dict(wt=2, yt=1)):
        assert call(L, **bad) == DTYPE, bad
    for bad in (dict(tokens=-1), dict(tokens=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1),
                dict(hidden=0), dict(hidden=65537)):
        assert call(L, **bad) == SHAPE, bad
    for bad in (dict(scale=float("nan")), dict(scale=float("inf")), dict(i64=2)):
        assert call(L, **bad) == ARG, bad
    for bad in (dict(ids=NULL), dict(w=NULL), dict(y=NULL)):
        assert call(L, **bad) == ERR_NULL, bad
    for bad in (dict(ids=0x1004), dict(w=0x100001), dict(y=0x200001),
                dict(ids=0x1002, i64=0)):
        assert call(L, **bad) == ALIGN, bad
    for bad in (dict(y=0x100000 + 16 * 128 - 2), dict(w=0x200000 - 2), dict(w=0x200000 + 1022)):
        assert call(L, **bad) == ARG, bad


def test_embedding_call_refusals(L):
    assert emb(L, y=0x1000 - 1022) == ARG and emb(L, tokens=0, y=NULL) == OK
    assert emb_bwd(L, w=0x1000 - 2046) == ARG and emb_bwd(L, acc=2) == ARG
    assert emb_bwd(L, tokens=0, acc=1) == OK
    # few tokens need no workspace; more do
    assert L.rms_norm_embedding_bwd_workspace_size(512, 16, 64) == 0
    need = L.rms_norm_embedding_bwd_workspace_size(600, 16, 64)
    many = dict(tokens=600, ids=0x20000)
    assert emb_bwd(L, ws=0x300008, **many) == ALIGN and emb_bwd(L, ws=NULL, **many) == ERR_NULL
    for at in (0x100000, 0x200000, 0x200000 + 600 * 128 - 16, 0x20000):
        assert emb_bwd(L, ws=at, **many) == ARG
    assert need > 0 and emb_bwd(L, ws_bytes=need - 1, **many) == WORKSPACE
    for bad in ((0, 16, 64), (-1, 16, 64), (8, 0, 64), (8, 16, 0), (8, 16, 65537)):
        assert L.rms_norm_embedding_bwd_workspace_size(*bad) == 0


def test_embedding_python_refusals(L):
    ids, w = torch.zeros(4, dtype=torch.int64), torch.zeros(8, 16)
    with pytest.raises(RuntimeError, match="CUDA"):
        L.rms_norm_embedding_fwd(ids, w)
    with pytest.raises(RuntimeError, match="vocab, hidden"):
        L.rms_norm_embedding_fwd(ids, w[0])
    with pytest.raises(RuntimeError, match="float32"):
        L.rms_norm_embedding_fwd(ids, w.bfloat16(), dtype=torch.float16)
    with pytest.raises(RuntimeError, match="int32 or int64"):
        L.rms_norm_embedding_fwd(ids.float(), w)
    with pytest.raises(RuntimeError, match="shape"):
        L.rms_norm_embedding_bwd(torch.zeros(3, 16), ids, 8)
    with pytest.raises(RuntimeError, match="accumulate"):
        L.rms_norm_embedding_bwd(torch.zeros(4, 16), ids, 8, accumulate=True)
    for pad in (-1, 8):
        with pytest.raises(L.RMSNormError):
            L.rms_norm_embedding_bwd(torch.zeros(4, 16), ids, 8, padding_idx=pad)


def test_modules(L):
    m = L.RMSNormRotary(64, offset=1, base=500000.0, rotary_dim=32)
    want = 500000.0 ** (torch.arange(16, dtype=torch.float64) * (-2.0 / 32))
    assert m.inv_freq.dtype == torch.float64 and torch.equal(m.inv_freq, want)
    m = m.to(torch.bfloat16)
    assert m.q_weight.dtype == torch.bfloat16 and torch.equal(m.inv_freq, want)
    assert sorted(m.state_dict()) == ["k_weight", "q_weight"] and not m.q_weight.any()
    assert L.RMSNormRotary(7).rotary_dim == 6
    for bad in (dict(offset=2), dict(rotary_dim=3), dict(rotary_dim=66)):
        with pytest.raises(ValueError):
            L.RMSNormRotary(64, **bad)
    e = L.RMSNormEmbedding(10, 4, padding_idx=3)
    assert not e.weight[3].any() and e.weight[2].any()
    with pytest.raises(ValueError):
        L.RMSNormEmbedding(10, 4, padding_idx=10)
