"""The head norm with rotation on the GPU against the float64 oracle.

Tolerances, from u = 2^-24 (half a step of fp32) and h = finfo(T).eps / 2
(the one rounding of a stored value).  rstd, a root of a sum of squares in
fp32, is within 1e-6 (a lane's few terms, then a tree).  An angle is held to
2^-25 of a half turn (1e-7), its sine and cosine to 2^-23 more; with the
products' roundings, elementwise, for the pair's columns i and j,

    y:      h |y| + 2e-6 (|u_i| + |u_j|)
    dv:     h |dv| + 4e-6 rstd (|gain| t + |vh| mean(|gain vh| t)),  t = |dy_i| + |dy_j|
    dgamma: ((n + 64) u + 2e-6) sum |vh| t over its n rows

plus the smallest subnormal of T, where a value underflows."""
import numpy as np
import pytest
import torch

from oracle import rotary as oro
from oracle.rms_norm import gain

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def near(got, ref, slack, what):
    h = torch.finfo(got.dtype).eps / 2
    off, most = np.abs(f64(got) - ref), h * np.abs(ref) + slack + TINY[got.dtype]
    bad = ~(off <= most)
    assert not bad.any(), (what, np.argwhere(bad)[0], off[bad][0], most[bad][0])


def laid_out(t, layout):
    """t [b, n, h, d] with the same values in another layout of memory."""
    b, n, h, d = t.shape
    if layout == "heads":          # a head's tokens next to one another
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "wide":           # in a buffer of wider rows: a packed product
        return torch.cat((t, t.new_full((b, n, 2, d), 77.0)), 2)[:, :, :h]
    if layout == "odd":            # from an odd element on, rows of an odd length
        flat = t.new_full((b, n, h * d + 3), 77.0)
        flat[:, :, 1:h * d + 1] = t.reshape(b, n, h * d)
        return flat[:, :, 1:h * d + 1].unflatten(-1, (h, d))
    return t.contiguous()


def make(b, n, hq, hk, d, rot, dtype, layout="", pos="ragged", base=10000.0, seed=0, std=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = T[dtype]
    c = {"q": (std * r(b, n, hq, d)).to(t), "k": (std * r(b, n, hk, d)).to(t) if hk else None,
         "q_gamma": (0.5 + 0.3 * r(d)).to(t), "k_gamma": (0.5 + 0.3 * r(d)).to(t) if hk else None,
         "dq": r(b, n, hq, d).to(t), "dk": r(b, n, hk, d).to(t) if hk else None}
    c = {k: None if v is None else laid_out(v.cuda(), layout) if v.dim() == 4 else v.cuda()
         for k, v in c.items()}
    p = torch.arange(rot // 2, dtype=torch.float64)
    c["freq"] = (base ** (p * (-2.0 / max(rot, 1)))).cuda()
    top = {"ragged": 5000, "far": 1 << 40}.get(pos, 1)
    c["pos"] = (torch.randint(-top if pos == "far" else 0, top, (b, n), generator=g).cuda()
                if pos != "none" else None)
    return c


def turn_of(c, interleaved):
    b, n, _, d = c["q"].shape
    pos = c["pos"].cpu().numpy() if c["pos"] is not None else np.tile(np.arange(n), (b, 1))
    return oro.matrices(np.broadcast_to(pos, (b, n)), f64(c["freq"]), d, interleaved)


def paired(t, pairs, interleaved):
    """|t_i| + |t_j| at a pair's columns, |t| elsewhere."""
    a = np.abs(t)
    out = a.copy()
    i = np.arange(pairs) * (2 if interleaved else 1)
    j = i + (1 if interleaved else pairs)
    out[..., i] = out[..., j] = a[..., i] + a[..., j]
    return out


def check_forward(c, got, eps, offset, interleaved):
    turn = turn_of(c, interleaved)
    for name, y, rs in (("q", got[0], got[2]), ("k", got[1], got[3])):
        if c[name] is None:
            assert y is None and rs is None
            continue
        ref, r, u = oro.forward(f64(c[name]), f64(c[name + "_gamma"]), turn, eps, offset)
        if rs is not None:
            assert np.max(np.abs(f64(rs) / r - 1)) <= 1e-6
        near(y, ref, 2e-6 * paired(u, len(c["freq"]), interleaved), name)


def check_backward(c, got, rstd, offset, interleaved):
    turn = turn_of(c, interleaved)
    for name, dv, dg, rs in (("q", got[0], got[2], rstd[0]), ("k", got[1], got[3], rstd[1])):
        if c[name] is None:
            assert dv is None and dg is None
            continue
        v, w, dy, r = f64(c[name]), f64(c[name + "_gamma"]), f64(c["d" + name]), f64(rs)
        ref, dw = oro.backward(dy, v, w, turn, r, offset)
        t, vh, a = paired(dy, len(c["freq"]), interleaved), np.abs(v * r[..., None]), np.abs(
            gain(w, offset))
        near(dv, ref, 4e-6 * r[..., None] * (a * t + vh * np.mean(a * vh * t, -1,
                                                                   keepdims=True)), "d" + name)
        n = int(np.prod(v.shape[:3]))
        near(dg, dw, ((n + 64) * U + 2e-6) * np.sum(vh * t, (0, 1, 2)), name + "_gamma")


def both(L, c, eps=1e-5, offset=0, interleaved=False):
    kind = dict(offset=offset, interleaved=interleaved)
    got = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"],
                                eps=eps, **kind)
    check_forward(c, got, eps, offset, interleaved)
    back = L.rms_norm_rotary_bwd(c["dq"], c["dk"], c["q"], c["k"], c["q_gamma"], c["k_gamma"],
                                 got[2], got[3], c["freq"], c["pos"], **kind)
    check_backward(c, back, got[2:], offset, interleaved)
    torch.cuda.synchronize()
    assert L.wait_timeouts() == 0
    return got, back


# (batch, tokens, q heads, k heads, head_dim, rotary_dim)
SIZES = [(1, 1, 1, 0, 2, 2), (1, 1, 1, 1, 1, 0), (1, 3, 2, 1, 3, 2), (2, 5, 3, 1, 7, 6),
         (1, 1, 32, 8, 128, 128), (1, 8, 32, 8, 128, 128), (3, 17, 4, 2, 64, 64),
         (1, 9, 5, 5, 80, 32), (2, 11, 7, 1, 40, 40), (1, 13, 6, 2, 72, 18), (2, 6, 3, 3, 112, 56),
         (1, 7, 8, 1, 96, 96), (1, 21, 2, 2, 192, 64), (1, 5, 9, 4, 256, 256), (1, 4, 2, 1, 512, 512),
         (1, 3, 2, 1, 1024, 1024), (1, 3, 1, 1, 1023, 1022), (2, 33, 16, 0, 128, 0),
         (1, 40, 71, 1, 64, 32), (1, 300, 8, 8, 8, 8), (1, 50, 3, 2, 16, 4), (1, 2, 1, 40, 24, 8)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(L, size, dtype, interleaved):
    odd = sum(size) % 2
    both(L, make(*size, dtype), offset=odd, interleaved=interleaved)


@pytest.mark.parametrize("layout", ["heads", "wide", "odd"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 32), (72, 36), (64, 16), (33, 10)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts(L, layout, dim, rot, dtype):
    for interleaved in (False, True):
        both(L, make(2, 19, 6, 2, dim, rot, dtype, layout), interleaved=interleaved)


def test_outputs_told_apart_from_inputs(L):
    # outputs between inputs of other strides in one buffer: what shares no element runs
    g = torch.Generator().manual_seed(12)
    c = make(2, 3, 2, 1, 16, 16, "bf16")
    number = lambda lo, hi: int(torch.randint(lo, hi, (1,), generator=g))  # noqa: E731
    ran = refused = 0
    for _ in range(400):
        buf = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
        spots = torch.arange(4096)
        views, taken = [], []
        row = number(200, 500)
        for n in (2, 1, 2, 1):
            h = number(16, 24)
            t = row if number(0, 4) else number(16 + h, 500)
            strides = (3 * max(row, t) if number(0, 4) else number(16 + h + 2 * t, 1600), t, h, 1)
            at = number(0, row)
            views.append(torch.as_strided(buf, (2, 3, n, 16), strides, at))
            taken.append(set(torch.as_strided(spots, (2, 3, n, 16), strides, at).flatten().tolist()))
        q, k, q_out, k_out = views
        if taken[0] & taken[1]:
            continue
        q.copy_(c["q"]), k.copy_(c["k"])
        args = q, k, c["q_gamma"], c["k_gamma"], c["freq"], c["pos"], 1e-5
        if (taken[0] | taken[1]) & (taken[2] | taken[3]) or taken[2] & taken[3]:
            with pytest.raises(L.RMSNormError):
                L.rms_norm_rotary_fwd(*args, q_out=q_out, k_out=k_out)
            refused += 1
        else:
            got = L.rms_norm_rotary_fwd(*args, q_out=q_out, k_out=k_out)
            check_forward(c, got, 1e-5, 0, False)
            ran += 1
    assert ran > 20 and refused > 20


@pytest.mark.parametrize("dim", [64, 33])
def test_offsets_beyond_32_bits(L, dim):
    # inputs and outputs side by side in one buffer of 2^32 elements and more
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    b, n, hq, hk = 2, 3, 4, 2
    far = (1 << 32) + (64 if dim == 64 else 65)
    buf = torch.empty(far + (3 << 30), dtype=torch.bfloat16, device="cuda")
    size = hq * 128

    def place(number, t):
        if t is None:
            return None
        view = torch.as_strided(buf, t.shape, (far, 1 << 30, 128, 1), number * size)
        return view.copy_(t)

    c = make(b, n, hq, hk, dim, 32, "bf16")
    c = dict(c, **{k: place(i, c[k]) for i, k in enumerate(("q", "k", "dq", "dk"))})
    out = [place(4, torch.zeros_like(c["q"])), place(5, torch.zeros_like(c["k"]))]
    got = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"],
                                eps=1e-5, q_out=out[0], k_out=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    check_forward(c, got, 1e-5, 0, False)
    back = L.rms_norm_rotary_bwd(c["dq"], c["dk"], c["q"], c["k"], c["q_gamma"], c["k_gamma"],
                                 got[2], got[3], c["freq"], c["pos"], dq=out[0], dk=out[1])
    check_backward(c, back, got[2:], 0, False)


@pytest.mark.parametrize("pos", ["none", "far"])
@pytest.mark.parametrize("dim", [64, 33])
def test_positions(L, pos, dim):
    c = make(2, 37, 3, 1, dim, 32, "f32", pos=pos, base=1e6)
    if pos == "far":
        # what 53 bits of an angle a position leave of 2^40 of them: turns * 2^-53 * 2^40 * 2 pi,
        # under 1e-3 of the tolerance at the frequency 2^-10 and below
        c["freq"] = c["freq"] * 2.0 ** -20
    both(L, c)
    if pos == "none":
        return
    for few in (c["pos"].remainder(1 << 20).int(), c["pos"].remainder(1 << 20)[1],
                c["pos"].repeat_interleave(3, 0)[::3]):      # int32, shared, strided rows
        both(L, dict(c, pos=few))
    both(L, dict(c, freq=c["freq"].float()))


def test_far_positions_at_full_frequency(L):
    """Positions to 2^31 at up to a radian each: 2^-63 of a turn a position is 1e-9 rad."""
    c = make(1, 40, 2, 1, 64, 64, "f32")
    at = torch.randint(0, 1 << 31, (1, 40), generator=torch.Generator().manual_seed(4))
    both(L, dict(c, pos=at.cuda()))
    both(L, dict(c, pos=at.int().cuda(), freq=c["freq"].float()))


def test_frequencies_of_any_size(L):
    # above a turn a position, negative, zero, tiny
    freq = torch.tensor([7.5, -0.3, 0.0, 1e-30, 6.283185307179586, -1e-25, 100.25, 3.0],
                        dtype=torch.float64).cuda()
    for pos in ("ragged", "none"):
        both(L, dict(make(1, 40, 2, 1, 16, 16, "f32", pos=pos), freq=freq))


def test_many_rows(L):
    # more units than warps at once, and sums of many partial rows
    for interleaved in (False, True):
        both(L, make(1, 3000, 9, 3, 64, 32, "bf16", pos="none"), interleaved=interleaved)
    both(L, make(1, 2500, 5, 1, 33, 32, "f16"))


@pytest.mark.parametrize("dim", [64, 33])
def test_rows_of_any_size(L, dim):
    c = make(1, 12, 2, 1, dim, 32, "f32")
    scale = torch.tensor([1e-30, 1e-18, 1e-6, 1.0, 1e6, 1e15, 1e18, 1e19, 1e25, 1e30, 1e37, 0.0])
    c["q"] = c["q"] * scale.cuda().view(1, 12, 1, 1)
    got, back = both(L, c, eps=1e-6)
    assert all(bool(torch.isfinite(t).all()) for t in (*got, *back))


@pytest.mark.parametrize("dim", [64, 33])
def test_values_that_are_not_finite_stay_in_their_row(L, dim):
    c = make(1, 6, 3, 2, dim, 32, "bf16")
    clean = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"])
    q = c["q"].clone()
    q[0, 2, 1, 5], q[0, 4, 0, 0] = float("nan"), float("inf")
    got = L.rms_norm_rotary_fwd(q, c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"])
    same = torch.ones(1, 6, 3, dtype=torch.bool)
    same[0, 2, 1] = same[0, 4, 0] = False
    assert torch.equal(got[0][same.cuda()], clean[0][same.cuda()])
    assert torch.equal(got[1], clean[1])
    assert bool(got[0][0, 2, 1].isnan().any()) and bool(got[0][0, 4, 0].isnan().any())


@pytest.mark.parametrize("dim,rot", [(128, 128), (72, 36), (33, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_in_a_packed_product(L, dim, rot, interleaved):
    b, n, hq, hk = 2, 23, 6, 2
    c = make(b, n, hq, hk, dim, rot, "bf16")
    args = c["q_gamma"], c["k_gamma"], c["freq"], c["pos"]
    want = L.rms_norm_rotary_fwd(c["q"], c["k"], *args, interleaved=interleaved)
    v = torch.full((b, n, hk, dim), 3.0, device="cuda", dtype=torch.bfloat16)
    for order in ((0, 1), (1, 2)):      # [b, n, heads, d] and [b, heads, n, d]
        move = lambda t: t.transpose(1, 2) if order == (1, 2) else t  # noqa: E731
        packed = torch.cat([move(t) for t in (c["q"], c["k"], v)], dim=3 - order[1])
        packed = packed.contiguous()
        q, k, rest = (move(t) for t in packed.split((hq, hk, hk), dim=3 - order[1]))
        version = packed._version
        got = L.rms_norm_rotary_fwd(q, k, *args, interleaved=interleaved, q_out=q, k_out=k,
                                    with_rstd=False)
        assert got[2] is None and got[3] is None and packed._version > version
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(rest, v)
    # the backward into the packed gradient, and over its own gradient
    grads = c["dq"], c["dk"], c["q"], c["k"], c["q_gamma"], c["k_gamma"], *want[2:], *args[2:]
    back = L.rms_norm_rotary_bwd(*grads, interleaved=interleaved)
    packed = torch.full((b, n, hq + 2 * hk, dim), 5.0, device="cuda", dtype=torch.bfloat16)
    dq, dk, rest = packed.split((hq, hk, hk), dim=2)
    got = L.rms_norm_rotary_bwd(*grads, interleaved=interleaved, dq=dq, dk=dk)
    assert all(torch.equal(a, e) for a, e in zip((dq, dk, *got[2:]), back))
    assert torch.equal(rest, torch.full_like(rest, 5.0))
    mine = [t.clone() for t in grads[:2]]
    got = L.rms_norm_rotary_bwd(*mine, *grads[2:], interleaved=interleaved, dq=mine[0], dk=mine[1])
    assert got[0] is mine[0] and all(torch.equal(a, e) for a, e in zip(got, back))


def test_three_dimensions_and_queries_alone(L):
    c = make(1, 20, 4, 2, 64, 64, "bf16")
    want = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"])
    got = L.rms_norm_rotary_fwd(c["q"][0], c["k"][0], c["q_gamma"], c["k_gamma"], c["freq"],
                                c["pos"][0])
    assert all(torch.equal(a, b[0]) for a, b in zip(got, want))
    alone = L.rms_norm_rotary_fwd(c["q"], None, c["q_gamma"], None, c["freq"], c["pos"])
    assert torch.equal(alone[0], want[0]) and alone[1] is None and alone[3] is None
    shared = c["q"][:, :, :1].expand(1, 20, 4, 64)      # one head for all
    got = L.rms_norm_rotary_fwd(shared, None, c["q_gamma"], None, c["freq"], c["pos"])
    assert torch.equal(got[0], want[0][:, :, :1].expand(1, 20, 4, 64))
    with pytest.raises(L.RMSNormError):
        L.rms_norm_rotary_fwd(shared, None, c["q_gamma"], None, c["freq"], c["pos"], q_out=shared)
    with pytest.raises(L.RMSNormError):                 # over the keys
        L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"],
                              k_out=c["q"][:, :, 1:3])


def test_no_tokens(L):
    c = make(1, 4, 3, 2, 64, 64, "bf16")
    e = lambda t: t[:, :0]  # noqa: E731
    got = L.rms_norm_rotary_fwd(e(c["q"]), e(c["k"]), c["q_gamma"], c["k_gamma"], c["freq"],
                                e(c["pos"]))
    assert got[0].shape == (1, 0, 3, 64) and got[3].shape == (1, 0, 2)
    back = L.rms_norm_rotary_bwd(e(c["dq"]), e(c["dk"]), e(c["q"]), e(c["k"]), c["q_gamma"],
                                 c["k_gamma"], got[2], got[3], c["freq"], e(c["pos"]))
    assert not back[2].any() and not back[3].any() and back[2].shape == (64,)


@pytest.mark.parametrize("dim", [128, 33])
def test_a_cluster_of_any_size_for_few_rows(L, dim):
    for tokens in (1, 2, 9, 33, 64, 255, 256, 257):     # 8 rows a token: to 2048 rows and beyond
        c = make(1, tokens, 8, 2, dim, 32, "f32")
        both(L, c)
        launches = L.last_launch_count()
        assert launches == (1 if tokens <= 256 else 2)
    try:
        for sms in (1, 3, 8):
            L.rms_norm_set_sm_budget(sms)
            both(L, make(1, 100, 4, 1, dim, 32, "bf16"))
    finally:
        L.rms_norm_set_sm_budget(0)


@pytest.mark.parametrize("tokens", [60, 500])
def test_same_bits_every_time_and_under_a_budget(L, tokens):
    c = make(1, tokens, 8, 2, 128, 128, "bf16")
    args = [c[k] for k in ("dq", "dk", "q", "k", "q_gamma", "k_gamma")]
    rstd = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"],
                                 c["pos"])[2:]
    first = L.rms_norm_rotary_bwd(*args, *rstd, c["freq"], c["pos"])
    for _ in range(3):
        again = L.rms_norm_rotary_bwd(*args, *rstd, c["freq"], c["pos"])
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    try:
        for sms in (1, 7):
            assert L.rms_norm_set_sm_budget(sms) is None or True
            both(L, c)
    finally:
        L.rms_norm_set_sm_budget(0)


def test_streams_and_graphs(L):
    c = make(2, 64, 8, 2, 128, 128, "bf16", "wide")
    names = "q_gamma", "k_gamma", "freq", "pos"
    fwd = lambda **k: L.rms_norm_rotary_fwd(c["q"], c["k"], *[c[n] for n in names], **k)  # noqa: E731
    want = fwd()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fwd(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    def step():
        y = fwd()
        return y, L.rms_norm_rotary_bwd(c["dq"], c["dk"], c["q"], c["k"], c["q_gamma"],
                                        c["k_gamma"], y[2], y[3], c["freq"], c["pos"])

    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, back = step()
    c["q"].mul_(-2.0)
    c["pos"].add_(17)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(c, y, 1e-6, 0, False)
    check_backward(c, back, y[2:], 0, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_autograd(L, interleaved):
    c = make(2, 9, 4, 2, 64, 32, "f32")
    leaves = [c[n].detach().clone().requires_grad_() for n in ("q", "k", "q_gamma", "k_gamma")]
    q, k = L.rms_norm_rotary(*leaves, c["freq"], c["pos"], 1e-5, 1, interleaved)
    torch.autograd.backward((q, k), (c["dq"], c["dk"]))
    rstd = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"],
                                 1e-5, 1, interleaved)[2:]
    check_backward(c, [t.grad for t in leaves], rstd, 1, interleaved)
    # against differences of the function itself, along a direction: its second-order
    # part is under 1e-4 of a step of 1e-3, its rounding 2e-7 * sqrt(terms) / 1e-3
    g = torch.Generator(device="cuda").manual_seed(3)
    to = [torch.randn(t.shape, generator=g, device="cuda") for t in leaves]

    def f(e):
        with torch.no_grad():
            y = L.rms_norm_rotary(*[t + e * d for t, d in zip(leaves, to)], c["freq"], c["pos"],
                                  1e-5, 1, interleaved)
        return sum(float((a.double() * b.double()).sum()) for a, b in zip(y, (c["dq"], c["dk"])))

    slope = sum(float((t.grad.double() * d.double()).sum()) for t, d in zip(leaves, to))
    assert abs((f(1e-3) - f(-1e-3)) / 2e-3 - slope) < 5e-2 + 1e-3 * abs(slope)
    # one output alone, and an input that is a view with a stride in its last dimension
    leaf = c["q"].detach().clone().requires_grad_()
    y = L.rms_norm_rotary(leaf.transpose(-1, -2).contiguous().transpose(-1, -2), c["k"],
                          c["q_gamma"], c["k_gamma"], c["freq"], c["pos"])[0]
    y.backward(c["dq"])
    assert leaf.grad.shape == leaf.shape and bool(leaf.grad.any())


def test_autograd_of_queries_alone_and_of_one_output(L):
    c = make(1, 9, 4, 2, 64, 32, "f32")
    q, w = (c[n].detach().clone().requires_grad_() for n in ("q", "q_gamma"))
    L.rms_norm_rotary(q, None, w, None, c["freq"], c["pos"]).backward(c["dq"])
    both_q, both_w, k = (c[n].detach().clone().requires_grad_() for n in ("q", "q_gamma", "k"))
    L.rms_norm_rotary(both_q, k, both_w, c["k_gamma"], c["freq"], c["pos"])[0].backward(c["dq"])
    assert torch.equal(q.grad, both_q.grad) and torch.equal(w.grad, both_w.grad)
    assert not k.grad.any()
    # one head of keys for all, and one row of positions for every batch entry
    one = torch.randn(2, 9, 1, 64, device="cuda", requires_grad=True)
    y = L.rms_norm_rotary(one.expand(2, 9, 4, 64), None, w, None, c["freq"],
                          torch.arange(9, device="cuda").expand(2, 9))
    y.sum().backward()
    assert one.grad.shape == one.shape and bool(one.grad.any())


def test_two_streams_at_once(L):
    cs = [make(1, 700, 8, 2, 128, 128, "bf16", seed=s) for s in (1, 2)]

    def step(c):
        y = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"])
        return *y, *L.rms_norm_rotary_bwd(c["dq"], c["dk"], c["q"], c["k"], c["q_gamma"],
                                          c["k_gamma"], y[2], y[3], c["freq"], c["pos"])

    want = [step(c) for c in cs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], [None, None]
    for _ in range(10):
        for i, (s, c) in enumerate(zip(streams, cs)):
            with torch.cuda.stream(s):
                got[i] = step(c)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for u, v in zip(got, want) for a, b in zip(u, v))


def test_inference_mode(L):
    c = make(1, 5, 4, 2, 64, 32, "bf16")
    with torch.inference_mode():
        q, k = c["q"].clone(), c["k"].clone()
        L.rms_norm_rotary_fwd(q, k, c["q_gamma"], c["k_gamma"], c["freq"], c["pos"], q_out=q,
                              k_out=k, with_rstd=False)
    want = L.rms_norm_rotary_fwd(c["q"], c["k"], c["q_gamma"], c["k_gamma"], c["freq"], c["pos"])
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_module(L):
    m = L.RMSNormRotary(64, base=500000.0, rotary_dim=32, device="cuda", dtype=torch.bfloat16)
    c = make(2, 9, 4, 2, 64, 32, "bf16", pos="none", base=500000.0)
    q, k = m(c["q"], c["k"])
    want = L.rms_norm_rotary_fwd(c["q"], c["k"], m.q_weight, m.k_weight, c["freq"])
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    (q.float().sum() + k.float().square().sum()).backward()
    assert m.q_weight.grad.dtype == torch.bfloat16 and bool(m.k_weight.grad.any())
