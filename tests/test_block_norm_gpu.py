"""The block norm on the GPU against the float64 oracle.

Tolerances, from u = 2^-24 (half a step of fp32) and h = finfo(T).eps / 2
(the one rounding of a stored value).  A sum over a row of n values in fp32,
in any order, is off by at most n u times the sum of the terms' sizes; the
kernels' orders (a thread's few columns, then trees) keep it under 32 u, and
rstd, a root of such a sum, within 1e-6.  So, elementwise,

    r:      h |r| + 2e-6 (|a res| + |b gate z|)         (rstd and 8 products)
    y:      h |y| + 4e-6 (rstd_next |w2| (|a res| + |b gate z|) + |y|)
    dres:   h |dres| + 4e-6 |a| t,  t = |dr| + rstd_next (|g| + |rh| mean|g rh|)
    dx:     h |dx| + 8e-6 rstd_post (|w| t + |xh| mean(|w xh| t))
    sums:   (n + 64) u sum|terms| over the n rows, plus 4e-6 sum |terms|

plus the smallest subnormal of T, where a value underflows."""
import itertools

import numpy as np
import pytest
import torch

from oracle import block_norm as obn
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
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def near(got, ref, slack, what):
    h = torch.finfo(got.dtype).eps / 2
    ref = np.asarray(ref).reshape(tuple(got.shape))
    off = np.abs(f64(got) - ref)
    most = h * np.abs(ref) + slack.reshape(ref.shape) + TINY[got.dtype]
    bad = ~(off <= most)
    assert not bad.any(), (what, np.argwhere(bad)[0], off[bad][0], most[bad][0])


def make(rows, hidden, dtype, res, post, gates, nxt, seed=0, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = dict(x=(n(rows, hidden) * 1.5 * std).to(T[dtype]),
             residual=(n(rows, hidden) * 2.0 * std).to(T[res]),
             post_gamma=(1 + 0.1 * n(hidden)).to(T[dtype]) if post else None,
             gate=(0.6 + 0.3 * n(gates, hidden)).to(T[dtype]) if gates else None,
             next_gamma=(1 + 0.1 * n(hidden)).to(T[dtype]) if nxt else None)
    g = dict(dy=n(rows, hidden).to(T[dtype]) if nxt else None,
             dresidual_out=n(rows, hidden).to(T[res]))
    return d, g


def cuda(d, move=lambda t: t.cuda()):
    return {k: None if v is None else move(v) for k, v in d.items()}


def oracle_args(d):
    return [f64(d[k]) for k in ("x", "residual", "post_gamma", "gate", "next_gamma")]


def check_forward(got, d, eps, offset, a, b):
    r, y, r1, r2 = got
    x, res, w1, gate, w2 = oracle_args(d)
    er, ey, er1, er2 = obn.forward(x, res, w1, gate, w2, eps, offset, a, b)
    rows, hidden = x.shape
    z = x if w1 is None else x * er1[:, None] * gain(w1, offset)
    terms = np.abs(a * res) + np.abs(b * obn.gate_rows(gate, rows, hidden) * z)
    near(r, er, 2e-6 * terms, "r")
    assert (y is None) == (w2 is None) and (r1 is None) == (w1 is None)
    if w1 is not None:
        assert np.max(np.abs(f64(r1).ravel() / er1 - 1)) <= 1e-6
    if w2 is not None:
        # the statistic of a sum that cancels is as exact as its terms
        worst = np.sqrt(np.mean(terms ** 2, -1) / (np.mean(er ** 2, -1) + eps))
        assert np.all(np.abs(f64(r2).ravel() / er2 - 1) <= 1e-6 * np.maximum(1, worst))
        near(y, ey, 4e-6 * (er2[:, None] * np.abs(gain(w2, offset)) * terms
                            + np.abs(ey) * np.maximum(1, worst)[:, None]), "y")


def check_backward(got, d, g, r, r1, r2, offset, a, b):
    """Against the oracle on the very r, rstd_post and rstd_next that the call read."""
    x, _, w1, gate, w2 = oracle_args(d)
    r, r1, r2 = f64(r), f64(r1), f64(r2)
    r1, r2 = (None if v is None else v.ravel() for v in (r1, r2))
    dy, dr = f64(g["dy"]), f64(g["dresidual_out"])
    ref = obn.backward(dy, dr, x, r, w1, gate, w2, r1, r2, offset, a, b)
    rows, hidden = x.shape
    n = rows + 64
    t = np.zeros_like(x) if dr is None else np.abs(dr)
    if w2 is not None:
        rh, gy = r * r2[:, None], dy * gain(w2, offset)
        t = t + r2[:, None] * (np.abs(gy) + np.abs(rh) * np.mean(np.abs(gy * rh), -1)[:, None])
        near(got[4], ref[4], (n * U + 4e-6) * np.sum(np.abs(dy * rh), 0), "dnext")
    near(got[1], ref[1], 4e-6 * abs(a) * t, "dresidual")
    xh = x if w1 is None else x * r1[:, None]
    gr = obn.gate_rows(gate, rows, hidden)
    one = np.ones(hidden) if w1 is None else gain(w1, offset)
    w = np.abs(b * gr * one)
    if w1 is None:
        near(got[0], ref[0], 8e-6 * w * t, "dx")
    else:
        m = np.mean(w * np.abs(xh) * t, -1)[:, None]
        near(got[0], ref[0], 8e-6 * r1[:, None] * (w * t + np.abs(xh) * m), "dx")
        near(got[2], ref[2], (n * U + 8e-6) * np.sum(np.abs(b * gr * xh) * t, 0), "dpost")
    if gate is not None:
        k = gate.size // hidden
        per = np.sum((np.abs(b * xh * one) * t).reshape(k, rows // k, hidden), 1)
        near(got[3], ref[3], (n * U + 8e-6) * per, "dgate")
    for v, w_ in zip(got[2:], (w1, gate, w2)):
        assert (v is None) == (w_ is None)


def run_and_check(L, d, g, eps=1e-5, offset=0, a=1.0, b=1.0, move=lambda t: t.cuda(), **kw):
    dc, gc = cuda(d, move), cuda(g, move)
    out = L.rms_norm_block_fwd(**dc, eps=eps, offset=offset, residual_scale=a, branch_scale=b)
    check_forward(out, d, eps, offset, a, b)
    r, _, r1, r2 = out
    args = (gc["dy"], gc["dresidual_out"], dc["x"], r, r1, r2)
    opts = dict(post_gamma=dc["post_gamma"], gate=dc["gate"], next_gamma=dc["next_gamma"],
                offset=offset, residual_scale=a, branch_scale=b)
    back = L.rms_norm_block_bwd(*args, **opts)
    check_backward(back, d, g, r, r1, r2, offset, a, b)
    again = L.rms_norm_block_bwd(*args, **opts)
    assert all(u is None or torch.equal(u, v) for u, v in zip(back, again))
    assert L.wait_timeouts() == 0
    return out, back


TYPES = [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")]
NORMS = [(True, True), (False, True), (True, False)]


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("post,nxt", NORMS)
@pytest.mark.parametrize("gates", [0, 1, 5])
def test_types_and_parts(L, dtype, res, post, nxt, gates):
    d, g = make(35, 512, dtype, res, post, gates, nxt, seed=gates)
    run_and_check(L, d, g, offset=0, a=0.5, b=1.25)


# one token to thousands, widths with every vector tail, odd widths, widths
# of one and several warps a row, rows split over a cluster, wider than that
SHAPES = [(1, 1), (1, 4096), (2, 7), (3, 8), (7, 24), (64, 128), (33, 250), (19, 264), (1000, 256),
          (5, 520), (305, 1000), (61, 1001), (700, 1024), (153, 2048), (9, 2056), (11, 2999),
          (160, 4096), (6, 4104), (155, 5120), (21, 8191), (157, 8192), (5, 8200), (7, 12288),
          (4, 16384), (3, 16392), (5, 24576), (2, 32768), (3, 65536), (2, 65535)]


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
def test_shapes(L, rows, hidden, dtype, res):
    d, g = make(rows, hidden, dtype, res, True, 1, True, seed=rows + hidden)
    run_and_check(L, d, g, offset=1, eps=1e-6)


@pytest.mark.parametrize("rows,hidden", [(4000, 512), (2500, 1024), (1300, 4096), (700, 8192),
                                         (400, 16384)])
@pytest.mark.parametrize("post,nxt", NORMS)
def test_many_rows_a_unit(L, rows, hidden, post, nxt):
    d, g = make(rows, hidden, "bf16", "bf16", post, 4, nxt, seed=hidden)
    run_and_check(L, d, g)


@pytest.mark.parametrize("rows,gates,hidden", [(1, 1, 256), (12, 12, 512), (600, 600, 264),
                                               (600, 200, 1024), (900, 3, 77), (1216, 76, 2048),
                                               (304, 152, 8192), (310, 310, 4096)])
@pytest.mark.parametrize("post", [True, False])
def test_gate_rows(L, rows, gates, hidden, post):
    """Gates for each row, for runs shorter and longer than a CTA's rows."""
    d, g = make(rows, hidden, "bf16", "bf16", post, gates, True, seed=gates)
    run_and_check(L, d, g, b=0.5)


@pytest.mark.parametrize("dtype,res", TYPES)
def test_no_gradient_from_the_stream(L, dtype, res):
    for hidden in (1024, 999):
        d, g = make(70, hidden, dtype, res, True, 2, True, seed=9)
        g["dresidual_out"] = None
        run_and_check(L, d, g)


def misaligned(t):
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype,res", TYPES)
def test_unaligned(L, dtype, res):
    d, g = make(45, 1024, dtype, res, True, 3, True, seed=4)
    run_and_check(L, d, g, move=misaligned)


@pytest.mark.parametrize("k", range(7))
def test_one_unaligned_tensor(L, k):
    d, g = make(20, 512, "bf16", "bf16", True, 2, True, seed=k)
    hit = list(range(7))[k]
    count = itertools.count()
    run_and_check(L, d, g, move=lambda t: misaligned(t) if next(count) == hit else t.cuda())


def test_no_dgate(L):
    d, g = make(40, 1024, "bf16", "bf16", True, 4, True)
    out, back = run_and_check(L, d, g)
    dc, gc = cuda(d), cuda(g)
    less = L.rms_norm_block_bwd(gc["dy"], gc["dresidual_out"], dc["x"], out[0], out[2], out[3],
                                dc["post_gamma"], dc["gate"], dc["next_gamma"], with_dgate=False)
    assert less[3] is None
    for i in (0, 1, 2, 4):
        assert torch.equal(less[i], back[i])


@pytest.mark.parametrize("hidden", [64, 1024, 4096, 1001])
def test_zero_rows(L, hidden):
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = e(hidden).fill_(1)
    r, y, r1, r2 = L.rms_norm_block_fwd(e(0, hidden), e(0, hidden), w, w, w)
    assert r.shape == y.shape == (0, hidden) and r1.shape == r2.shape == (0,)
    got = L.rms_norm_block_bwd(e(0, hidden), e(0, hidden), e(0, hidden), r, r1, r2, w, w, w)
    for v in got[2:]:
        assert v.shape == (hidden,) and torch.count_nonzero(v).item() == 0


@pytest.mark.parametrize("hidden", [1024, 8192, 1001])
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32")])
def test_sums_of_squares_beyond_fp32(L, dtype, res, hidden):
    """Rows whose squares overflow fp32 are finite after their norms."""
    d, g = make(9, hidden, dtype, res, True, 1, True, seed=2)
    d["x"][::2] *= 2.0 ** 90
    d["residual"][1::3] *= 2.0 ** 85
    out = L.rms_norm_block_fwd(**cuda(d), eps=1e-5)
    check_forward(out, d, 1e-5, 0, 1.0, 1.0)


@pytest.mark.parametrize("hidden", [1024, 1001])
def test_rows_of_zeros_and_of_infinities(L, hidden):
    d, g = make(6, hidden, "f32", "f32", True, 0, True, seed=1)
    d["x"][0] = 0.0
    d["residual"][0] = 0.0
    d["x"][2, 5] = float("inf")
    d["residual"][3, 6] = float("nan")
    r, y, r1, r2 = L.rms_norm_block_fwd(**cuda(d), eps=0.0)
    # an all-zero row with eps 0: rstd is infinite and 0 * inf is not a number
    assert torch.isinf(r1[0]).item() and torch.isnan(r[0]).all().item()
    # an infinity: rstd 0, the element itself is inf * 0
    assert r1[2].item() == 0.0 and torch.isnan(r[2, 5]).item()
    assert torch.isnan(y[2]).all().item() and torch.isnan(y[3]).all().item()
    keep = [1, 4, 5]
    sub = {k: (v[keep] if v is not None and v.dim() == 2 else v) for k, v in d.items()}
    check_forward((r[keep], y[keep], r1[keep], r2[keep]), sub, 0.0, 0, 1.0, 1.0)


def test_outputs_stay_in_bounds(L):
    """What stands before and behind the outputs is left as it was."""
    for rows, hidden in ((37, 1024), (5, 8192), (3, 16392), (11, 1001), (1, 4096)):
        d, g = make(rows, hidden, "bf16", "bf16", True, 1, True)
        pad, n = 64, rows * hidden
        bufs = [torch.full((n + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda")
                for _ in range(4)]
        r, y, dx, dres = (v[pad:pad + n].view(rows, hidden) for v in bufs)
        dc, gc = cuda(d), cuda(g)
        out = L.rms_norm_block_fwd(**dc, residual_out=r, y=y)
        L.rms_norm_block_bwd(gc["dy"], gc["dresidual_out"], dc["x"], r, out[2], out[3],
                             dc["post_gamma"], dc["gate"], dc["next_gamma"], dx=dx, dresidual=dres)
        for v in bufs:
            assert (v[:pad] == 7).all().item() and (v[pad + n:] == 7).all().item()


def test_offsets_past_32_bits(L):
    """More than 2^31 elements: the last rows against the oracle."""
    rows, hidden = (1 << 31) // 4096 + 40, 4096
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    res = torch.empty_like(x).normal_(generator=gen)
    w = torch.rand(hidden, generator=gen, device="cuda").to(torch.bfloat16)
    r, y, r1, r2 = L.rms_norm_block_fwd(x, res, w, None, w, eps=1e-5)
    tail = slice(rows - 48, rows)
    d = dict(x=x[tail], residual=res[tail], post_gamma=w, gate=None, next_gamma=w)
    check_forward((r[tail], y[tail], r1[tail], r2[tail]), d, 1e-5, 0, 1.0, 1.0)
    back = L.rms_norm_block_bwd(x, res, x, r, r1, r2, w, None, w)
    # dx and dresidual are of their own row alone; the sums are of all rows
    ref = obn.backward(f64(x[tail]), f64(res[tail]), f64(x[tail]), f64(r[tail]), f64(w), None,
                       f64(w), f64(r1[tail]), f64(r2[tail]))
    for got, want in zip(back[:2], ref):
        off = np.abs(f64(got[tail]) - want)
        assert np.all(off <= 2.0 ** -8 * np.abs(want) + 1e-4 * np.abs(want).max())


def test_another_stream_and_its_workspace(L):
    d, g = make(300, 2048, "bf16", "bf16", True, 4, True)
    dc, gc = cuda(d), cuda(g)
    out, back = run_and_check(L, d, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = L.rms_norm_block_fwd(**dc, eps=1e-5, stream=side)
    b = L.rms_norm_block_bwd(gc["dy"], gc["dresidual_out"], dc["x"], o[0], o[2], o[3],
                             dc["post_gamma"], dc["gate"], dc["next_gamma"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for u, v in zip(out + back, o + b):
        assert torch.equal(u, v)


def test_sm_budget(L):
    """Fewer CTAs, each with more rows."""
    d, g = make(2000, 1024, "bf16", "bf16", True, 2, True)
    L.rms_norm_set_sm_budget(7)
    try:
        run_and_check(L, d, g)
    finally:
        L.rms_norm_set_sm_budget(0)


def test_captured_and_replayed(L):
    """Two graphs, each with its own workspace, replayed with new inputs."""
    d, g = make(130, 4096, "bf16", "bf16", True, 2, True)
    dc, gc = cuda(d), cuda(g)
    names = ("post_gamma", "gate", "next_gamma")

    def step():
        o = L.rms_norm_block_fwd(**dc)
        return o, L.rms_norm_block_bwd(gc["dy"], gc["dresidual_out"], dc["x"], o[0], o[2], o[3],
                                       **{k: dc[k] for k in names})

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(step())
    for seed in (5, 6):
        d2, g2 = make(130, 4096, "bf16", "bf16", True, 2, True, seed=seed)
        for k, v in {**d2, **g2}.items():
            (dc if k in dc else gc)[k].copy_(v)
        for gr in graphs:
            gr.replay()
        want = step()
        for got in outs:
            for u, v in zip(got[0] + got[1], want[0] + want[1]):
                assert torch.equal(u, v)


@pytest.mark.parametrize("dtype,res", TYPES)
def test_autograd_matches_direct_calls(L, dtype, res):
    d, g = make(24, 768, dtype, res, True, 4, True)
    out, back = run_and_check(L, d, g, offset=1, a=0.5)
    leaf = {k: v.clone().view(4, 6, 768) if k in ("x", "residual") else v.clone()
            for k, v in cuda(d).items()}
    for v in leaf.values():
        v.requires_grad_()
    r, y = L.rms_norm_block(leaf["x"], leaf["residual"], leaf["post_gamma"],
                            leaf["gate"].view(4, 1, 768), leaf["next_gamma"], 1e-5, 1, 0.5)
    gc = cuda(g)
    torch.autograd.backward([r, y], [gc["dresidual_out"].view(r.shape), gc["dy"].view(y.shape)])
    assert torch.equal(r.detach().view(24, 768), out[0])
    assert torch.equal(y.detach().view(24, 768), out[1])
    for k, v in zip(("x", "residual", "post_gamma", "gate", "next_gamma"), back):
        got = leaf[k].grad
        assert got.dtype == leaf[k].dtype
        assert torch.equal(got.reshape(v.shape), v.to(got.dtype)), k


def test_autograd_with_one_output_used(L):
    d, g = make(24, 512, "f32", "f32", True, 1, True)
    for post in (True, False):
        w = dict(cuda(d), post_gamma=cuda(d)["post_gamma"] if post else None)
        d1 = dict(d, post_gamma=d["post_gamma"] if post else None)
        for use in ("r", "y"):
            t = {k: None if v is None else v.clone().requires_grad_() for k, v in w.items()}
            r, y = L.rms_norm_block(t["x"], t["residual"], t["post_gamma"], t["gate"],
                                    t["next_gamma"])
            up = torch.randn(24, 512, device="cuda")
            (r if use == "r" else y).backward(up)
            _, _, r1, r2 = obn.forward(*oracle_args(d1), 1e-6)
            zero = np.zeros((24, 512))
            ref = obn.backward(f64(up) if use == "y" else zero, f64(up) if use == "r" else zero,
                               f64(t["x"]), f64(r), f64(t["post_gamma"]), f64(t["gate"]),
                               f64(t["next_gamma"]), r1, r2)
            for k, v in zip(("x", "residual", "post_gamma", "gate"), ref):
                if v is not None:
                    assert np.allclose(f64(t[k].grad), v, rtol=1e-4, atol=1e-4), (post, use, k)


def test_autograd_against_differences(L):
    """The gradient of a scalar of the fp32 outputs against central
    differences of the same scalar from the float64 oracle."""
    d, _ = make(3, 16, "f32", "f32", True, 3, True, seed=8)
    t = {k: v.cuda().requires_grad_() for k, v in d.items()}
    rng = np.random.default_rng(0)
    u, v = rng.standard_normal((2, 3, 16)).astype(np.float32)
    r, y = L.rms_norm_block(t["x"], t["residual"], t["post_gamma"], t["gate"], t["next_gamma"],
                            1e-5, 0, 0.9, 1.1)
    ((r * torch.from_numpy(u).cuda()).sum() + (y * torch.from_numpy(v).cuda()).sum()).backward()
    base = oracle_args(d)

    def loss(args):
        r, y, _, _ = obn.forward(*args, 1e-5, 0, 0.9, 1.1)
        return np.sum(r * u) + np.sum(y * v)

    for i, k in enumerate(("x", "residual", "post_gamma", "gate", "next_gamma")):
        got = f64(t[k].grad)
        for at in [tuple(rng.integers(0, n) for n in base[i].shape) for _ in range(12)]:
            up, down = [w.copy() for w in base], [w.copy() for w in base]
            up[i][at] += 1e-5
            down[i][at] -= 1e-5
            want = (loss(up) - loss(down)) / 2e-5
            # fp32 gradients of sums of under 100 terms of size about 1
            assert abs(got[at] - want) <= 100 * 8 * U * 10 + 1e-8, (k, at)


def test_module_trains_in_a_stack(L):
    """Layers in a row, one feeding the next: gradients reach every weight."""
    torch.manual_seed(0)
    layers = [L.RMSNormBlock(256, gate_init=0.1, device="cuda") for _ in range(3)]
    h = torch.randn(2, 5, 256, device="cuda", requires_grad=True)
    r, y = h, h
    for m in layers:
        r, y = m(torch.tanh(y), r)
    (y.square().mean() + r.mean()).backward()
    for m in layers:
        for p in m.parameters():
            assert p.grad.shape == p.shape and torch.isfinite(p.grad).all().item()
            assert p.grad.abs().max().item() > 0
    assert torch.isfinite(h.grad).all().item()


# rows that start anywhere in 16 bytes: periods of 2, 4 and 8 rows, narrow ones
# (several to a stage) to ones over several CTAs, tensors whose last row ends
# inside 16 bytes
ODD = [(65601, 65), (32800, 132), (16401, 257), (4203, 1001), (1031, 2050), (514, 4093),
       (259, 8191), (177, 12001), (133, 16002), (129, 16389), (128, 65535)]


@pytest.mark.parametrize("rows,hidden", ODD)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
def test_odd_widths(L, rows, hidden, dtype, res):
    d, g = make(rows, hidden, dtype, res, True, rows % 2, True, seed=rows + hidden)
    run_and_check(L, d, g, a=0.5)


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("post,nxt", NORMS)
def test_odd_widths_and_parts(L, post, nxt, dtype, res):
    d, g = make(1037, 2051, dtype, res, post, 1, nxt, seed=6)
    run_and_check(L, d, g, offset=1)
    g["dresidual_out"] = g["dresidual_out"] if not nxt else None
    run_and_check(L, d, g, offset=1)


@pytest.mark.parametrize("post,nxt", NORMS)
@pytest.mark.parametrize("rows,gates,hidden", [(1290, 5, 1033), (6150, 3, 131), (600, 2, 4098),
                                               (768, 3, 2049), (8192, 32, 1026)])
def test_odd_widths_and_gate_rows(L, post, nxt, rows, gates, hidden):
    d, g = make(rows, hidden, "bf16", "bf16", post, gates, nxt, seed=gates)
    run_and_check(L, d, g, b=0.5)


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,hidden", [(32800, 130), (4206, 1001), (520, 4093), (260, 9001)])
def test_odd_widths_beside_infinities(L, dtype, res, rows, hidden):
    """What is copied of the rows before and after a row does not reach it."""
    d, g = make(rows, hidden, dtype, res, True, 1, True, seed=3)

    def run():
        c = cuda(d)
        out = L.rms_norm_block_fwd(**c, eps=1e-5)
        weights = [c[k] for k in ("post_gamma", "gate", "next_gamma")]
        back = L.rms_norm_block_bwd(g["dy"].cuda(), g["dresidual_out"].cuda(), c["x"], out[0],
                                    out[2], out[3], *weights)
        return [v.reshape(rows, -1) for v in list(out) + list(back[:2])]

    clean = run()
    for k in ("x", "residual"):
        d[k][::2] = float("nan")
    for k in ("dy", "dresidual_out"):
        g[k][::2] = float("inf")
    for u, v in zip(clean, run()):
        assert torch.equal(u[1::2], v[1::2])
        assert torch.isnan(v[::2]).any(-1).all()


@pytest.mark.parametrize("rows,hidden,gates", [(4100, 1024, 1), (600, 4096, 0), (8300, 512, 0),
                                               (1024, 4096, 2)])
def test_unaligned_weights_alone(L, rows, hidden, gates):
    d, g = make(rows, hidden, "bf16", "bf16", True, gates, True, seed=5)
    run_and_check(L, d, g, move=lambda t: t.cuda() if t.shape[0] == rows else misaligned(t))


@pytest.mark.parametrize("rows,gates", [(700, 350), (4000, 4000), (640, 20), (5000, 40)])
@pytest.mark.parametrize("hidden", [256, 77])
def test_gate_rows_of_few_segments(L, rows, gates, hidden):
    d, g = make(rows, hidden, "f32", "f32", True, gates, True, seed=7)
    run_and_check(L, d, g)


@pytest.mark.parametrize("rows,hidden", [(3, 65536), (200, 65536), (5, 65535), (2, 1), (300, 1)])
@pytest.mark.parametrize("dtype,res", [("bf16", "f32"), ("f32", "f32")])
def test_widest_and_narrowest(L, rows, hidden, dtype, res):
    d, g = make(rows, hidden, dtype, res, True, 1, True, seed=8)
    run_and_check(L, d, g)


# which kernels a shape runs: one that falls to a slower family keeps every
# comparison of results green
@pytest.mark.parametrize("rows,hidden,gates,fwd,bwd", [
    (8, 4096, 0, "block_fwd_tma", "block_bwd_tma"), (512, 128, 1, "block_fwd_tma", "block_bwd_tma"),
    (300, 4096, 3, "block_fwd_tma", "block_bwd_tma"), (64, 65536, 1, "block_fwd_tma",
                                                       "block_bwd_tma"),
    (300, 8200, 1, "block_fwd_tma", "block_bwd_tma"), (1100, 4097, 1, "block_fwd_tma",
                                                       "block_bwd_tma"),
    (1000, 1001, 8, "block_fwd_loop", "block_bwd_loop"), (777, 1001, 0, "block_fwd_loop",
                                                          "block_bwd_tma"),
    (8, 4097, 0, "block_fwd_loop", "block_bwd_loop"), (1100, 33, 1, "block_fwd_loop",
                                                       "block_bwd_loop")])
def test_kernels_a_shape_runs(L, rows, hidden, gates, fwd, bwd):
    d, g = make(rows, hidden, "bf16", "bf16", True, gates, True)
    dc, gc = cuda(d), cuda(g)
    out = L.rms_norm_block_fwd(**dc)
    assert fwd in L.last_kernels()[0], L.last_kernels()
    L.rms_norm_block_bwd(gc["dy"], gc["dresidual_out"], dc["x"], out[0], out[2], out[3],
                         dc["post_gamma"], dc["gate"], dc["next_gamma"])
    names = L.last_kernels()
    assert len(names) == 2 and bwd in names[0] and "block_bwd_sums" in names[1], names


@pytest.mark.parametrize("sms", [1, 7, 8, 20, 100])
@pytest.mark.parametrize("rows,hidden,gates", [(1100, 4097, 1), (1280, 1033, 5), (300, 8200, 0)])
def test_odd_widths_on_few_sms(L, sms, rows, hidden, gates):
    d, g = make(rows, hidden, "bf16", "bf16", True, gates, True, seed=sms)
    L.rms_norm_set_sm_budget(sms)
    try:
        run_and_check(L, d, g)
        if sms < 8 and hidden % 2:
            assert "block_bwd_loop" in L.last_kernels()[0]
    finally:
        L.rms_norm_set_sm_budget(0)
