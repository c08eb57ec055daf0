"""The gradient norm and clip on the GPU against sums in 64 bits.

Tolerances, from u = 2^-24: squares are added in fp32 within at most 32
elements of a thread in a tree of 8 (at most 32 + 3 roundings, one of them
the square's own), to about u^2 beyond, so the sum is within 36 u, its root
within 18 u, and the fp32 norm within 19 u.  The factor has that error and one
rounding, an output the product's and that of its type: h + 22 u, h =
finfo(T).eps / 2, plus the smallest subnormal where it underflows."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
DT = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


def make(sizes, dtypes, seed=0, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * std).to(dtypes[k % len(dtypes)])
            for k, n in enumerate(sizes)]


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def factor64(norm, max_norm, eps=1e-6):
    return min(1.0, max_norm / (norm + eps)) if math.isfinite(norm) and norm + eps > 0 else 1.0


def check(L, grads, max_norm, out=None, in_place=True, eps=1e-6):
    keep = [g.clone() for g in grads]
    want = norm64(keep)
    got = L.rms_norm_grad_norm(grads)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(got.item() - want) <= 19 * U * want + 2.0 ** -149
    f = factor64(want, max_norm, eps)
    norm = L.rms_norm_grad_clip(grads, max_norm, eps, out)
    assert norm.item() == got.item()
    for k, o in zip(keep, grads if out is None else out):
        ref = k.double() * f
        off = (o.double() - ref).abs()
        most = (torch.finfo(o.dtype).eps / 2 + 22 * U) * ref.abs() + TINY[o.dtype]
        assert bool((off <= most).all()), (k.dtype, o.dtype, off.max().item())
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(keep, grads))


SIZES = [[1], [7], [4096], [8191, 8192, 8193], [1, 2, 3, 5, 8, 1000, 64, 1023],
         [0, 5, 0, 0, 70000, 0], [4097] * 40, list(range(1, 300)), [1_000_003, 17, 2_500_000]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtypes", [[d] for d in DT] + [DT])
def test_in_place(L, sizes, dtypes):
    check(L, make(sizes, dtypes), 1.0)
    check(L, make(sizes, dtypes), 1e6)


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("pad", [1, 64])
def test_into_a_flat_fp32_buffer(L, sizes, pad):
    """Every alignment of the outputs against the gradients'."""
    grads = make(sizes, [torch.bfloat16, torch.float16, torch.float32], seed=1)
    at = [0]
    for n in sizes:
        at.append(-(-(at[-1] + n) // pad) * pad)
    flat = torch.full((at[-1] + 64,), 7.0, device="cuda")
    out = [flat[a:a + n] for a, n in zip(at, sizes)]
    check(L, grads, 0.5, out)
    gaps = torch.ones_like(flat, dtype=torch.bool)
    for a, n in zip(at, sizes):
        gaps[a:a + n] = False
    assert bool((flat[gaps] == 7.0).all())


@pytest.mark.parametrize("dtype", DT)
def test_unaligned_views(L, dtype):
    flat = make([60000], [dtype], seed=2)[0]
    cuts = [0, 1, 4, 11, 20000, 20001, 40009, 59999]
    grads = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
    check(L, grads, 1.0)
    others = make([b - a for a, b in zip(cuts, cuts[1:])], [dtype], seed=3)
    check(L, grads, 1.0, out=others)
    check(L, others, 1.0, out=grads)


def test_more_tensors_than_a_launch_holds(L):
    sizes = [1 + 37 * k % 501 for k in range(2500)]
    check(L, make(sizes, DT, seed=4), 1.0)
    assert L.last_launch_count() == 6          # three tables for the norm, three for the scaling


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 64, 2.0 ** -50, 2.0 ** -100, 2.0 ** -120])
def test_squares_beyond_fp32(L, dtype, scale):
    grads = [g * scale for g in make([10000, 3, 999], [dtype], seed=5)]
    want = norm64(grads)
    got = L.rms_norm_grad_norm(grads).item()
    assert abs(got - want) <= 19 * U * want
    # one large element among small ones, and a small tensor beside a large one
    grads[0][17] = 2.0 ** 60
    check(L, grads, 1.0 if scale > 1 else 2.0 ** 50)


def test_subnormal_gradients(L):
    g = torch.full((5000,), 2.0 ** -140, device="cuda")
    got = L.rms_norm_grad_norm([g]).item()
    want = 2.0 ** -140 * math.sqrt(5000)
    assert abs(got - want) <= 2.0 ** -149


def test_zeros(L):
    grads = [torch.zeros(9000, device="cuda"), torch.zeros(3, device="cuda")]
    assert L.rms_norm_grad_clip(grads, 1.0, eps=0.0).item() == 0.0
    assert all(torch.count_nonzero(g).item() == 0 for g in grads)
    empty = [torch.empty(0, device="cuda")]
    assert L.rms_norm_grad_norm(empty).item() == 0.0
    assert L.rms_norm_grad_clip(empty, 1.0).item() == 0.0


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", DT)
def test_not_finite(L, bad, dtype):
    """The norm says so and the gradients stay as they are."""
    grads = make([5000, 33], [dtype], seed=6)
    grads[1][7] = bad
    keep = [g.clone() for g in grads]
    out = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    n = L.rms_norm_grad_clip(grads, 1.0, out=out)
    assert not math.isfinite(n.item())
    assert math.isnan(n.item()) == math.isnan(bad)
    L.rms_norm_grad_clip(grads, 1.0)
    for g, k, o in zip(grads, keep, out):
        assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(k))
        assert torch.equal(torch.nan_to_num(o, 1.0, 2.0, 3.0),
                           torch.nan_to_num(k.float(), 1.0, 2.0, 3.0))


def test_limits_of_max_norm(L):
    g = make([3000], [torch.float32], seed=7)
    check(L, [g[0].clone()], 0.0)
    check(L, [g[0].clone()], float("inf"))
    check(L, [g[0].clone()], norm64(g) * 2)


def test_given_norm(L):
    """Two ranks' lists scaled by the norm over both."""
    a, b = make([4000, 5], [torch.bfloat16], seed=8), make([77], [torch.float32], seed=9)
    total = torch.sqrt(L.rms_norm_grad_norm(a) ** 2 + L.rms_norm_grad_norm(b) ** 2)
    f = factor64(norm64(a + b), 2.0)
    for part in (a, b):
        keep = [g.clone() for g in part]
        n = L.rms_norm_grad_clip(part, 2.0, total_norm=total)
        assert n.item() == total.item() and L.last_launch_count() == 1
        for k, g in zip(keep, part):
            ref = k.double() * f
            most = (torch.finfo(g.dtype).eps / 2 + 26 * U) * ref.abs() + TINY[g.dtype]
            assert bool(((g.double() - ref).abs() <= most).all())


def test_deterministic(L):
    grads = make([300_000, 7, 65_537], DT, seed=10)
    first = L.rms_norm_grad_norm(grads)
    for _ in range(5):
        assert torch.equal(first, L.rms_norm_grad_norm(grads))


def test_list_past_32_bits(L):
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1000:] = 3.0
    g[:1000] = 4.0
    assert L.rms_norm_grad_clip([g], 1.0, eps=0.0).item() == pytest.approx(math.sqrt(25e3), rel=2e-6)
    want = torch.tensor(3.0 / math.sqrt(25e3)).to(torch.bfloat16).item()
    assert bool((g[-1000:] == want).all()) and torch.count_nonzero(g).item() == 2000


def test_another_stream_and_captured(L):
    grads = make([5000, 70001, 3], DT, seed=11)
    out = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    want = L.rms_norm_grad_clip(grads, 1.0, out=out).clone()
    ref = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = L.rms_norm_grad_clip(grads, 1.0, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(out, ref))
    graphs, norms = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            norms.append(L.rms_norm_grad_clip(grads, 1.0, out=out))
    for seed in (12, 13):
        for g, new in zip(grads, make([5000, 70001, 3], DT, seed=seed)):
            g.copy_(new)
        for gr, n in zip(graphs, norms):
            for o in out:
                o.zero_()
            gr.replay()
            got = [o.clone() for o in out]
            want = L.rms_norm_grad_clip(grads, 1.0, out=out)
            assert torch.equal(n, want) and all(torch.equal(a, b) for a, b in zip(got, out))


def test_step_of_block_norms_and_clip(L):
    """A training step: block norms forward and backward, then the norm over
    all gradients and the clip, against the same step in float64."""
    torch.manual_seed(1)
    hidden, layers = 192, 3
    mods = [L.RMSNormBlock(hidden, gate_init=0.3, device="cuda") for _ in range(layers)]
    mats = [(torch.randn(hidden, hidden, device="cuda") / 14).requires_grad_()
            for _ in range(layers)]
    x = torch.randn(10, hidden, device="cuda")
    up = torch.randn(10, hidden, device="cuda")
    r, y = x, x
    for m, w in zip(mods, mats):
        r, y = m(y @ w, r)
    (y * up).sum().backward()
    params = [p for m in mods for p in m.parameters()] + mats
    norm = L.rms_norm_grad_clip([p.grad for p in params], 0.1)
    ref = [p.detach().double().requires_grad_() for p in params]
    by = iter(ref)
    weights = [{n: next(by) for n, _ in m.named_parameters()} for m in mods]
    r = y = x.double()
    rms = lambda v, w: torch.nn.functional.rms_norm(v, (hidden,), w, 1e-6)  # noqa: E731
    for d, w in zip(weights, list(by)):
        r = r + d["gate"] * rms(y @ w, d["post_weight"])
        y = rms(r, d["next_weight"])
    (y * up.double()).sum().backward()
    want = norm64([p.grad for p in ref])
    assert norm.item() == pytest.approx(want, rel=1e-3)
    f = factor64(want, 0.1)
    for p, q in zip(params, ref):
        scale = q.grad.abs().max().item() * f
        assert (p.grad.double() - q.grad * f).abs().max().item() <= 5e-3 * scale
