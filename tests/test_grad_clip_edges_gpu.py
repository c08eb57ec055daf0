"""The gradient norm and clip where values leave the usual range or repeat.
Tolerances are those of test_grad_clip_gpu.py: h + 22 u and the smallest
subnormal of the output's type."""
import pytest
import torch

from test_grad_clip_gpu import TINY, U, check, factor64, make, norm64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


def near(got, kept, f):
    for o, k in zip(got, kept):
        ref = k.double() * f
        most = (torch.finfo(o.dtype).eps / 2 + 22 * U) * ref.abs() + TINY[o.dtype]
        bad = ~((o.double() - ref).abs() <= most)
        assert not bool(bad.any()), (k.dtype, o.dtype, o[bad][0].item(), ref[bad][0].item())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("large,max_norm", [(30, 2.0 ** -110), (100, 2.0 ** -40), (100, 2.0 ** -72),
                                            (110, 0.01), (20, 2.0 ** -110), (100, 2.0 ** -130)])
def test_factors_below_the_normal_numbers(L, dtype, large, max_norm):
    """The factor is a subnormal fp32 value, or none; the results are not."""
    std = 2.0 ** large
    check(L, make([5000, 3, 999], [dtype], seed=1, std=std), max_norm)
    out = [torch.empty(n, device="cuda") for n in (5000, 3, 999)]
    check(L, make([5000, 3, 999], [dtype], seed=2, std=std), max_norm, out=out)
    grads = make([5000, 3, 999], [dtype], seed=3, std=std)
    total = L.rms_norm_grad_norm(grads)
    keep = [g.clone() for g in grads]
    L.rms_norm_grad_clip(grads, max_norm, total_norm=total)
    near(grads, keep, factor64(total.item(), max_norm))


@pytest.mark.parametrize("value,dtype,n", [
    (3e38, torch.float32, 16), (3e38, torch.bfloat16, 16), (1e38, torch.float32, 1_000_003),
    (-3.3e38, torch.bfloat16, 70_001), (2e38, torch.float32, 3)])
@pytest.mark.parametrize("max_norm", [1.0, 1e30, 3e38, 2.0 ** -20, 0.0, float("inf")])
def test_finite_lists_whose_norm_is_beyond_fp32(L, value, dtype, n, max_norm):
    """The norm is infinite in fp32, but the list is clipped by its own."""
    grads = [torch.full((n,), value, device="cuda").to(dtype),
             torch.tensor([1.0, -2.0 ** 100, 0.0], device="cuda").to(dtype)]
    keep = [g.clone() for g in grads]
    f = factor64(norm64(keep), max_norm)
    out = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    assert L.rms_norm_grad_norm(grads).item() == float("inf")
    assert L.rms_norm_grad_clip(grads, max_norm, out=out).item() == float("inf")
    near(out, keep, f)
    assert L.rms_norm_grad_clip(grads, max_norm).item() == float("inf")
    near(grads, keep, f)


@pytest.mark.parametrize("eps", [1e38, 3.4e38])
def test_norm_and_eps_together_beyond_fp32(L, eps):
    grads = [torch.full((4,), 1.5e38, device="cuda")]
    keep = [g.clone() for g in grads]
    assert L.rms_norm_grad_clip(grads, 2.0, eps=eps).item() == pytest.approx(3e38, rel=1e-6)
    near(grads, keep, factor64(norm64(keep), 2.0, eps))
    total = torch.tensor(3e38, device="cuda")
    grads = [g.clone() for g in keep]
    L.rms_norm_grad_clip(grads, 2.0, eps=eps, total_norm=total)
    near(grads, keep, factor64(total.double().item(), 2.0, eps))


def best_us(f, n=20):
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times)[n // 4]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_zeros_are_read_once(L, dtype, zero):
    """Zeros among other gradients (an embedding's unused rows, a frozen branch)
    take the time of any others; read twice they take 1.45 times that."""
    first = torch.full((1 << 25,), 0.01, dtype=dtype, device="cuda")
    lists = [[first, torch.full((1 << 27,), v, dtype=dtype, device="cuda")] for v in (0.01, zero)]
    want = norm64(lists[1])
    assert abs(L.rms_norm_grad_norm(lists[1]).item() - want) <= 19 * U * want
    for _ in range(3):
        L.rms_norm_grad_norm(lists[0])
    a, b = (best_us(lambda g=g: L.rms_norm_grad_norm(g)) for g in lists)
    assert b <= 1.2 * a, (a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_smallest_values_among_zeros(L, dtype):
    """Squares that vanish in fp32, one a share of a thread at most, and signs."""
    tiny = 2.0 ** -149 if dtype is torch.float32 else 2.0 ** -133
    for at in (0, 1, 7, 8, 4099, 16383, 16384, 29_999):
        for value in (tiny, -tiny, 2.0 ** -80):
            g = torch.full((30_000,), -0.0, dtype=dtype, device="cuda")
            g[at] = value
            assert L.rms_norm_grad_norm([g]).item() == abs(value)
            assert L.rms_norm_grad_norm([g[1:], g[:1]]).item() == abs(value)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("large", [2.0 ** -5, 2.0 ** -9, 2.0 ** -12, 2.0 ** -20, 2.0 ** -40])
@pytest.mark.parametrize("small", [2.0 ** -46, 2.0 ** -60, 2.0 ** -90])
def test_small_shares_beside_larger_ones(L, dtype, large, small):
    """Around the sums from which a small share is taken as it is."""
    g = torch.full((30_000_000,), small, dtype=dtype, device="cuda")
    g[:20_000_000:64] = large
    want = norm64([g])
    assert abs(L.rms_norm_grad_norm([g]).item() - want) <= 19 * U * want
