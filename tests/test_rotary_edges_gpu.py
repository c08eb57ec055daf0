"""Calls of the head norm with rotation at its edges: frequencies of the user's own,
values that are not finite, what becomes of results by themselves, SM budgets.

Tolerances as in test_rotary_gpu.py: y within h |y| + 2e-6 (|u_i| + |u_j|), dgamma
within ((n + 64) u + 2e-6) sum |vh| (|dy_i| + |dy_j|) over its n rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
U = 2.0 ** -24


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


def test_assigned_frequencies_move_to_the_gpu(L):
    m = L.RMSNormRotary(64, base=500000.0, rotary_dim=32)
    want = m.inv_freq / 8
    m.inv_freq = want.clone()
    m = m.cuda().bfloat16()
    assert m.inv_freq.dtype == torch.float64 and m.inv_freq.is_cuda
    assert torch.equal(m.inv_freq.cpu(), want)
    x = torch.randn((2, 9, 6, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, k = x[:, :, :4], x[:, :, 4:]
    got = m(q, k)
    ref = L.rms_norm_rotary_fwd(q, k, m.q_weight, m.k_weight, want.cuda())
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def partner(dim, rot, interleaved):
    """The other column of each column's pair, -1 where it does not rotate."""
    j = torch.arange(dim, device="cuda")
    other = j ^ 1 if interleaved else torch.where(j < rot // 2, j + rot // 2, j - rot // 2)
    return torch.where(j < rot, other, -1)


def turned(t, at, freq, other, interleaved, sign):
    """Rows t [tokens, heads, dim] with the first columns turned, element for element."""
    rot = int((other >= 0).sum())
    j = torch.arange(rot, device="cuda")
    pair = j // 2 if interleaved else j % (rot // 2)
    first = j % 2 == 0 if interleaved else j < rot // 2
    angle = (at[:, None].double() * freq)[:, pair]
    c, s = angle.cos()[:, None], angle.sin()[:, None] * sign
    u, w = t[..., :rot], t[..., other[:rot]]
    return torch.cat((torch.where(first, u * c - w * s, u * c + w * s), t[..., rot:]), -1)


def same_kind(got, ref, most, what):
    """Equal where ref is not finite, within `most` of it elsewhere."""
    got = got.double()
    fine = torch.where(ref.isfinite(), (got - ref).abs() <= most,
                       (got == ref) | (got.isnan() & ref.isnan()))
    assert bool(fine.all()), (what, (~fine).nonzero()[0].tolist(), got[~fine][0], ref[~fine][0])


# whole vectors of halves, neighbours (a part of a vector), halves of no whole vectors,
# rows of no whole vectors
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 32, False), (64, 32, True), (64, 18, True),
                                                 (64, 64, True), (72, 36, False), (256, 128, False),
                                                 (33, 20, False), (33, 20, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_columns_that_do_not_rotate_keep_what_is_not_finite(L, dim, rot, interleaved, dtype):
    g = torch.Generator().manual_seed(3)
    make = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    n, heads, h = 2 * (dim - rot) + 2, 3, torch.finfo(dtype).eps / 2
    q, dy, clean = make(n, heads, dim), make(n, heads, dim), make(dim) * 0.3 + 1
    at, other = torch.arange(n, device="cuda"), partner(dim, rot, interleaved)
    freq = 10000.0 ** (torch.arange(rot // 2, device="cuda", dtype=torch.float64) * (-2.0 / rot))
    # of every column that does not rotate an infinity and a NaN, in rows of their own
    bad_q, bad_dy = q.clone(), dy.clone()
    for i, j in enumerate(range(rot, dim)):
        bad_q[2 * i, i % heads, j], bad_q[2 * i + 1, i % heads, j] = -INF, NAN
        bad_dy[2 * i, i % heads, j] = INF
    gammas = [clean]
    for j in sorted({rot, rot + 1, (rot + dim) // 2, dim - 1} & set(range(rot, dim))):
        for value in (INF, NAN):
            gammas.append(clean.clone())
            gammas[-1][j] = value

    def check(v, up, gamma):
        y, _, rstd, _ = L.rms_norm_rotary_fwd(v, None, gamma, None, freq, eps=1e-6,
                                              interleaved=interleaved)
        x, w, d = v.double(), gamma.double(), up.double()
        r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        same_kind(rstd, r[..., 0], 1e-6 * r[..., 0], "rstd")
        u = x * r * w
        ref = turned(u, at, freq, other, interleaved, 1)
        pair = lambda t: t.abs() + torch.where(other >= 0, t[..., other].abs(), 0.0)  # noqa: E731
        same_kind(y, ref, h * ref.abs() + 2e-6 * pair(u) + 2.0 ** -24, "y")
        back = L.rms_norm_rotary_bwd(up, None, v, None, gamma, None, rstd, None, freq,
                                     interleaved=interleaved)
        r = rstd.double()[..., None]
        du, vh = turned(d, at, freq, other, interleaved, -1), x * r
        ref = (du * vh).sum((0, 1))
        same_kind(back[2], ref, ((n * heads + 64) * U + 2e-6) * (vh.abs() * pair(d)).sum((0, 1)),
                  "dgamma")
        fine = (r * (du * w - vh * (du * w * vh).mean(-1, keepdim=True))).isfinite()
        assert torch.equal(back[0].isfinite(), fine)

    for gamma in gammas:
        check(q, dy, gamma)
    check(bad_q, dy, clean)
    check(q, bad_dy, clean)
    check(bad_q, bad_dy, clean)


@pytest.mark.parametrize("tokens", [9, 700])
def test_each_result_has_memory_of_its_own(L, tokens):
    g = torch.Generator().manual_seed(5)
    make = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    q, k, w, v = make(tokens, 4, 64), make(tokens, 2, 64), make(64), make(64)
    freq = torch.ones(32, device="cuda")
    out = L.rms_norm_rotary_fwd(q, k, w, v, freq)
    back = L.rms_norm_rotary_bwd(out[0], out[1], q, k, w, v, out[2], out[3], freq)
    want = [t.clone() for t in (*out, *back)]
    assert len({t.untyped_storage().data_ptr() for t in (*out, *back)}) == 8
    # what a user does with one leaves the others what they are: it grows, or gives its memory back
    out[2].resize_(2 * tokens * 4).fill_(7.0)
    back[2].resize_(128).fill_(7.0)
    assert torch.equal(out[3], want[3]) and torch.equal(back[3], want[7])
    leaves = [t.clone().requires_grad_() for t in (q, k, w, v)]
    torch.autograd.backward(L.rms_norm_rotary(*leaves, freq), out[:2])
    assert torch.equal(leaves[2].grad, want[6]) and torch.equal(leaves[3].grad, want[7])
    leaves[2].grad.untyped_storage().resize_(0)
    assert torch.equal(leaves[3].grad, want[7])


@pytest.mark.parametrize("tokens,dim", [(60, 128), (500, 128), (500, 33)])
def test_same_bits_under_the_same_budget(L, tokens, dim):
    g = torch.Generator().manual_seed(6)
    make = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, dq, dk = (make(tokens, n, dim) for n in (8, 2, 8, 2))
    w, v, freq = make(dim), make(dim), torch.ones(dim // 2, device="cuda")
    rstd = L.rms_norm_rotary_fwd(q, k, w, v, freq)[2:]
    back = lambda: L.rms_norm_rotary_bwd(dq, dk, q, k, w, v, *rstd, freq)  # noqa: E731
    # two sums of the same terms in fp32, each within (n + 64) u of the terms' sizes
    other, off = partner(dim, dim // 2 * 2, False), []
    for x, up, r in ((q, dq, rstd[0]), (k, dk, rstd[1])):
        d = up.double().abs()
        size = (x.double() * r.double()[..., None]).abs() * (
            d + torch.where(other >= 0, d[..., other], 0.0))
        off.append(2 * (r.numel() + 64) * U * size.sum((0, 1)))
    whole = back()
    bits = set()
    try:
        for sms in (1, 7, 40, 0):
            L.rms_norm_set_sm_budget(sms)
            assert sms == 0 or L.rms_norm_sm_budget() == sms
            first = back()
            for _ in range(3):
                assert all(torch.equal(a, b) for a, b in zip(first, back()))
            # the rows' gradients know nothing of the budget; the sums' order does
            assert torch.equal(first[0], whole[0]) and torch.equal(first[1], whole[1])
            for a, b, most in zip(first[2:], whole[2:], off):
                assert bool(((a - b).double().abs() <= most).all())
            bits.add(first[2].cpu().numpy().tobytes())
    finally:
        L.rms_norm_set_sm_budget(0)
    assert torch.equal(back()[2], whole[2]) and len(bits) > 1
