"""The operators around a transformer's matrix products together, as a training
step uses them: embedding, norm, head norm with rotation, block norm, backward,
the gradients clipped; against the same step in float64 on the CPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu
VOCAB, HIDDEN, HEADS, KEYS, DIM, TOKENS = 97, 128, 4, 2, 32, 24


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


def params(device, dtype):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ps = {"table": 0.1 * r(VOCAB, HIDDEN), "norm": 1 + 0.1 * r(HIDDEN),
          "qkv": r((HEADS + 2 * KEYS) * DIM, HIDDEN) / HIDDEN ** 0.5,
          "q": 1 + 0.1 * r(DIM), "k": 1 + 0.1 * r(DIM),
          "out": r(HIDDEN, HEADS * DIM) / HIDDEN ** 0.5, "post": 1 + 0.1 * r(HIDDEN),
          "next": 1 + 0.1 * r(HIDDEN)}
    return {k: v.to(device=device, dtype=dtype).requires_grad_() for k, v in ps.items()}


def attention(q, k, v):
    q, k, v = (t.transpose(1, 2) for t in (q, k, v))
    k, v = (t.repeat_interleave(HEADS // KEYS, 1) for t in (k, v))
    s = q @ k.transpose(-1, -2) / DIM ** 0.5
    mask = torch.ones(TOKENS, TOKENS, device=q.device).triu(1).bool()
    return (s.masked_fill(mask, float("-inf")).softmax(-1) @ v).transpose(1, 2).flatten(2)


def norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def rotate(x, freq):
    a = torch.arange(TOKENS, dtype=x.dtype)[:, None, None] * freq
    i, j = x[..., :DIM // 2], x[..., DIM // 2:]
    return torch.cat((i * a.cos() - j * a.sin(), j * a.cos() + i * a.sin()), -1)


def split(t):
    t = t.unflatten(-1, (-1, DIM))
    return t[:, :, :HEADS], t[:, :, HEADS:HEADS + KEYS], t[:, :, HEADS + KEYS:]


def test_training_step(L):
    freq = 10000.0 ** (-torch.arange(DIM // 2, dtype=torch.float64) / (DIM // 2))
    ids = torch.randint(0, VOCAB, (2, TOKENS), generator=torch.Generator().manual_seed(1))
    ids[1, -5:] = -1                                       # a shorter sequence, padded
    p = params("cpu", torch.float64)
    x = torch.where(ids[..., None] >= 0, p["table"][ids.clamp(0)] * HIDDEN ** 0.5, 0.0)
    q, k, v = split(norm(x, p["norm"]) @ p["qkv"].T)
    a = attention(rotate(norm(q, p["q"]), freq), rotate(norm(k, p["k"]), freq), v)
    r = x + norm(a @ p["out"].T, p["post"])
    norm(r, p["next"]).square().mean().backward()
    want = {n: t.grad for n, t in p.items()}
    total = torch.stack([g.norm() for g in want.values()]).norm()

    p = params("cuda", torch.float32)
    ids = ids.cuda()

    def step():
        x = L.rms_norm_embedding(ids, p["table"], HIDDEN ** 0.5)
        q, k, v = split(L.rms_norm(x, p["norm"], 1e-6) @ p["qkv"].T)
        q, k = L.rms_norm_rotary(q, k, p["q"], p["k"], freq.cuda())
        a = attention(q, k, v) @ p["out"].T
        _, y = L.rms_norm_block(a, x, p["post"], None, p["next"])
        y.square().mean().backward()

    step()
    # fp32 throughout (matrix products too): 1e-4 of the largest gradient, some hundred
    # roundings of 2^-24 along the way and sums of up to 48 rows
    for n, t in p.items():
        assert float((t.grad.cpu().double() - want[n]).abs().max()) <= (
            1e-4 * float(want[n].abs().max())), n
    grads = [t.grad for t in p.values()]
    got = L.rms_norm_grad_clip(grads, 0.01)
    assert abs(float(got) / float(total) - 1) < 1e-4
    assert abs(float(torch.stack([g.norm() for g in grads]).norm()) / 0.01 - 1) < 1e-4


def test_single_tokens_follow_a_prompt(L):
    """A prompt at once, and its tokens one by one: the same keys, the same queries."""
    g = torch.Generator().manual_seed(2)
    table = torch.randn(VOCAB, HIDDEN, generator=g).cuda().bfloat16()
    w = [torch.randn(DIM, generator=g).cuda().bfloat16() for _ in range(2)]
    proj = torch.randn((HEADS + 2 * KEYS) * DIM, HIDDEN, generator=g).cuda().bfloat16()
    freq = (10000.0 ** (-torch.arange(DIM // 2) / (DIM // 2))).cuda()
    ids = torch.randint(0, VOCAB, (TOKENS,), generator=g).cuda()
    packed = (L.rms_norm_embedding_fwd(ids, table, 11.3) @ proj.T).unflatten(-1, (-1, DIM))
    whole = packed.clone()
    q, k = whole[:, :HEADS], whole[:, HEADS:HEADS + KEYS]
    L.rms_norm_rotary_fwd(q, k, *w, freq, q_out=q, k_out=k, with_rstd=False)
    assert torch.equal(whole[:, HEADS + KEYS:], packed[:, HEADS + KEYS:])
    for t in range(TOKENS):
        one = packed[t:t + 1].clone()
        at = torch.tensor([t], dtype=torch.int32).cuda()
        q, k = one[:, :HEADS], one[:, HEADS:HEADS + KEYS]
        L.rms_norm_rotary_fwd(q, k, *w, freq, at, q_out=q, k_out=k, with_rstd=False)
        assert torch.equal(one[0], whole[t])
