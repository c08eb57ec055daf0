"""The embedding on the GPU against the float64 oracle.

Tolerances, from u = 2^-24 and h = finfo(T).eps / 2: the forward is one product
in fp32 and one rounding, of a scale that is itself rounded: (h + 2 u) |y|.  A
row of the gradient is a sum of n terms in fp32, its scaling, the addition to
what was there and a rounding: h |dw| + (n + 4) u sum |terms|, the row that was
there among them; plus the smallest subnormal of T, where a value underflows."""
import numpy as np
import pytest
import torch

from oracle import embedding as oem

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
U = 2.0 ** -24
PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32"),
         ("f32", "bf16"), ("f32", "f16")]


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


def make_ids(kind, tokens, vocab, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        return torch.full((tokens,), vocab // 2)
    if kind == "each":                    # every id once, as far as they go
        return torch.randperm(max(tokens, vocab), generator=g)[:tokens] % vocab
    ids = (vocab ** torch.rand(tokens, generator=g, dtype=torch.float64)).long() - 1
    ids = ids.clamp(0, vocab - 1)
    if kind == "padded":
        out = torch.tensor([-1, vocab, vocab + 5, -(1 << 30), -100])
        ids = torch.where(torch.rand(tokens, generator=g) < 0.3,
                          out[torch.randint(0, 5, (tokens,), generator=g)], ids)
    if kind == "none":
        ids = torch.full((tokens,), -1)
    return ids


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(T[dtype]).cuda()


def check_fwd(L, ids, weight, out, scale=1.0):
    y = L.rms_norm_embedding_fwd(ids, weight, scale, T[out])
    ref = oem.forward(f64(ids.flatten()).astype(np.int64), f64(weight), scale)
    assert y.shape == (*ids.shape, weight.shape[1]) and y.dtype == T[out]
    near(y.flatten(0, -2) if y.dim() > 1 else y, ref, 2 * U * np.abs(ref), "y")


def check_bwd(L, ids, dy, vocab, out, scale=1.0, pad=None, start=None):
    ref, size, count = oem.backward(f64(dy).reshape(-1, dy.shape[-1]),
                                    ids.flatten().cpu().numpy(), vocab, scale, pad,
                                    None if start is None else f64(start))
    if start is None:
        got = L.rms_norm_embedding_bwd(dy, ids, vocab, scale, pad, T[out])
    else:
        got = L.rms_norm_embedding_bwd(dy, ids, vocab, scale, pad, dweight=start, accumulate=True)
        assert got is start
    near(got, ref, (count[:, None] + 4) * U * size, "dweight")
    return got


@pytest.mark.parametrize("kind", ["text", "padded", "same", "each", "none"])
@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 1, 1), (1, 10, 64), (31, 7, 33), (32, 40, 8),
                                                 (33, 40, 256), (8, 50, 4096), (100, 300, 1001),
                                                 (1000, 700, 40), (4097, 1000, 24)])
def test_kinds(L, kind, tokens, vocab, hidden):
    ids = make_ids(kind, tokens, vocab).cuda()
    for few in (ids, ids.clamp(-(1 << 31), (1 << 31) - 1).int()):
        check_fwd(L, few, randn((vocab, hidden), "bf16", 1), "bf16", 3.7)
        check_bwd(L, few, randn((tokens, hidden), "bf16", 2), vocab, "f32", 3.7)


@pytest.mark.parametrize("types", PAIRS, ids="-".join)
@pytest.mark.parametrize("hidden", [1, 12, 64, 264, 1001, 2048])
def test_types(L, types, hidden):
    ids = make_ids("padded", 150, 60).cuda()
    check_fwd(L, ids, randn((60, hidden), types[0], 1), types[1], 0.3)
    check_bwd(L, ids, randn((150, hidden), types[0], 2), 60, types[1], 0.3, pad=0)
    check_bwd(L, ids, randn((150, hidden), types[0], 2), 60, types[1], -2.0,
              start=randn((60, hidden), types[1], 3))


@pytest.mark.parametrize("vocab", [2, 255, 256, 511, 512, 513, 40000, 262144, 300000, 1 << 20])
def test_tables(L, vocab):
    # one to three digits of an id, and ids at the ends of the table
    ids = make_ids("each", 2000, vocab, 5)
    ids[:3] = torch.tensor([0, vocab - 1, vocab - 1])
    check_bwd(L, ids.cuda(), randn((2000, 4), "f32", 2), vocab, "f32")


def test_largest_ids(L):
    # five digits; the table's own bytes are never touched but at the rows
    vocab = (1 << 30) - 7
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * vocab * 2:
        pytest.skip("not enough free memory for the largest table")
    table = torch.zeros((vocab, 1), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, 1 << 29, vocab, vocab - 1, (1 << 29) - 1, 5, -1]).cuda()
    dy = torch.arange(1, 9, dtype=torch.float32, device="cuda").bfloat16().view(8, 1)
    L.rms_norm_embedding_bwd(dy, ids, vocab, dweight=table, accumulate=True)
    at = torch.tensor([0, 5, (1 << 29) - 1, 1 << 29, vocab - 1]).cuda()
    assert table[at, 0].tolist() == [2.0, 7.0, 6.0, 3.0, 6.0]
    assert int(table.count_nonzero()) == 5
    y = L.rms_norm_embedding_fwd(ids, table)
    assert y[:, 0].tolist() == [6.0, 2.0, 3.0, 0.0, 6.0, 6.0, 7.0, 0.0]


@pytest.mark.parametrize("tokens", [300, 700])
def test_tables_beyond_32_bits(L, tokens):
    vocab, hidden = (1 << 19) + 3, 8200
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough free memory")
    # the table's first row, its last, and rows on both sides of 2^31 and 2^32 elements
    near_ = [0, (1 << 31) // hidden, (1 << 31) // hidden + 1, (1 << 32) // hidden,
             (1 << 32) // hidden + 1, vocab - 1]
    ids = torch.tensor(near_).repeat(tokens // 6 + 1)[:tokens].cuda()
    dy = torch.randint(-3, 4, (tokens, hidden), generator=torch.Generator().manual_seed(3)).cuda()
    ref = torch.stack([dy[ids == v].sum(0) for v in near_])    # whole numbers: exact
    assert int(ref.abs().max()) <= 256                         # in bf16 too
    dy = dy.bfloat16()
    table = torch.ones((vocab, hidden), dtype=torch.bfloat16, device="cuda")
    L.rms_norm_embedding_bwd(dy, ids, vocab, dweight=table)
    assert torch.equal(table[near_], ref.bfloat16())
    assert sum(int(part.count_nonzero()) for part in table.split(1 << 16)) == int(
        ref.count_nonzero())
    assert torch.equal(L.rms_norm_embedding_fwd(ids, table), table[ids])
    L.rms_norm_embedding_bwd(dy, ids, vocab, scale=-1.0, dweight=table, accumulate=True)
    assert not any(bool(part.any()) for part in table.split(1 << 16))


def test_tokens_beyond_32_bits(L):
    tokens, vocab, hidden = (1 << 19) + 5, 50, 8200
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough free memory")
    ids = make_ids("padded", tokens, vocab, 7).cuda()
    weight = randn((vocab, hidden), "bf16", 8)
    y = L.rms_norm_embedding_fwd(ids, weight)
    zero = torch.cat((weight, torch.zeros_like(weight[:1])))
    where = torch.where((ids >= 0) & (ids < vocab), ids, vocab)
    for a in range(0, tokens, 1 << 16):
        assert torch.equal(y[a:a + (1 << 16)], zero[where[a:a + (1 << 16)]])
    dy = y.fill_(0.0)                     # whole numbers below 2^24 in sum: exact
    dy[:] = (torch.arange(tokens, device="cuda") % 8)[:, None]
    got = L.rms_norm_embedding_bwd(dy, ids, vocab)
    ref = torch.zeros(vocab + 1, dtype=torch.float64, device="cuda").index_add_(
        0, where, (torch.arange(tokens, device="cuda") % 8).double())
    assert torch.equal(got, ref[:vocab, None].float().expand(vocab, hidden))


@pytest.mark.parametrize("types", PAIRS, ids="-".join)
@pytest.mark.parametrize("hidden", [1, 64, 257, 1000, 1088])
def test_types_of_many_tokens(L, types, hidden):
    """The sorted tokens' way: ids of one piece, of two, and of dozens."""
    ids = make_ids("padded", 900, 200).cuda()
    check_bwd(L, ids, randn((900, hidden), types[0], 2), 200, types[1], 0.3, pad=0)
    check_bwd(L, ids, randn((900, hidden), types[0], 2), 200, types[1], -2.0,
              start=randn((200, hidden), types[1], 3))


@pytest.mark.parametrize("kind", ["text", "same", "each", "padded"])
def test_many_tokens(L, kind):
    # several entries a lane of the sort; ids that go on over thousands of pieces
    tokens, vocab = 300001, 50000
    ids = make_ids(kind, tokens, vocab)
    dy = torch.randint(-8, 9, (tokens, 8), generator=torch.Generator().manual_seed(1))
    # sums of whole numbers below 2^24 are exact in any order
    want = torch.zeros((vocab + 1, 8), dtype=torch.int64)
    inside = (ids >= 0) & (ids < vocab)
    want.index_add_(0, torch.where(inside, ids, vocab), dy)
    got = L.rms_norm_embedding_bwd(dy.float().cuda(), ids.cuda(), vocab)
    assert torch.equal(got.cpu().long(), want[:-1])


def test_order_of_the_tokens(L):
    """The terms of a piece of sorted entries are added in the order of the tokens."""
    dy = torch.tensor([1e8, 1.0, -1e8, 1.0], device="cuda").view(4, 1).repeat(1, 64)
    ids = torch.tensor([3, 3, 3, 3]).cuda()
    assert L.rms_norm_embedding_bwd(dy, ids, 5)[3].tolist() == [1.0] * 64


@pytest.mark.parametrize("tokens,hidden", [(100, 72), (3000, 72), (3000, 71)])
def test_rows_that_are_not_touched(L, tokens, hidden):
    """Values behind the rows of the tokens stay what they are, not a number among them."""
    ids = make_ids("padded", tokens, 500).cuda()
    start = torch.full((500, hidden), float("nan"), device="cuda")
    inside = ids[(ids >= 0) & (ids < 500)]
    start[inside] = 1.0
    dy = randn((tokens, hidden), "bf16", 1)
    dy[(ids < 0) | (ids >= 500)] = float("inf")
    got = L.rms_norm_embedding_bwd(dy, ids, 500, dweight=start, accumulate=True)
    touched = torch.zeros(500, dtype=torch.bool, device="cuda")
    touched[inside] = True
    assert bool(got[~touched].isnan().all()) and bool(got[touched].isfinite().all())
    whole = L.rms_norm_embedding_bwd(dy, ids, 500)
    assert not whole[~touched].any() and bool(whole.isfinite().all())


def test_shapes_and_alignment(L):
    ids = make_ids("text", 60, 30).view(3, 4, 5).cuda()
    check_fwd(L, ids, randn((30, 64), "f16", 1), "f16")
    check_bwd(L, ids, randn((3, 4, 5, 64), "f16", 2), 30, "f16")
    y = L.rms_norm_embedding_fwd(ids[0, 0, 0], randn((30, 64), "f16", 1))
    assert y.shape == (64,)
    # rows of whole vectors that start beside 16 bytes
    odd = randn((30 * 64 + 1,), "bf16", 3)[1:].view(30, 64)
    check_fwd(L, ids, odd, "f32")
    dy = randn((60 * 64 + 1,), "bf16", 4)[1:].view(3, 4, 5, 64)
    start = torch.zeros(30 * 64 + 1, device="cuda")[1:].view(30, 64)
    check_bwd(L, ids, dy, 30, "f32", start=start)
    out = torch.full((30 * 64 + 2,), 7.0, device="cuda")
    L.rms_norm_embedding_bwd(dy, ids, 30, dweight=out[1:-1].view(30, 64))
    assert float(out[0]) == float(out[-1]) == 7.0 and torch.equal(out[1:-1].view(30, 64), start)


def test_given_outputs_and_refusals(L):
    ids = make_ids("text", 40, 30).cuda()
    w, dy = randn((30, 64), "bf16", 1), randn((40, 64), "bf16", 2)
    y = torch.empty((40, 64), dtype=torch.bfloat16, device="cuda")
    version = y._version
    assert L.rms_norm_embedding_fwd(ids, w, y=y) is y and y._version > version
    many, up = make_ids("text", 800, 30).cuda(), randn((800, 64), "bf16", 2)
    ws = torch.empty(L.rms_norm_embedding_bwd_workspace_size(800, 30, 64), dtype=torch.uint8,
                     device="cuda")
    assert torch.equal(L.rms_norm_embedding_bwd(up, many, 30, workspace=ws),
                       L.rms_norm_embedding_bwd(up, many, 30))
    with pytest.raises(L.RMSNormError):
        L.rms_norm_embedding_bwd(up, many, 30, workspace=ws[:-16])
    with pytest.raises(L.RMSNormError):
        L.rms_norm_embedding_bwd(dy, ids, 30, dweight=dy[:30])
    with pytest.raises(L.RMSNormError):
        L.rms_norm_embedding_fwd(ids[:30], w, y=w)
    with pytest.raises(RuntimeError, match="contiguous"):
        L.rms_norm_embedding_fwd(ids, w[:, ::2])
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        L.rms_norm_embedding_fwd(ids, w.cpu())


def test_no_tokens(L):
    none = torch.zeros((2, 0), dtype=torch.int64, device="cuda")
    assert L.rms_norm_embedding_fwd(none, randn((5, 8), "bf16", 1)).shape == (2, 0, 8)
    dy = torch.zeros((2, 0, 8), device="cuda")
    assert not L.rms_norm_embedding_bwd(dy, none, 5).any()
    start = torch.ones((5, 8), device="cuda")
    assert bool((L.rms_norm_embedding_bwd(dy, none, 5, dweight=start, accumulate=True) == 1).all())


def test_same_bits_every_time_and_under_a_budget(L):
    ids = make_ids("text", 20000, 3000).cuda()
    dy = randn((20000, 256), "bf16", 1)
    first = L.rms_norm_embedding_bwd(dy, ids, 3000)
    for _ in range(4):
        assert torch.equal(L.rms_norm_embedding_bwd(dy, ids, 3000), first)
    try:
        for sms in (1, 5, 40):
            L.rms_norm_set_sm_budget(sms)
            assert torch.equal(L.rms_norm_embedding_bwd(dy, ids, 3000), first)
            check_fwd(L, ids[:100], randn((3000, 256), "bf16", 2), "bf16")
    finally:
        L.rms_norm_set_sm_budget(0)


def test_streams_and_graphs(L):
    ids = make_ids("text", 3000, 500).cuda()
    w, dy = randn((500, 128), "bf16", 1), randn((3000, 128), "bf16", 2)
    want = L.rms_norm_embedding_fwd(ids, w), L.rms_norm_embedding_bwd(dy, ids, 500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (L.rms_norm_embedding_fwd(ids, w, stream=side),
           L.rms_norm_embedding_bwd(dy, ids, 500, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two graphs, one after the other, replayed in turn with other ids
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = L.rms_norm_embedding_fwd(ids, w), L.rms_norm_embedding_bwd(dy, ids, 500)
        graphs.append((graph, got))
    ids.copy_(make_ids("padded", 3000, 500, 9))
    want = L.rms_norm_embedding_fwd(ids, w), L.rms_norm_embedding_bwd(dy, ids, 500)
    for graph, got in graphs + graphs:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once(L):
    sets = [(make_ids("text", n, 4000, n).cuda(), randn((n, 264), "bf16", n)) for n in (5000, 300)]
    want = [L.rms_norm_embedding_bwd(dy, ids, 4000) for ids, dy in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [None, None]
    for _ in range(10):
        for i, (s, (ids, dy)) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i] = L.rms_norm_embedding_bwd(dy, ids, 4000)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_and_module(L):
    m = L.RMSNormEmbedding(50, 64, scale=8.0, padding_idx=4, out_dtype=torch.float32,
                           device="cuda", dtype=torch.bfloat16)
    ids = make_ids("text", 60, 50).view(6, 10).cuda()
    ids[0, :4] = torch.tensor([4, -1, 50, 4])
    dy = randn((6, 10, 64), "f32", 1)
    y = m(ids)
    assert y.dtype == torch.float32 and not y[0, 1:3].any()
    y.backward(dy)
    ref, size, count = oem.backward(f64(dy).reshape(-1, 64), ids.flatten().cpu().numpy(), 50, 8.0,
                                    4)
    near(m.weight.grad, ref, (count[:, None] + 4) * U * size, "grad")
    assert not m.weight.grad[4].any()
    # the gradient is linear in y's: exactly what a difference gives
    w = m.weight.detach().float()
    at = [L.rms_norm_embedding(ids, w + s * 0.5 * ref_like(w), 8.0).double() for s in (1, -1)]
    slope = float(((at[0] - at[1]) * dy.double()).sum())
    full = oem.backward(f64(dy).reshape(-1, 64), ids.flatten().cpu().numpy(), 50, 8.0)[0]
    assert abs(slope - float((f64(ref_like(w)) * full).sum())) < 1e-3


def ref_like(w):
    return torch.randn(w.shape, generator=torch.Generator().manual_seed(7)).to(w)
