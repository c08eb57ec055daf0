"""The embedding's gradient of many tokens, over every way that its kernels have.

Terms, tables and scales are whole numbers and powers of two whose sums stay below
2^24: exact in fp32 in any order, so that a result is the exact sum, rounded once
where the table is of 16 bits.  Where terms are not exact, their order is the
documented one and gives the same bits on the host."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


def piece_of(L, tokens, vocab, hidden):
    """The entries of a piece, from the room for two rows of open sums of each."""
    room = L.rms_norm_embedding_bwd_workspace_size(tokens, vocab, hidden)
    pieces = (room - 16 * (tokens + tokens % 2)) // (8 * hidden)
    return next(p for p in (8, 16, 32) if -(-tokens // p) == pieces)


def make_ids(kind, tokens, vocab, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        return torch.full((tokens,), vocab // 2)
    if kind == "each":
        return torch.randperm(vocab, generator=g)[torch.arange(tokens) % vocab]
    if kind == "dense":                   # neighbouring rows by the thousand
        return torch.arange(tokens) % (tokens // 2) + vocab // 3
    if kind == "uniform":
        return torch.randint(0, vocab, (tokens,), generator=g)
    ids = (vocab ** torch.rand(tokens, generator=g, dtype=torch.float64)).long() - 1
    if kind == "frequent":                # half of the tokens have one id
        ids[torch.rand(tokens, generator=g) < 0.5] = 11
    ids[::50] = torch.tensor([-1, vocab])[torch.arange(len(ids[::50])) % 2]
    return ids


def whole(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)


def beside(shape, dtype, value, by):
    """A tensor from the `by`-th element of its buffer on, with guards around it."""
    n = int(np.prod(shape))
    buf = torch.full((n + by + 16,), value, dtype=dtype, device="cuda")
    return buf, buf[by:by + n].view(shape)


def exact(ids, dy, vocab, scale, start=None):
    where = torch.where((ids >= 0) & (ids < vocab), ids, vocab)
    total = torch.zeros((vocab + 1, dy.shape[1]), dtype=torch.float64, device="cuda")
    total.index_add_(0, where, dy.double())
    total = scale * total[:vocab]
    assert float(total.abs().max()) < 1 << 23
    return total if start is None else total + start.double()


# what is cleared beside the sort (40 MB and 1 KB a token) and beside the joins (64 MB)
# leaves rows of these tables to the warps beside the sums, and to those beside the
# joins rows with tokens among them
@pytest.mark.parametrize("tokens,vocab,hidden,dtype,out,by", [
    (40000, 60000, 1024, "bf16", "f32", 0),      # long runs of tokens, few rows
    (2000, 9500000, 4, "f32", "f32", 0),         # thousands of rows a warp, more than once
    (30000, 60000, 1001, "f16", "f32", 1),       # odd rows, beside 16 bytes
    (5000, 3500000, 33, "bf16", "bf16", 3),
    (700, 150000, 520, "f32", "bf16", 0)])
@pytest.mark.parametrize("kind", ["frequent", "uniform", "dense"])
def test_rows_without_a_token_of_large_tables(L, kind, tokens, vocab, hidden, dtype, out, by):
    row = hidden * T[out].itemsize
    assert vocab * row > (40 << 20) + 1024 * tokens + (64 << 20) + 4096 * row
    ids = make_ids(kind, tokens, vocab, 1).cuda()
    if kind == "frequent":
        ids[:2] = torch.tensor([0, vocab - 1])
    dy = whole((tokens, hidden), T[dtype], 2)
    buf, table = beside((vocab, hidden), T[out], NAN, by)
    assert L.rms_norm_embedding_bwd(dy, ids, vocab, 2.0, dweight=table) is table
    ref = exact(ids, dy, vocab, 2.0).to(T[out])
    assert torch.equal(table, ref)
    assert bool(buf[:by].isnan().all()) and bool(buf[by + table.numel():].isnan().all())


@pytest.mark.parametrize("tokens,hidden,piece", [
    (900, 64, 8), (8000, 64, 8), (3000, 1088, 8), (9000, 64, 16), (9000, 71, 16),
    (9000, 1088, 16), (9000, 1027, 16), (20000, 72, 32), (20000, 71, 32), (20000, 300, 32),
    (17000, 1088, 32), (17000, 1027, 32)])
@pytest.mark.parametrize("kind", ["text", "same", "each"])
@pytest.mark.parametrize("types", [("bf16", "f32"), ("f32", "f32"), ("f16", "f16"),
                                   ("f32", "bf16")], ids="-".join)
def test_pieces(L, kind, tokens, hidden, piece, types):
    vocab = tokens if kind == "each" else 400
    assert piece_of(L, tokens, vocab, hidden) == piece
    ids = make_ids(kind, tokens, vocab, 3).cuda()
    dy = whole((tokens, hidden), T[types[0]], 4)
    scale = -2.0 if types[1] != "f16" else 0.125   # within fp16's numbers
    ref = exact(ids, dy, vocab, scale)
    assert torch.equal(L.rms_norm_embedding_bwd(dy, ids, vocab, scale, dtype=T[types[1]]),
                       ref.to(T[types[1]]))
    start = whole((vocab, hidden), T[types[1]], 5)
    ref = exact(ids, dy, vocab, scale, start).to(T[types[1]])
    L.rms_norm_embedding_bwd(dy, ids, vocab, scale, dweight=start, accumulate=True)
    assert torch.equal(start, ref)


# digits of 10 bits, two and three of them, and four of 8
@pytest.mark.parametrize("vocab", [1 << 19, (1 << 20) - 1, 1 << 21, (1 << 27) + 5, 1 << 29,
                                   (1 << 30) - 7, 1 << 30])
def test_ids_of_every_bit(L, vocab):
    if torch.cuda.mem_get_info()[0] < 4 * vocab + (4 << 30):
        pytest.skip("not enough free memory for the table")
    g = torch.Generator().manual_seed(6)
    bits = vocab.bit_length()
    some = torch.cat([torch.tensor([0, vocab - 1, vocab // 2]),
                      2 ** torch.arange(bits - 1), 2 ** torch.arange(1, bits) - 1,
                      torch.randint(0, vocab, (400,), generator=g)])
    ids = torch.cat([some, some.flip(0), torch.tensor([vocab, -1, vocab + 1, 1 << 40])])
    ids = ids[torch.randperm(len(ids), generator=g)].cuda()
    assert len(ids) > 512
    dy = torch.randint(1, 4, (len(ids), 1), generator=g).bfloat16().cuda()
    inside = (ids >= 0) & (ids < vocab)
    rows, at = ids[inside].unique(return_inverse=True)
    ref = torch.zeros(len(rows), dtype=torch.float64, device="cuda").index_add_(
        0, at, dy[inside, 0].double())
    assert float(ref.max()) <= 256                       # exact in bf16
    table = torch.zeros((vocab, 1), dtype=torch.bfloat16, device="cuda")
    L.rms_norm_embedding_bwd(dy, ids, vocab, dweight=table, accumulate=True)
    assert torch.equal(table[rows, 0], ref.bfloat16()) and int(table.count_nonzero()) == len(rows)
    table.fill_(NAN)
    L.rms_norm_embedding_bwd(dy, ids, vocab, dweight=table)
    assert torch.equal(table[rows, 0], ref.bfloat16()) and int(table.count_nonzero()) == len(rows)


@pytest.mark.parametrize("tokens,hidden", [(900, 64), (3000, 71), (9000, 72), (9000, 1088),
                                           (20000, 65), (17000, 1032)])
def test_terms_are_added_in_the_order_of_the_tokens(L, tokens, hidden):
    """Within a piece of sorted entries one after another, then the pieces' sums."""
    g = torch.Generator().manual_seed(7)
    vocab = tokens // 9
    ids = torch.randint(0, vocab, (tokens,), generator=g)
    piece = piece_of(L, tokens, vocab, hidden)
    assert int(ids.bincount().max()) < 31 * piece       # not so many that runs of pieces are
    size = 10.0 ** torch.randint(-3, 8, (tokens, 1), generator=g)
    dy = torch.randn((tokens, hidden), generator=g) * size
    got = L.rms_norm_embedding_bwd(dy.cuda(), ids.cuda(), vocab).cpu().numpy()
    order = ids.argsort(stable=True).numpy()
    terms, key = dy.numpy()[order], ids.numpy()[order]
    want = np.zeros((vocab, hidden), dtype=np.float32)
    part, open_id = np.zeros(hidden, dtype=np.float32), -1
    for i in range(tokens):
        part = part + terms[i]
        if i + 1 == tokens or key[i + 1] != key[i] or (i + 1) % piece == 0:
            want[key[i]] = want[key[i]] + part if open_id == key[i] else part
            part, open_id = np.zeros(hidden, dtype=np.float32), key[i]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("hidden", [64, 71, 1088])
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16"),
                                   ("f32", "f16")], ids="-".join)
@pytest.mark.parametrize("by", [(0, 1), (1, 0), (3, 5)])
def test_any_alignment_of_many_tokens(L, hidden, types, by):
    tokens, vocab = 700, 120
    ids = make_ids("text", tokens, vocab, 8).cuda()
    _, dy = beside((tokens, hidden), T[types[0]], NAN, by[0])
    dy.copy_(whole((tokens, hidden), T[types[0]], 9))
    buf, table = beside((vocab, hidden), T[types[1]], 7.0, by[1])
    ref = exact(ids, dy, vocab, 0.5)
    L.rms_norm_embedding_bwd(dy, ids, vocab, 0.5, dweight=table)
    assert torch.equal(table, ref.to(T[types[1]]))
    L.rms_norm_embedding_bwd(dy, ids, vocab, -0.5, dweight=table, accumulate=True)
    assert not table.any()
    assert bool((buf[:by[1]] == 7).all()) and bool((buf[by[1] + table.numel():] == 7).all())
