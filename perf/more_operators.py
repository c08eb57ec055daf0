"""The head norms with rotation and the embedding: cases, plain forms, bytes.

Four operators are measured here.

Head norm and rotation, forward and backward: every head's row v of the
queries and keys is normalised, u = v * rstd(v) * gain(gamma), and the first
``rotary`` of its columns are rotated by the token's position: pair p, of
columns (p, p + rotary / 2) or, interleaved, (2 p, 2 p + 1), by the angle
position * inv_freq[p].  The backward gives the gradients of both inputs and
of both gammas.

Embedding, forward and backward: y[t] = scale * weight[ids[t]], a row of zeros
for an id outside the vocabulary; dweight[v] = scale * the sum of dy[t] over
the tokens t of id v, written over the whole table, or added to it.

``run`` computes a case in elementary torch operations where ``own`` is
false and through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
MAX_HEADS_WORK = 32768 * 72 * 128 * 2  # bytes of q and k in the largest listed forward
MAX_TABLE_WORK = 128000 * 4096         # elements of the largest listed table


def _rotary(name, op, batch, tokens, q_heads, k_heads, dim, rotary, dtype, interleaved=False,
            layout="packed", pos="none", freq="f32", base=10000.0, offset=0, eps=1e-6):
    return {"name": name, "op": op, "batch": batch, "tokens": tokens, "q_heads": q_heads,
            "k_heads": k_heads, "dim": dim, "rotary": rotary, "dtype": dtype,
            "interleaved": interleaved, "layout": layout, "pos": pos, "freq": freq, "base": base,
            "offset": offset, "eps": eps}


def _embed(name, op, tokens, vocab, hidden, dtype, out, scale=1.0, pad=0.0, wide_ids=True,
           accumulate=False):
    return {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "hidden": hidden,
            "dtype": dtype, "out": out, "scale": scale, "pad": pad, "wide_ids": wide_ids,
            "accumulate": accumulate}


def listed():
    return [
        # one decoding step of a batch of eight sequences at positions of their own
        _rotary("rotary fwd 8x(32+8)x128 bf16", "rotary_fwd", 1, 8, 32, 8, 128, 128, "bf16",
                pos="each", base=500000.0),
        # sequences of odd lengths one after another, part of each head rotated, fp16
        _rotary("rotary fwd 777x(5+5)x80 f16", "rotary_fwd", 1, 777, 5, 5, 80, 32, "f16", True,
                "apart", "ragged", offset=1),
        # a large prompt batch, queries and keys inside the packed product
        _rotary("rotary fwd 32768x(64+8)x128 bf16", "rotary_fwd", 4, 8192, 64, 8, 128, 128, "bf16",
                base=500000.0, freq="f64"),
        # a small fp32 model
        _rotary("rotary bwd 256x(8+8)x64 f32", "rotary_bwd", 2, 128, 8, 8, 64, 64, "f32", True,
                "apart"),
        # training, 4 sequences of 1024 tokens
        _rotary("rotary bwd 4096x(32+8)x128 bf16", "rotary_bwd", 4, 1024, 32, 8, 128, 128, "bf16",
                base=500000.0),
        # a large batch of packed sequences, wide heads of which half is rotated
        _rotary("rotary bwd 16384x(32+16)x256 bf16", "rotary_bwd", 1, 16384, 32, 16, 256, 128,
                "bf16", pos="ragged", offset=1),
        # one decoding step of a batch of eight
        _embed("embed fwd 8x4096 bf16", "embed_fwd", 8, 32000, 4096, "bf16", "bf16"),
        # odd widths, padded sequences, an fp32 residual stream
        _embed("embed fwd 1000x1001 f16->f32", "embed_fwd", 1000, 5003, 1001, "f16", "f32", 2.0,
               0.1, False),
        # a large batch, scaled by the root of the width
        _embed("embed fwd 32768x4096 bf16", "embed_fwd", 32768, 128000, 4096, "bf16", "bf16", 64.0),
        # a small table of an odd width
        _embed("embed bwd 300x1001 f16->f32", "embed_bwd", 300, 5003, 1001, "f16", "f32", 1.0, 0.1,
               False),
        # training, 8 sequences of 1024 tokens, the whole gradient in fp32
        _embed("embed bwd 8192x4096 bf16->f32", "embed_bwd", 8192, 32000, 4096, "bf16", "f32",
               64.0),
        # a large batch, added to the gradient of an output layer that shares the table
        _embed("embed bwd 32768x4096 bf16 +f32", "embed_bwd", 32768, 128000, 4096, "bf16", "f32",
               1.0, accumulate=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary_fwd", "rotary_bwd", "embed_fwd", "embed_bwd"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op in ("rotary_fwd", "rotary_bwd"):
        dim = rng.choice((32, 40, 64, 64, 72, 80, 96, 112, 128, 128, 128, 192, 256))
        rotary = rng.choice((dim, dim, dim, dim // 2, dim // 4 // 2 * 2))
        k_heads = rng.choice((1, 2, 4, 5, 8, 8, 16))
        q_heads = k_heads * rng.choice((1, 2, 4, 4, 7, 8))
        heads = q_heads + k_heads
        most = MAX_HEADS_WORK // (heads * dim * BYTES[dtype] * (2 if op == "rotary_bwd" else 1))
        tokens = _log_int(rng, 1, min(most, 65536))
        batch = rng.choice((1, 1, 2, 4)) if tokens >= 4 else 1
        case = _rotary("", op, batch, tokens // batch, q_heads, k_heads, dim, rotary, dtype,
                       rng.random() < 0.4, rng.choice(("packed", "packed", "apart", "heads")),
                       rng.choice(("none", "each", "ragged")), rng.choice(("f32", "f64")),
                       rng.choice((1e4, 5e5, 1e6)), rng.choice((0, 1)), rng.choice((1e-5, 1e-6)))
    else:
        hidden = _log_int(rng, 64, 8192)
        if rng.random() < 0.75:
            hidden = max(64, hidden // 64 * 64)
        vocab = _log_int(rng, 300, min(260000, MAX_TABLE_WORK // hidden))
        tokens = _log_int(rng, 1, min(100000, 32768 * 4096 // hidden))
        out = rng.choice((dtype, "f32")) if dtype != "f32" else rng.choice(("f32", "bf16"))
        case = _embed("", op, tokens, vocab, hidden, dtype, out,
                      rng.choice((1.0, 1.0, round(math.sqrt(hidden), 3))),
                      rng.choice((0.0, 0.0, 0.2)), rng.random() < 0.5,
                      op == "embed_bwd" and out == "f32" and rng.random() < 0.5)
    del case["name"]
    return case


def _randn(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(std).add_(mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("embed_fwd", "embed_bwd"):
        return _prepare_embed(case, gen)
    t, dim, s = DTYPES[case["dtype"]], case["dim"], dict(case)
    s["q"], s["k"] = _heads(case, gen, t, 1.5)
    mean = 0.0 if case["offset"] else 1.0
    s["q_gamma"] = _randn(gen, (dim,), t, 0.1, mean)
    s["k_gamma"] = _randn(gen, (dim,), t, 0.1, mean)
    p = torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64)
    s["inv_freq"] = case["base"] ** (p * (-2.0 / case["rotary"]))
    if case["freq"] == "f32":
        s["inv_freq"] = s["inv_freq"].float()
    s["positions"] = _positions(case, gen)
    if case["op"] == "rotary_bwd":
        # what the forward left for the backward, and the gradients from above
        s["rstd_q"], s["rstd_k"] = _rstd(s["q"], case["eps"]), _rstd(s["k"], case["eps"])
        s["dq_out"], s["dk_out"] = _heads(dict(case, layout="apart"), gen, t, 1.0)
    return s


def _heads(case, gen, t, std):
    """Queries and keys [batch, tokens, heads, dim]: views of the packed product of
    queries, keys and values, tensors of their own, or tensors that hold a
    head's tokens next to one another."""
    b, n, hq, hk, d = (case[x] for x in ("batch", "tokens", "q_heads", "k_heads", "dim"))
    if case["layout"] == "packed":
        packed = _randn(gen, (b, n, hq + 2 * hk, d), t, std)
        return packed[:, :, :hq], packed[:, :, hq:hq + hk]
    if case["layout"] == "heads":
        return (_randn(gen, (b, hq, n, d), t, std).transpose(1, 2),
                _randn(gen, (b, hk, n, d), t, std).transpose(1, 2))
    return _randn(gen, (b, n, hq, d), t, std), _randn(gen, (b, n, hk, d), t, std)


def _positions(case, gen):
    b, n = case["batch"], case["tokens"]
    if case["pos"] == "none":       # 0, 1, ... in every sequence
        return None
    if case["pos"] == "each":       # each token somewhere in a long text
        return torch.randint(0, 1 << 20, (b, n), generator=gen, device="cuda")
    # sequences of odd lengths after one another: positions start again with each
    starts = torch.rand((b, n), generator=gen, device="cuda") < 1.0 / 300.0
    at = torch.arange(n, device="cuda").expand(b, n)
    return at - torch.cummax(torch.where(starts, at, 0), 1).values


def _prepare_embed(case, gen):
    n, v, h = case["tokens"], case["vocab"], case["hidden"]
    s = dict(case)
    # log-uniform ids: the most frequent token is some 6 % of a text
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(v + 1)) - 1).long().clamp_(0, v - 1)
    if case["pad"]:
        ids = torch.where(torch.rand(n, generator=gen, device="cuda") < case["pad"], -1, ids)
    s["ids"] = ids if case["wide_ids"] else ids.int()
    if case["op"] == "embed_fwd":
        s["weight"] = _randn(gen, (v, h), DTYPES[case["dtype"]], 0.02)
    else:
        s["dy"] = _randn(gen, (n, h), DTYPES[case["dtype"]])
        s["dweight"] = _randn(gen, (v, h), DTYPES[case["out"]]) if case["accumulate"] else None
    return s


def _rstd(x, eps):
    x = x.float()
    return torch.rsqrt((x * x).mean(-1) + eps)


def run(state):
    op = state["op"]
    if own:
        return _run_own(state, op)
    if op == "rotary_fwd":
        turn = _turn(state)
        q, rstd_q = _plain_fwd(state, state["q"], state["q_gamma"], turn)
        k, rstd_k = _plain_fwd(state, state["k"], state["k_gamma"], turn)
        return q, k, rstd_q, rstd_k
    if op == "rotary_bwd":
        turn = _turn(state)
        dq, dgq = _plain_bwd(state, "q", turn)
        dk, dgk = _plain_bwd(state, "k", turn)
        return dq, dk, dgq, dgk
    ids = state["ids"].long()
    inside = ((ids >= 0) & (ids < state["vocab"]))[:, None]
    ids = ids.clamp(0, state["vocab"] - 1)
    if op == "embed_fwd":
        y = state["weight"][ids].float() * state["scale"]
        return torch.where(inside, y, 0.0).to(DTYPES[state["out"]])
    terms = torch.where(inside, state["dy"].float() * state["scale"], 0.0)
    if state["accumulate"]:
        return state["dweight"].index_add_(0, ids, terms)
    total = torch.zeros((state["vocab"], state["hidden"]), device="cuda")
    return total.index_add_(0, ids, terms).to(DTYPES[state["out"]])


def _run_own(s, op):
    import bwd_rms_norm_gb300 as rmsn

    if op == "rotary_fwd":
        return rmsn.rms_norm_rotary_fwd(
            s["q"], s["k"], s["q_gamma"], s["k_gamma"], s["inv_freq"], s["positions"],
            eps=s["eps"], offset=s["offset"], interleaved=s["interleaved"])
    if op == "rotary_bwd":
        return rmsn.rms_norm_rotary_bwd(
            s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_gamma"], s["k_gamma"], s["rstd_q"],
            s["rstd_k"], s["inv_freq"], s["positions"], offset=s["offset"],
            interleaved=s["interleaved"])
    if op == "embed_fwd":
        return rmsn.rms_norm_embedding_fwd(s["ids"], s["weight"], scale=s["scale"], dtype=DTYPES[s["out"]])
    if s["accumulate"]:
        return rmsn.rms_norm_embedding_bwd(s["dy"], s["ids"], s["vocab"], scale=s["scale"],
                                  dweight=s["dweight"], accumulate=True)
    return rmsn.rms_norm_embedding_bwd(s["dy"], s["ids"], s["vocab"], scale=s["scale"],
                              dtype=DTYPES[s["out"]])


def _turn(s):
    """Cosines and sines [batch, tokens, 1, rotary / 2] of every token's angles."""
    at = s["positions"]
    if at is None:
        at = torch.arange(s["tokens"], device="cuda").expand(s["batch"], -1)
    angle = at.double()[:, :, None, None] * s["inv_freq"].double()
    return angle.cos().float(), angle.sin().float()


def _rotate(s, u, cos, sin):
    rot = s["rotary"]
    half = rot // 2
    if s["interleaved"]:
        a, b = u[..., 0:rot:2], u[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = u[..., :half], u[..., half:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, u[..., rot:]), -1)


def _plain_fwd(s, x, gamma, turn):
    rstd = _rstd(x, s["eps"])
    u = x.float() * rstd[..., None] * (gamma.float() + float(s["offset"]))
    return _rotate(s, u, *turn).to(x.dtype), rstd


def _plain_bwd(s, name, turn):
    x, gain = s[name].float(), s[name + "_gamma"].float() + float(s["offset"])
    rstd = s["rstd_" + name][..., None]
    du = _rotate(s, s["d" + name + "_out"].float(), turn[0], -turn[1])
    xh = x * rstd
    g = du * gain
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(s[name].dtype), (du * xh).sum((0, 1, 2))


def _distinct(case):
    """Rows of the table that a batch of log-uniform ids is expected to touch."""
    v = case["vocab"]
    edges = torch.log(torch.arange(1, v + 2, dtype=torch.float64)) / math.log(v + 1)
    p = edges[1:] - edges[:-1]
    n = case["tokens"] * (1.0 - case["pad"])
    return float((1.0 - torch.exp(n * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


def work(case):
    if case["op"] in ("embed_fwd", "embed_bwd"):
        n, h, t, o = case["tokens"], case["hidden"], BYTES[case["dtype"]], BYTES[case["out"]]
        ids = n * (8 if case["wide_ids"] else 4)
        if case["op"] == "embed_fwd":
            return {"bytes": ids + _distinct(case) * h * t + n * h * o, "flops": n * h}
        table = 2 * _distinct(case) * h * o if case["accumulate"] else case["vocab"] * h * o
        return {"bytes": ids + n * h * t + table, "flops": 2 * n * h}
    tokens, t = case["batch"] * case["tokens"], BYTES[case["dtype"]]
    rows = tokens * (case["q_heads"] + case["k_heads"])
    n = rows * case["dim"]
    small = (2 * case["dim"] * t + case["rotary"] // 2 * (8 if case["freq"] == "f64" else 4)
             + (0 if case["pos"] == "none" else 8 * tokens))
    if case["op"] == "rotary_fwd":
        return {"bytes": 2 * n * t + 4 * rows + small, "flops": 7 * n}
    return {"bytes": 3 * n * t + 4 * rows + small + 8 * case["dim"], "flops": 14 * n}


def exact(case, seed):
    """What ``run`` returns, in 64 bits from the definitions: the rotation as a
    product of complex numbers, the backward as inner products of each row, the
    table's gradient from sorted tokens."""
    s = prepare(case, seed)
    if case["op"] == "embed_fwd":
        ids = s["ids"].long()
        known = torch.cat((s["weight"].double() * case["scale"],
                           torch.zeros((1, case["hidden"]), dtype=torch.float64, device="cuda")))
        return known[torch.where((ids < 0) | (ids >= case["vocab"]), case["vocab"], ids)]
    if case["op"] == "embed_bwd":
        return _exact_embed_bwd(case, s)
    at = s["positions"]
    if at is None:
        at = torch.arange(case["tokens"], device="cuda").repeat(case["batch"], 1)
    angle = torch.einsum("bt,p->btp", at.double(), s["inv_freq"].double())[:, :, None]
    turn = torch.polar(torch.ones_like(angle), angle)
    got = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_gamma"].double() + case["offset"]
        if case["op"] == "rotary_fwd":
            r = (x.norm(dim=-1).square() / case["dim"] + case["eps"]).pow(-0.5)
            got[name] = _turned(case, x * w * r[..., None], turn), r
        else:
            r = s["rstd_" + name].double()[..., None]
            du = _turned(case, s["d" + name + "_out"].double(), turn.conj())
            xh = x * r
            inner = torch.einsum("bthd,bthd->bth", du * w, xh)[..., None] / case["dim"]
            got[name] = (du * w - xh * inner) * r, torch.einsum("bthd,bthd->d", du, xh)
    return got["q"][0], got["k"][0], got["q"][1], got["k"][1]


def _turned(case, u, turn):
    rot = case["rotary"]
    head = u[..., :rot]
    if not case["interleaved"]:
        head = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    else:
        head = head.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
    if not case["interleaved"]:
        z = z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), u[..., rot:]), -1)


def _exact_embed_bwd(case, s):
    h = case["hidden"]
    ids = s["ids"].long()
    ids, order = torch.sort(torch.where((ids < 0) | (ids >= case["vocab"]), case["vocab"], ids),
                            stable=True)
    rows, counts = torch.unique_consecutive(ids, return_counts=True)
    total = torch.zeros((case["vocab"] + 1, h), dtype=torch.float64, device="cuda")
    sums = torch.segment_reduce(s["dy"].double()[order] * case["scale"], "sum", lengths=counts)
    total[rows] = sums
    total = total[:-1]
    return total if s["dweight"] is None else total + s["dweight"].double()
