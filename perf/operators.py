"""The residual-stream operators and the gradient clip: cases, plain forms, bytes.

Two operators are measured here.

Block norm, forward and backward: the norms after and before a transformer
block, fused with the block's gate and the scaled residual sum,

    z = x * rstd(x) * gain(post)                (z = x without a post norm)
    r = residual_scale * residual + branch_scale * gate * z
    y = r * rstd(r) * gain(next)                (no y without a next norm)

with rstd(v) = 1 / sqrt(mean(v^2) + eps) over the last dimension and
gain(w) = w, or 1 + w with offset 1.  The gate has one row for every
rows / gate_rows consecutive rows.

Gradient norm and clip: the 2-norm over a list of gradients, and the list
times min(1, max_norm / (norm + 1e-6)), written to the buffers an optimizer
reads.

``run`` computes a case in elementary torch operations where ``own`` is
false and through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
CLIP_EPS = 1e-6


def _block(name, op, rows, hidden, dtype, res, post, gate_rows, nxt, offset=0, res_scale=1.0,
           branch_scale=1.0, eps=1e-5):
    return {"name": name, "op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "res": res,
            "post": post, "gate_rows": gate_rows, "next": nxt, "offset": offset,
            "res_scale": res_scale, "branch_scale": branch_scale, "eps": eps}


def _grads(name, op, tensors, total, sizes, dtype, out, pad, max_norm):
    return {"name": name, "op": op, "tensors": tensors, "total": total, "sizes": sizes,
            "dtype": dtype, "out": out, "pad": pad, "max_norm": max_norm}


def listed():
    return [
        # one decoding step of a batch of eight: both norms around the residual sum
        _block("block fwd 8x4096 bf16", "block_fwd", 8, 4096, "bf16", "bf16", True, 0, True, 1),
        # training, 4 sequences of 1024 tokens: both norms and a per-channel gate
        _block("block fwd 4096x4096 bf16", "block_fwd", 4096, 4096, "bf16", "bf16", True, 1, True,
               1, 1.0, 1.0, 1e-6),
        # odd widths (a pruned model), a gate for each of 8 sequences, fp16
        _block("block fwd 1000x1001 f16", "block_fwd", 1000, 1001, "f16", "f16", True, 8, True),
        # a large batch with the residual stream kept in fp32: residual sum and the next norm
        _block("block fwd 16384x8192 bf16+f32", "block_fwd", 16384, 8192, "bf16", "f32", False, 0,
               True, 0, 1.0, 0.22),
        # a small fp32 model
        _block("block bwd 256x1024 f32", "block_bwd", 256, 1024, "f32", "f32", True, 1, True, 0,
               1.0, 1.0, 1e-6),
        # training, 4 sequences of 1024 tokens, a gate for each sequence
        _block("block bwd 4096x4096 bf16", "block_bwd", 4096, 4096, "bf16", "bf16", True, 4, True,
               1, 1.0, 0.5, 1e-6),
        # the odd width, without a gate, fp32 residual stream
        _block("block bwd 777x1001 f16+f32", "block_bwd", 777, 1001, "f16", "f32", True, 0, True),
        # a large batch, everything
        _block("block bwd 16384x8192 bf16", "block_bwd", 16384, 8192, "bf16", "bf16", True, 1,
               True, 0, 0.5, 1.0),
        # the norm weights of a few layers, clipped before their update
        _grads("clip 9 f32, 37 K", "clip", 9, 36864, 1, "f32", "f32", 64, 1.0),
        # the norm over the fp32 gradients of many parameters of mixed sizes, biases among them
        _grads("norm 300 f32, 200 M", "norm", 300, 200_000_000, 2, "f32", "", 0, 1.0),
        # odd bf16 gradients clipped into an optimizer's packed fp32 buffer
        _grads("clip 61 bf16->f32, 30 M odd", "clip", 61, 30_000_001, 3, "bf16", "f32", 1, 1.0),
        # bf16 gradients of a large model's shard, clipped into an fp32 buffer
        _grads("clip 150 bf16->f32, 250 M", "clip", 150, 250_000_000, 4, "bf16", "f32", 64, 1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("block_fwd", "block_bwd", "block_fwd", "block_bwd", "clip", "norm"))
    if kind in ("block_fwd", "block_bwd"):
        hidden = _log_int(rng, 128, 8192)
        if rng.random() < 0.75:
            hidden = max(128, hidden // 64 * 64)
        rows = _log_int(rng, 1, 16384)
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        # four bytes an element in half the rows: no more than the largest listed case
        res = "f32" if dtype == "f32" or rng.random() < 0.3 else dtype
        if res == "f32":
            rows = max(1, rows // 2)
        post, nxt = rng.choice(((True, True), (True, True), (False, True), (True, False)))
        gate_rows = rng.choice((0, 1, 1, 2, 4, 8))
        if gate_rows > 1:
            rows = -(-rows // gate_rows) * gate_rows
        case = _block("", kind, rows, hidden, dtype, res, post, gate_rows, nxt, rng.choice((0, 1)),
                      rng.choice((1.0, 1.0, 0.5)), rng.choice((1.0, 1.0, 0.25)),
                      rng.choice((1e-5, 1e-6)))
    else:
        tensors = _log_int(rng, 1, 300)
        total = max(tensors, _log_int(rng, 1000, 150_000_000))
        dtype, out = rng.choice((("bf16", "f32"), ("f16", "f32"), ("f32", "f32"),
                                 ("bf16", "bf16")))
        case = _grads("", kind, tensors, total, rng.randrange(1 << 20), dtype,
                      out if kind == "clip" else "", rng.choice((1, 64, 64)) if kind == "clip"
                      else 0, rng.choice((1.0, 1.0, 1e6)))
    del case["name"]
    return case


def _sizes(case):
    """Element counts of the list: log-uniform shares over three decades of
    the total, every one at least 1."""
    rng = random.Random(case["sizes"])
    w = [math.exp(rng.uniform(0.0, math.log(1000.0))) for _ in range(case["tensors"])]
    spare = case["total"] - case["tensors"]
    got = [1 + int(spare * v / sum(w)) for v in w]
    got[rng.randrange(len(got))] += case["total"] - sum(got)
    return got


def _randn(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(std).add_(mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("clip", "norm"):
        return _prepare_grads(case, gen)
    t, ts = DTYPES[case["dtype"]], DTYPES[case["res"]]
    shape, hidden = (case["rows"], case["hidden"]), case["hidden"]
    mean = 0.0 if case["offset"] else 1.0
    s = dict(case)
    s["x"] = _randn(gen, shape, t, 1.5)
    s["residual"] = _randn(gen, shape, ts, 2.0)
    s["post_gamma"] = _randn(gen, (hidden,), t, 0.1, mean) if case["post"] else None
    s["next_gamma"] = _randn(gen, (hidden,), t, 0.1, mean) if case["next"] else None
    s["gate"] = (_randn(gen, (case["gate_rows"], hidden), t, 0.3, 0.6)
                 if case["gate_rows"] else None)
    if case["op"] == "block_bwd":
        # what the forward left for the backward, and the gradients from above
        x, r = s["x"].float(), s["residual"].float()
        s["rstd_post"] = _rstd(x, case["eps"]) if case["post"] else None
        r = _stream(s, x, r, s["rstd_post"])
        s["rstd_next"] = _rstd(r, case["eps"]) if case["next"] else None
        s["res_out"] = r.to(ts)
        s["dy"] = _randn(gen, shape, t) if case["next"] else None
        s["dres_out"] = _randn(gen, shape, ts)
        del s["residual"]
    return s


def _prepare_grads(case, gen):
    t = DTYPES[case["dtype"]]
    sizes = _sizes(case)
    grads = [_randn(gen, (n,), t, 10.0 ** -(k % 4)) for k, n in enumerate(sizes)]
    s = dict(case, grads=grads)
    if case["op"] == "clip":
        # the optimizer's flat buffer; each parameter starts on a multiple of `pad` elements
        at = [0]
        for n in sizes:
            at.append(-(-(at[-1] + n) // case["pad"]) * case["pad"])
        s["flat"] = torch.zeros(at[-1], dtype=DTYPES[case["out"]], device="cuda")
        s["out"] = [s["flat"][a:a + n] for a, n in zip(at, sizes)]
    return s


def _gain(w, offset):
    return w.float() + float(offset)


def _rstd(v, eps):
    return torch.rsqrt((v * v).mean(-1) + eps)


def _gate_of(s, rows):
    """The gate row of every row, as [groups, 1, hidden] against [groups, rows / groups, hidden]."""
    return s["gate"].float().unsqueeze(1), (s["gate"].shape[0], rows // s["gate"].shape[0], -1)


def _stream(s, x, residual, rstd_post):
    z = x
    if rstd_post is not None:
        z = x * rstd_post[:, None] * _gain(s["post_gamma"], s["offset"])
    if s["gate"] is not None:
        gate, split = _gate_of(s, x.shape[0])
        z = (z.view(split) * gate).view(x.shape)
    return s["res_scale"] * residual + s["branch_scale"] * z


def run(state):
    op = state["op"]
    if own:
        return _run_own(state, op)
    if op == "block_fwd":
        return _plain_fwd(state)
    if op == "block_bwd":
        return _plain_bwd(state)
    flat = torch.cat([g.view(-1).float() for g in state["grads"]])
    norm = flat.double().square().sum().sqrt()
    if op == "norm":
        return norm.float()
    factor = (state["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    flat *= factor
    torch._foreach_copy_(state["out"], list(flat.split([g.numel() for g in state["grads"]])))
    return norm.float(), state["flat"]


def _run_own(s, op):
    import bwd_rms_norm_gb300 as rmsn

    if op == "block_fwd":
        return rmsn.rms_norm_block_fwd(
            s["x"], s["residual"], post_gamma=s["post_gamma"], gate=s["gate"],
            next_gamma=s["next_gamma"], eps=s["eps"], offset=s["offset"],
            residual_scale=s["res_scale"], branch_scale=s["branch_scale"])
    if op == "block_bwd":
        return rmsn.rms_norm_block_bwd(
            s["dy"], s["dres_out"], s["x"], s["res_out"], s["rstd_post"], s["rstd_next"],
            post_gamma=s["post_gamma"], gate=s["gate"], next_gamma=s["next_gamma"],
            offset=s["offset"], residual_scale=s["res_scale"], branch_scale=s["branch_scale"])
    if op == "norm":
        return rmsn.rms_norm_grad_norm(s["grads"])
    norm = rmsn.rms_norm_grad_clip(s["grads"], s["max_norm"], eps=CLIP_EPS, out=s["out"])
    return norm, s["flat"]


def _plain_fwd(s):
    t, ts = s["x"].dtype, s["residual"].dtype
    x = s["x"].float()
    rstd_post = _rstd(x, s["eps"]) if s["post"] else None
    r = _stream(s, x, s["residual"].float(), rstd_post)
    if not s["next"]:
        return r.to(ts), None, rstd_post, None
    rstd_next = _rstd(r, s["eps"])
    y = r * rstd_next[:, None] * _gain(s["next_gamma"], s["offset"])
    return r.to(ts), y.to(t), rstd_post, rstd_next


def _plain_bwd(s):
    t, ts = s["x"].dtype, s["res_out"].dtype
    x = s["x"].float()
    d = s["dres_out"].float()
    dnext = None
    if s["next"]:
        rs = s["rstd_next"][:, None]
        rh = s["res_out"].float() * rs
        dy = s["dy"].float()
        g = dy * _gain(s["next_gamma"], s["offset"])
        d = d + rs * (g - rh * (g * rh).mean(-1, keepdim=True))
        dnext = (dy * rh).sum(0)
    dres = (s["res_scale"] * d).to(ts)
    db = s["branch_scale"] * d
    xh, z = x, x
    if s["post"]:
        xh = x * s["rstd_post"][:, None]
        z = xh * _gain(s["post_gamma"], s["offset"])
    dz, dgate = db, None
    if s["gate"] is not None:
        gate, split = _gate_of(s, x.shape[0])
        dgate = (db * z).view(split).sum(1)
        dz = (db.view(split) * gate).view(x.shape)
    dx, dpost = dz, None
    if s["post"]:
        dpost = (dz * xh).sum(0)
        g = dz * _gain(s["post_gamma"], s["offset"])
        dx = s["rstd_post"][:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(t), dres, dpost, dgate, dnext


def work(case):
    if case["op"] in ("clip", "norm"):
        n = case["total"]
        b = n * BYTES[case["dtype"]] + 4
        if case["op"] == "norm":
            return {"bytes": b, "flops": 2 * n}
        return {"bytes": b + n * BYTES[case["out"]], "flops": 3 * n}
    rows, hidden = case["rows"], case["hidden"]
    n, t, ts = rows * hidden, BYTES[case["dtype"]], BYTES[case["res"]]
    norms = int(case["post"]) + int(case["next"])
    params = (norms + case["gate_rows"]) * hidden
    if case["op"] == "block_fwd":
        # read x, the residual, the weights; write the stream, y, the row statistics
        b = n * (t + 2 * ts + (t if case["next"] else 0)) + params * t + 4 * rows * norms
        return {"bytes": b, "flops": n * (4 + 4 * norms)}
    # read x, the gradients, the stream (next norm), statistics, weights; write dx, dres and fp32 sums
    b = n * (2 * t + 2 * ts + ((t + ts) if case["next"] else 0))
    return {"bytes": b + params * (t + 4) + 4 * rows * norms, "flops": n * (4 + 9 * norms)}


def exact(case, seed):
    """What ``run`` returns, in 64 bits from the definitions: the forward
    written with norms of the rows, the backward as the derivative's inner
    products, row by row."""
    s = prepare(case, seed)
    if case["op"] in ("clip", "norm"):
        total = torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]])
        total = torch.linalg.vector_norm(total)
        if case["op"] == "norm":
            return total
        want = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
        factor = 1.0 if float(total) + CLIP_EPS <= case["max_norm"] else (
            case["max_norm"] / (float(total) + CLIP_EPS))
        for o, g in zip(s["out"], s["grads"]):
            a = o.storage_offset()
            want[a:a + g.numel()] = g.double() * factor
        return total, want
    rows, hidden, dbl = case["rows"], case["hidden"], torch.float64
    one = torch.ones(hidden, dtype=dbl, device="cuda")
    w1 = s["post_gamma"].to(dbl) + case["offset"] if case["post"] else one
    w2 = s["next_gamma"].to(dbl) + case["offset"] if case["next"] else None
    groups = max(1, case["gate_rows"])
    gate = s["gate"].to(dbl) if case["gate_rows"] else one[None]
    gate = gate.repeat_interleave(rows // groups, dim=0) if groups > 1 else gate
    mix = gate * w1 * case["branch_scale"]  # d stream / d x_hat
    x = s["x"].to(dbl)
    if case["op"] == "block_fwd":
        r1 = (x.norm(dim=1).square() / hidden + case["eps"]).pow(-0.5) if case["post"] else None
        if case["post"]:
            x = x * r1[:, None]
        r = case["res_scale"] * s["residual"].to(dbl) + mix * x
        if w2 is None:
            return r, None, r1, None
        r2 = (r.norm(dim=1).square() / hidden + case["eps"]).pow(-0.5)
        return r, r * r2[:, None] * w2, r1, r2
    d = s["dres_out"].to(dbl)
    dw2 = None
    if w2 is not None:
        r2 = s["rstd_next"].to(dbl)
        rh, dy = s["res_out"].to(dbl) * r2[:, None], s["dy"].to(dbl)
        inner = torch.einsum("ij,ij->i", dy * w2, rh) / hidden
        d = d + (dy * w2 - rh * inner[:, None]) * r2[:, None]
        dw2 = torch.einsum("ij,ij->j", dy, rh)
    dres = case["res_scale"] * d
    xh = x * s["rstd_post"].to(dbl)[:, None] if case["post"] else x
    byrow = (d * xh).view(groups, rows // groups, hidden).sum(1) * case["branch_scale"]
    dgate = byrow * w1 if case["gate_rows"] else None
    if not case["post"]:
        return d * mix, dres, None, dgate, dw2
    dw1 = (byrow * (s["gate"].to(dbl) if case["gate_rows"] else 1.0)).sum(0)
    g = d * mix
    dx = (g - xh * (torch.einsum("ij,ij->i", g, xh) / hidden)[:, None])
    return dx * s["rstd_post"].to(dbl)[:, None], dres, dw1, dgate, dw2
